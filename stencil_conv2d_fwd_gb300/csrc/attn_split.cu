// Copies queries, keys and values to the workspace in the order of the tensor
// cores' tiles: fp32 ones split into three bf16 planes, bf16 ones (whose
// strides the tiles' copies cannot address) as they are.
//   x0 = bf16(x), x1 = bf16(x - x0), x2 = bf16(x - x0 - x1)
// so that x = x0 + x1 + x2 to 24 bits (the differences are exact; under 2^-110
// the last planes are subnormal, and x keeps 2^-134).  A product x y is then
// x0 y0 + x0 y1 + x1 y0 + (x0 y2 + x1 y1 + x2 y0), the terms left out below
// 2^-24 |x y|.  x0 is at most bf16's largest value, which lies below fp32's; the
// rest goes to x1.  An infinity (or NaN) is (0, 0, x): the last plane meets the
// first of the other operand only, so that a finite y gives the infinity of y's
// sign, as in x y, and not the NaN of an infinity times a plane that is 0 or has
// the other sign.  Bound by memory: 4 bytes read and 6 written an element.
#include <cuda_bf16.h>

#include "attn.h"
#include "launch.h"

namespace sc {

namespace {

constexpr int kSplitThreads = 256;

struct SplitPart {
    const void *x;
    uint32_t *y;                 // bf16 planes, plane_words words apart
    long long plane_words;
    HeadStrides s;
    int T, H, G;                 // rows [n][T][H] of x; written as [n][H / G][T][G]
    long long chunks;            // rows * D / 8
};

struct SplitArgs {
    SplitPart p[3];
    int D8;                      // D / 8
};

template <bool BF16>
__global__ void __launch_bounds__(kSplitThreads) attn_split_kernel(const SplitArgs a)
{
    pdl_trigger();   // the attention kernel may be set up; its copies wait for this grid's end
    const SplitPart &p = a.p[blockIdx.y];
    const long long stride = (long long)gridDim.x * kSplitThreads;
    for (long long e = (long long)blockIdx.x * kSplitThreads + threadIdx.x; e < p.chunks; e += stride) {
        const long long row = e / a.D8;
        const int c = (int)(e - row * a.D8);
        const long long nt = row / p.H;
        const int h = (int)(row - nt * p.H), n = (int)(nt / p.T), t = (int)(nt - (long long)n * p.T);
        const long long at = n * p.s.n + t * p.s.t + h * p.s.h + c * 8;
        const long long orow = (((long long)n * (p.H / p.G) + h / p.G) * p.T + t) * p.G + h % p.G;
        uint32_t *dst = p.y + (orow * a.D8 + c) * 4;
        if constexpr (BF16) {
            *reinterpret_cast<uint4 *>(dst) =
                *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.x) + at);
            continue;
        }
        const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(p.x) + at);
        const float4 v0 = src[0], v1 = src[1];
        const float x[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = fabsf(x[i]) < INFINITY ? x[i] : 0.f;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (k == 2) {
                    f[2 * i] = fabsf(x[2 * i]) < INFINITY ? f[2 * i] : x[2 * i];
                    f[2 * i + 1] = fabsf(x[2 * i + 1]) < INFINITY ? f[2 * i + 1] : x[2 * i + 1];
                }
                const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                w[i] = k == 0 ? pack_bf16_finite(f[2 * i], f[2 * i + 1]) : *reinterpret_cast<const uint32_t *>(&b);
                f[2 * i] -= __uint_as_float(w[i] << 16);
                f[2 * i + 1] -= __uint_as_float(w[i] & 0xffff0000u);
            }
            *reinterpret_cast<uint4 *>(dst + k * p.plane_words) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

}  // namespace

cudaError_t launch_attn_split(const AttnArgs &a, bool bf16, void *const (&planes)[3], cudaStream_t st)
{
    SplitArgs s;
    s.D8 = a.D / 8;
    const void *x[3] = {a.q, a.k, a.v};
    const HeadStrides hs[3] = {a.qs, a.ks, a.vs};
    long long most = 0;
    for (int i = 0; i < 3; ++i) {
        SplitPart &p = s.p[i];
        p.x = x[i];
        p.y = static_cast<uint32_t *>(planes[i]);
        p.s = hs[i];
        p.T = i ? a.Tk : a.Tq;
        p.H = i ? a.Hkv : a.Hq;
        p.G = i ? 1 : a.G;
        const long long rows = (long long)a.N * p.T * p.H;
        p.chunks = rows * s.D8;
        p.plane_words = rows * a.D / 2;
        if (p.chunks > most) most = p.chunks;
    }
    long long blocks = (most + kSplitThreads - 1) / kSplitThreads;
    const long long cap = 16LL * device_sm_count();
    if (blocks > cap) blocks = cap;
    if (bf16)
        attn_split_kernel<true><<<dim3((unsigned)blocks, 3), kSplitThreads, 0, st>>>(s);
    else
        attn_split_kernel<false><<<dim3((unsigned)blocks, 3), kSplitThreads, 0, st>>>(s);
    return cudaGetLastError();
}

}  // namespace sc
