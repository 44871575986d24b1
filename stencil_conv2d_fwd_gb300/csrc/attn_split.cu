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
#include "layer.h"

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
__device__ __forceinline__ void split_part(const SplitPart &p, int D8)
{
    const long long stride = (long long)gridDim.x * kSplitThreads;
    for (long long e = (long long)blockIdx.x * kSplitThreads + threadIdx.x; e < p.chunks; e += stride) {
        const long long row = e / D8;
        const int c = (int)(e - row * D8);
        const long long nt = row / p.H;
        const int h = (int)(row - nt * p.H), n = (int)(nt / p.T), t = (int)(nt - (long long)n * p.T);
        const long long at = n * p.s.n + t * p.s.t + h * p.s.h + c * 8;
        const long long orow = (((long long)n * (p.H / p.G) + h / p.G) * p.T + t) * p.G + h % p.G;
        uint32_t *dst = p.y + (orow * D8 + c) * 4;
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

template <bool BF16>
__global__ void __launch_bounds__(kSplitThreads) attn_split_kernel(const SplitArgs a)
{
    pdl_trigger();   // the attention kernel may be set up; its copies wait for this grid's end
    split_part<BF16>(a.p[blockIdx.y], a.D8);
}

// 8-bit states for the tensor cores: codes as bf16, or fp16 (the values of bf16
// tensors), which hold every one exactly (0 for states that are not valid), and the factor of each 16 keys, which lie in
// one block:
//   keys    scale of the block * scale * log2 e, fp32's smallest normal number where it is smaller (so that
//           it times an infinity, the score of a key that is not valid, is not NaN)
//   values  the block's scale
// Groups without a valid state get that smallest number and 0, whatever their scale
// is.  Bound by memory: a byte read and two written an element.
struct ExpandArgs {
    AttnQ8Args a;
    SplitPart q;                 // chunks 0: not copied
    int D8;
    uint32_t *k, *v;
    float *k_factor, *v_factor;
    int groups;
    long long rows;              // N * Hkv * Tk
    float scale;                 // scale log2 e
};

template <bool E4M3>
__device__ __forceinline__ uint32_t pair_to_bf16(uint32_t two)   // the two low bytes
{
    if constexpr (E4M3) {
        uint32_t h;
        asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %1;\ncvt.rn.f16x2.e4m3x2 %0, l;\n}\n" : "=r"(h) : "r"(two));
        float lo, hi;
        asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\ncvt.f32.f16 %0, l;\ncvt.f32.f16 %1, h;\n}\n" : "=f"(lo), "=f"(hi) : "r"(h));
        const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&b);
    } else {
        // 2^23 + (x + 128) in fp32, less 2^23 + 128: exact, and its upper half is the bf16
        const uint32_t u = two ^ 0x8080u;
        const float lo = __uint_as_float(0x4b000000u | (u & 0xffu)) - 8388736.f;
        const float hi = __uint_as_float(0x4b000000u | (u >> 8 & 0xffu)) - 8388736.f;
        return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
    }
}

template <bool E4M3>
__device__ __forceinline__ uint32_t pair_to_f16(uint32_t two)
{
    uint32_t h;
    if constexpr (E4M3) {
        asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %1;\ncvt.rn.f16x2.e4m3x2 %0, l;\n}\n" : "=r"(h) : "r"(two));
    } else {
        // 1024 + (x + 128) in fp16, less 1152
        const uint32_t u = __byte_perm(two ^ 0x8080u, 0x64646464u, 0x4140);
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(h) : "r"(u), "r"(0x64806480u));
    }
    return h;
}

template <bool BF16, bool E4M3>
__global__ void __launch_bounds__(kSplitThreads) attn_expand_kernel(const ExpandArgs x)
{
    pdl_trigger();   // the attention kernel may be set up; its copies wait for this grid's end
    if (blockIdx.y == 3) {
        split_part<BF16>(x.q, x.D8);
        return;
    }
    const AttnQ8Args &a = x.a;
    const long long stride = (long long)gridDim.x * kSplitThreads, first = (long long)blockIdx.x * kSplitThreads + threadIdx.x;
    auto length = [&](int n) { return a.k_len ? max(0, min(a.Tk, a.k_len[n])) : a.Tk; };
    if (blockIdx.y == 2) {
        const long long all = (long long)a.N * a.Hkv * x.groups;
        for (long long e = first; e < all; e += stride) {
            const long long nh = e / x.groups;
            const int grp = (int)(e - nh * x.groups), n = (int)(nh / a.Hkv);
            const int t0 = grp * 16, t1 = min(t0 + 16, length(n));
            bool any = t0 < t1;
            if (any && a.key_mask) {
                any = false;
                for (int t = t0; t < t1; ++t) any |= a.key_mask[(long long)n * a.Tk + t] != 0;
            }
            float kf = 0x1p-126f, vf = 0.f;
            if (any) {
                const long long at = nh * a.blocks + (t0 >> a.log2_block);
                kf = a.k_scale[at] * x.scale;
                if (fabsf(kf) < 0x1p-126f) kf = 0x1p-126f;   // (a NaN stays)
                vf = a.v_scale[at];
            }
            x.k_factor[e] = kf;
            x.v_factor[e] = vf;
        }
        return;
    }
    const bool value = blockIdx.y == 1;
    const unsigned char *src = static_cast<const unsigned char *>(value ? a.v : a.k);
    const HeadStrides &s = value ? a.vs : a.ks;
    uint32_t *dst = value ? x.v : x.k;
    const int chunks = a.D / 16;
    const long long all = x.rows * chunks;
    for (long long e = first; e < all; e += stride) {
        const long long row = e / chunks, nh = row / a.Tk;
        const int c = (int)(e - row * chunks), t = (int)(row - nh * a.Tk), n = (int)(nh / a.Hkv), h = (int)(nh - (long long)n * a.Hkv);
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        const bool on = t < length(n) && (!a.key_mask || a.key_mask[(long long)n * a.Tk + t] != 0);
        if (on) w = __ldg(reinterpret_cast<const uint4 *>(src + n * s.n + t * s.t + h * s.h + c * 16));
        const uint32_t b[4] = {w.x, w.y, w.z, w.w};
        uint32_t y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // the values of bf16 tensors meet weights in fp16
            y[2 * i] = !on ? 0u : (BF16 && value ? pair_to_f16<E4M3>(b[i] & 0xffffu) : pair_to_bf16<E4M3>(b[i] & 0xffffu));
            y[2 * i + 1] = !on ? 0u : (BF16 && value ? pair_to_f16<E4M3>(b[i] >> 16) : pair_to_bf16<E4M3>(b[i] >> 16));
        }
        uint4 *out = reinterpret_cast<uint4 *>(dst + e * 8);
        out[0] = make_uint4(y[0], y[1], y[2], y[3]);
        out[1] = make_uint4(y[4], y[5], y[6], y[7]);
    }
}

SplitPart split_part_of(const void *x, void *y, const HeadStrides &s, int N, int T, int H, int G, int D)
{
    const long long rows = (long long)N * T * H;
    return SplitPart{x, static_cast<uint32_t *>(y), rows * D / 2, s, T, H, G, rows * (D / 8)};
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
        if (!planes[i]) {   // not asked for
            s.p[i] = SplitPart{};
            continue;
        }
        s.p[i] = split_part_of(x[i], planes[i], hs[i], a.N, i ? a.Tk : a.Tq, i ? a.Hkv : a.Hq, i ? 1 : a.G, a.D);
        if (s.p[i].chunks > most) most = s.p[i].chunks;
    }
    long long blocks = (most + kSplitThreads - 1) / kSplitThreads;
    const long long cap = 16LL * device_sm_count();
    if (blocks > cap) blocks = cap;
    const dim3 grid((unsigned)blocks, planes[1] ? 3 : 1);
    if (bf16)
        attn_split_kernel<true><<<grid, kSplitThreads, 0, st>>>(s);
    else
        attn_split_kernel<false><<<grid, kSplitThreads, 0, st>>>(s);
    return cudaGetLastError();
}

cudaError_t launch_attn_expand(const AttnQ8Args &a, bool bf16, bool e4m3, void *q, void *k, void *v, float *k_factor, float *v_factor,
                               int groups, cudaStream_t st)
{
    ExpandArgs x;
    x.a = a;
    x.D8 = a.D / 8;
    x.q = q ? split_part_of(a.q, q, a.qs, a.N, a.Tq, a.Hq, a.G, a.D) : SplitPart{};
    x.k = static_cast<uint32_t *>(k);
    x.v = static_cast<uint32_t *>(v);
    x.k_factor = k_factor;
    x.v_factor = v_factor;
    x.groups = groups;
    x.rows = (long long)a.N * a.Hkv * a.Tk;
    x.scale = a.scale * kLog2e;
    long long most = x.rows * (a.D / 16);
    if (x.q.chunks > most) most = x.q.chunks;
    long long blocks = (most + kSplitThreads - 1) / kSplitThreads;
    const long long cap = 16LL * device_sm_count();
    if (blocks > cap) blocks = cap;
    const dim3 grid((unsigned)blocks, q ? 4 : 3);
    if (bf16) {
        if (e4m3)
            attn_expand_kernel<true, true><<<grid, kSplitThreads, 0, st>>>(x);
        else
            attn_expand_kernel<true, false><<<grid, kSplitThreads, 0, st>>>(x);
    } else {
        if (e4m3)
            attn_expand_kernel<false, true><<<grid, kSplitThreads, 0, st>>>(x);
        else
            attn_expand_kernel<false, false><<<grid, kSplitThreads, 0, st>>>(x);
    }
    return cudaGetLastError();
}

}  // namespace sc
