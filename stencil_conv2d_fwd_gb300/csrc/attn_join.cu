// Joins partial attention results of disjoint parts of the keys:
//   m = max_i m_i,  l = sum_i l_i 2^(m_i - m),  out = sum_i o_i 2^(m_i - m) / l
// in an order that the sizes alone give, so the result does not depend on
// which part finished first.  Bound by reading the partials: a thread has four
// elements of a row; with many parts, `groups` threads share them, each every
// groups-th part, and are joined in order.
#include <cuda_bf16.h>

#include "attn.h"
#include "launch.h"

namespace sc {

namespace {

constexpr int kJoinThreads = 256;
constexpr int kAhead = 8;

// m, l, o <- joined with (m2, l2, o2)
__device__ __forceinline__ void join4(float &m, float &l, float4 &o, float m2, float l2, const float4 &o2)
{
    const float mm = fmaxf(m, m2), ms = mm == -INFINITY ? 0.f : mm;
    const float f1 = ex2(m - ms), f2 = ex2(m2 - ms);
    m = mm;
    l = l * f1 + l2 * f2;
    o.x = o.x * f1 + o2.x * f2;
    o.y = o.y * f1 + o2.y * f2;
    o.z = o.z * f1 + o2.z * f2;
    o.w = o.w * f1 + o2.w * f2;
}

struct JoinGeom {
    int quads;    // D / 4: threads of a row and group
    int groups;   // threads that share a row's parts
    int rows;     // rows of a CTA: quads * groups * rows <= kJoinThreads
};

template <bool BF16>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const AttnArgs a, const AttnPartials p, const JoinGeom g)
{
    __shared__ float4 so[kJoinThreads];
    __shared__ float2 sml[kJoinThreads];
    pdl_wait();
    const int rows = a.Tq * a.G;
    const long long nrow = (long long)a.N * a.Hkv * rows;
    const int c = threadIdx.x % g.quads, grp = threadIdx.x / g.quads % g.groups, r = threadIdx.x / (g.quads * g.groups);
    const long long at0 = (long long)blockIdx.x * g.rows + r;
    const bool act = r < g.rows && at0 < nrow;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (act) {
        // kAhead parts' loads at a time
        for (int i0 = grp; i0 < p.parts; i0 += kAhead * g.groups) {
            float2 ml[kAhead];
            float4 q[kAhead];
            float mm = m;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = i0 + k * g.groups;
                const long long at = i * nrow + at0;
                ml[k] = i < p.parts ? p.ml[at] : make_float2(-INFINITY, 0.f);
                q[k] = i < p.parts ? *reinterpret_cast<const float4 *>(p.o + at * a.D + 4 * c) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) mm = fmaxf(mm, ml[k].x);
            const float ms = mm == -INFINITY ? 0.f : mm, f0 = ex2(m - ms);
            l *= f0;
            o = make_float4(o.x * f0, o.y * f0, o.z * f0, o.w * f0);
            m = mm;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const float f = ex2(ml[k].x - ms);
                l = fmaf(ml[k].y, f, l);
                o.x = fmaf(q[k].x, f, o.x);
                o.y = fmaf(q[k].y, f, o.y);
                o.z = fmaf(q[k].z, f, o.z);
                o.w = fmaf(q[k].w, f, o.w);
            }
        }
    }
    if (g.groups > 1) {
        so[threadIdx.x] = o;
        sml[threadIdx.x] = make_float2(m, l);
        __syncthreads();
        if (!act || grp != 0) return;
        for (int j = 1; j < g.groups; ++j) {
            const int e = threadIdx.x + j * g.quads;
            join4(m, l, o, sml[e].x, sml[e].y, so[e]);
        }
    }
    if (!act) return;
    const int nh = (int)(at0 / rows), row = (int)(at0 - (long long)nh * rows);
    const int n = nh / a.Hkv, h = nh % a.Hkv;
    const int t = row / a.G, hq = h * a.G + row % a.G;
    const long long oat = n * a.os.n + t * a.os.t + hq * a.os.h + 4 * c;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const float y[4] = {l == 0.f ? 0.f : o.x * inv, l == 0.f ? 0.f : o.y * inv, l == 0.f ? 0.f : o.z * inv,
                        l == 0.f ? 0.f : o.w * inv};
    if constexpr (BF16) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(y[0], y[1]), hi = __floats2bfloat162_rn(y[2], y[3]);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + oat) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + oat) = make_float4(y[0], y[1], y[2], y[3]);
    }
    if (c == 0 && a.lse) a.lse[((long long)n * a.Hq + hq) * a.Tq + t] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
}

}  // namespace

cudaError_t launch_attn_join(const AttnArgs &a, bool bf16, const AttnPartials &p, cudaStream_t st)
{
    JoinGeom g;
    g.quads = a.D / 4;
    // a group has at least four parts; more than one only as far as threads go
    g.groups = p.parts / 4;
    if (g.groups > kJoinThreads / g.quads) g.groups = kJoinThreads / g.quads;
    if (g.groups < 1) g.groups = 1;
    g.rows = kJoinThreads / (g.quads * g.groups);
    const long long nrow = (long long)a.N * a.Hkv * a.Tq * a.G;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((nrow + g.rows - 1) / g.rows));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return bf16 ? cudaLaunchKernelEx(&cfg, attn_join_kernel<true>, a, p, g)
                : cudaLaunchKernelEx(&cfg, attn_join_kernel<false>, a, p, g);
}

}  // namespace sc
