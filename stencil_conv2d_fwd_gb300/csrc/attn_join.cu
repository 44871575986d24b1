// Joins partial attention results of disjoint parts of the keys:
//   m = max_i m_i,  l = sum_i l_i 2^(m_i - m),  out = sum_i o_i 2^(m_i - m) / l
// in the order of i, so the result does not depend on which part finished
// first.  One CTA per row; its threads are (part group, element) pairs.
#include <cuda_bf16.h>

#include "attn.h"
#include "launch.h"

namespace sc {

namespace {

constexpr int kJoinThreads = 256;

template <bool BF16>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const AttnArgs a, const AttnPartials p)
{
    __shared__ float so[kJoinThreads], sl[kJoinThreads], sm[kJoinThreads];
    pdl_wait();
    const int rows = a.Tq * a.G;
    const int row = blockIdx.x % rows, nh = blockIdx.x / rows;
    const int n = nh / a.Hkv, h = nh % a.Hkv;
    const int groups = kJoinThreads / a.D;
    const int d = threadIdx.x % a.D, grp = threadIdx.x / a.D;
    const long long nrow = (long long)a.N * a.Hkv * rows, at0 = (long long)nh * rows + row;
    float m = -INFINITY, l = 0.f, o = 0.f;
    if (grp < groups) {
        for (int i = grp; i < p.parts; i += groups) {
            const long long at = i * nrow + at0;
            const float2 ml = p.ml[at];
            const float oi = p.o[at * a.D + d];
            const float mm = fmaxf(m, ml.x), ms = mm == -INFINITY ? 0.f : mm;
            const float f1 = ex2(m - ms), f2 = ex2(ml.x - ms);
            l = l * f1 + ml.y * f2;
            o = o * f1 + oi * f2;
            m = mm;
        }
    }
    so[threadIdx.x] = o;
    sl[threadIdx.x] = l;
    sm[threadIdx.x] = m;
    __syncthreads();
    if (grp != 0) return;
    for (int j = 1; j < groups; ++j) {
        const int e = j * a.D + d;
        const float mm = fmaxf(m, sm[e]), ms = mm == -INFINITY ? 0.f : mm;
        const float f1 = ex2(m - ms), f2 = ex2(sm[e] - ms);
        l = l * f1 + sl[e] * f2;
        o = o * f1 + so[e] * f2;
        m = mm;
    }
    const int t = row / a.G, hq = h * a.G + row % a.G;
    const long long oat = n * a.os.n + t * a.os.t + hq * a.os.h + d;
    const float y = l == 0.f ? 0.f : o / l;
    if constexpr (BF16)
        static_cast<__nv_bfloat16 *>(a.out)[oat] = __float2bfloat16_rn(y);
    else
        static_cast<float *>(a.out)[oat] = y;
    if (d == 0 && a.lse) a.lse[((long long)n * a.Hq + hq) * a.Tq + t] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
}

}  // namespace

cudaError_t launch_attn_join(const AttnArgs &a, bool bf16, const AttnPartials &p, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)a.N * a.Hkv * a.Tq * a.G));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return bf16 ? cudaLaunchKernelEx(&cfg, attn_join_kernel<true>, a, p)
                : cudaLaunchKernelEx(&cfg, attn_join_kernel<false>, a, p);
}

}  // namespace sc
