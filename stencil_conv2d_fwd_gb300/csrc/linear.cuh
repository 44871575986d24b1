// What the kernels of linear_fwd share: activations, and loads and stores of
// both element types.
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "layer.h"

namespace sc {

// 1 - Phi(z) of the normal distribution, z >= 0, to 13 units of 2^-24 and 1.5 z^2 more (of
// z^2's rounding in the exponent): exp(-z^2 / 2) t P(t) / 2, t = 1 / (1 + 0.4 y), y = z / sqrt 2,
// with P fitted to exp(y^2) erfc(y) / t by weighted least squares in relative error, 5.8e-8 at
// most for y up to 9.6.  0 above z = 13.2, where it is below 2^-126.
__device__ __forceinline__ float normal_tail(float z)
{
    float t;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.28284271247461901f, z, 1.f)));
    float p = fmaf(0.0404752344f, t, -0.136495486f);
    p = fmaf(p, t, 0.0759917572f);
    p = fmaf(p, t, 0.0972286686f);
    p = fmaf(p, t, 0.0732681453f);
    p = fmaf(p, t, 0.196198076f);
    p = fmaf(p, t, 0.201158658f);
    p = fmaf(p, t, 0.226546988f);
    p = fmaf(p, t, 0.225628033f);
    return 0.5f * p * t * ex2(z * z * (-0.5f * kLog2e));
}

// act as sc_act; a NaN stays one.  fp32 gelu takes the tail that v is on, where 1 + erf
// would cancel (nothing is left of that from v = -5.5 on), in no more time: 14401 x 1024 x
// 4096 425 to 432 us, with erff 434, with erfcf 580.
// BF16: an output that is rounded to bf16 next.  gelu then takes the normal distribution
// from Hastings' approximation of erf (Abramowitz and Stegun, "Handbook of Mathematical
// Functions", 7.1.26: off by up to 1.5e-7 of 1, on the negative side by 0.4% of the tail at
// v = -6 and 2% at -10, where that is 10^-9 and 10^-23), one reciprocal, one exponential and
// eight products; with erff the epilogue was what large products waited for (65536 x 2048 x
// 8192: 1545 us, without activation 1258).  silu takes the hardware's exponential and division,
// 2^-16 of itself at most (-87 < v), and 0 below.
template <bool BF16>
__device__ __forceinline__ float activate(float v, int act)
{
    if constexpr (BF16) {
        if (act == 2) {
            const float z = fabsf(v) * 0.70710678118654752f;
            float t, e;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.3275911f, z, 1.f)));
            e = ex2(z * z * -kLog2e);
            float p = fmaf(1.061405429f, t, -1.453152027f);
            p = fmaf(p, t, 1.421413741f);
            p = fmaf(p, t, -0.284496736f);
            p = fmaf(p, t, 0.254829592f);
            const float q = 0.5f * p * t * e;   // 1 - Phi(|v|)
            return v * (v < 0.f ? q : 1.f - q);
        }
        if (act == 3) return __fdividef(v, 1.f + __expf(-v));
    }
    if (act == 1) return v < 0.f ? 0.f : v;
    if (act == 2) {
        const float q = normal_tail(fabsf(v));
        return v * (v < 0.f ? q : 1.f - q);
    }
    if (act == 3) return v / (1.f + expf(-v));
    return v;
}
template <bool BF16>
__device__ __forceinline__ void activate32(float (&v)[32], int act)
{
    if (act == 0) return;
    if (act == 1) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = activate<BF16>(v[j], 1);
    } else if (act == 2) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = activate<BF16>(v[j], 2);
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = activate<BF16>(v[j], 3);
    }
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void store_as(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_as(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ float ld_shared_f32(uint32_t at)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(v) : "r"(at) : "memory");
    return v;
}

}  // namespace sc
