// The norm behind a block, its gate, the residual stream and the norm before
// the next block, in one pass over the rows:
//
//   t = post(x),  s = scale * residual + gate * t,  sum = s,  y = pre(s)
//
// Bound by memory: x and residual are read once and sum and y written once; a
// row stays in registers, eight elements a chunk and up to four chunks a
// thread, from its reading to its writing.  A mean and a variance are a
// reduction each (the variance of the elements' distances to the mean, not of
// squares), over the warps of the row.  The vectors (weights, biases, gates) are
// read again for each row, from the caches.
#include <cuda_bf16.h>

#include "common.cuh"
#include "launch.h"
#include "layer.h"
#include "tc_common.cuh"

namespace sc {

namespace {

constexpr int kMaxWarps = 16;   // of a row, and of a CTA

// Eight elements, as stored.
template <class T>
struct Raw8;
template <>
struct Raw8<float> {
    uint4 w[2];
    __device__ __forceinline__ float get(int i) const
    {
        const uint4 &v = w[i / 4];
        return __uint_as_float(i % 4 == 0 ? v.x : (i % 4 == 1 ? v.y : (i % 4 == 2 ? v.z : v.w)));
    }
};
template <>
struct Raw8<__nv_bfloat16> {
    uint4 w[1];
    __device__ __forceinline__ float get(int i) const
    {
        const uint32_t v = i / 2 == 0 ? w[0].x : (i / 2 == 1 ? w[0].y : (i / 2 == 2 ? w[0].z : w[0].w));
        return __uint_as_float(i % 2 == 0 ? v << 16 : v & 0xffff0000u);
    }
};

// (not a read-only load: a row may be written where it was read)
__device__ __forceinline__ uint4 ld_row16(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
template <class T>
__device__ __forceinline__ Raw8<T> load8(const T *p)
{
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.w[i] = ld_row16(reinterpret_cast<const uint4 *>(p) + i);
    return r;
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8])
{
    *reinterpret_cast<uint4 *>(p) = make_uint4(tc::pack_bf16(v[0], v[1]), tc::pack_bf16(v[2], v[3]), tc::pack_bf16(v[4], v[5]),
                                               tc::pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void vec8(const float *p, int at, float (&v)[8])
{
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p + at)), b = __ldg(reinterpret_cast<const float4 *>(p + at) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// Sum over the threads of a row (W warps); `slot` is a row of kMaxWarps floats
// that this reduction alone uses (the next one has another, so one barrier is
// enough).
template <bool ONE>
__device__ __forceinline__ float row_sum(float v, float *slot, int W, int w, int lane)
{
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) v += __shfl_xor_sync(0xffffffffu, v, i);
    if (ONE) return v;
    if (lane == 0) slot[w] = v;
    __syncthreads();
    float sum = 0.f;
    for (int i = 0; i < W; ++i) sum += slot[i];
    return sum;
}

// v <- norm(v) of a row whose elements of this thread are v[NV][8]; chunks past
// the row's end are zero and stay out of the sums.
template <int NV, bool ONE>
__device__ __forceinline__ void norm_row(float (&v)[NV][8], const NormArgs &n, int C, int step, int first, float *slot, int W,
                                         int w, int lane)
{
    if (n.kind == 0) return;
    const float inv_c = 1.f / (float)C;
    if (n.kind == 2) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += v[i][j];
        const float mean = row_sum<ONE>(sum, slot, W, w, lane) * inv_c;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (first + i * step < C) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] -= mean;
            }
    }
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) sq = fmaf(v[i][j], v[i][j], sq);
    const float r = 1.f / sqrtf(row_sum<ONE>(sq, slot + kMaxWarps, W, w, lane) * inv_c + n.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = first + i * step;
        if (at >= C) continue;
        float g[8];
        if (n.weight) {
            vec8(n.weight, at, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] *= r * g[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] *= r;
        }
        if (n.bias) {
            vec8(n.bias, at, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] += g[j];
        }
    }
}

// W warps a row, blockDim.y rows a CTA (ONE: W is 1); NV chunks a thread.
template <class T, int NV, bool ONE>
__global__ void __launch_bounds__(32 * kMaxWarps) residual_norm_kernel(const ResidualNormArgs a)
{
    __shared__ float slots[ONE ? 1 : 4 * kMaxWarps];   // a row (a CTA has one): four reductions
    const int lane = threadIdx.x & 31, w = ONE ? 0 : threadIdx.x >> 5, W = ONE ? 1 : blockDim.x >> 5;
    const int row = blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= a.rows) return;   // whole warps; with several warps a row a CTA has one row
    const int first = threadIdx.x * 8, step = blockDim.x * 8;
    const T *xp = static_cast<const T *>(a.x) + row * a.xs;
    const T *rp = static_cast<const T *>(a.residual) + (a.residual ? row * a.rs : 0);
    Raw8<T> xr[NV], rr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (first + i * step < a.C) xr[i] = load8(xp + first + i * step);
    if (a.residual) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (first + i * step < a.C) rr[i] = load8(rp + first + i * step);
    }
    float v[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = first + i * step < a.C ? xr[i].get(j) : 0.f;
    norm_row<NV, ONE>(v, a.post, a.C, step, first, slots, W, w, lane);
    const float *gate = a.gate ? a.gate + (long long)(row / a.gate_rows) * a.C : nullptr;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = first + i * step;
        if (at >= a.C) continue;
        if (gate) {
            float g[8];
            vec8(gate, at, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] *= g[j];
        }
        if (a.residual) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = fmaf(a.scale, rr[i].get(j), v[i][j]);
        }
        if (a.sum) store8(static_cast<T *>(a.sum) + row * a.ss + at, v[i]);
    }
    if (!a.y) return;
    norm_row<NV, ONE>(v, a.pre, a.C, step, first, ONE ? slots : slots + 2 * kMaxWarps, W, w, lane);
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (first + i * step < a.C) store8(static_cast<T *>(a.y) + row * a.ys + first + i * step, v[i]);
}

template <class T, int NV>
cudaError_t launch(const ResidualNormArgs &a, int warps, cudaStream_t st)
{
    // a warp a row: four rows a CTA, unless the rows are few
    const int per = warps == 1 && a.rows > 4 * device_sm_count() ? 4 : 1;
    const dim3 block(32 * warps, per), grid((unsigned)((a.rows + per - 1) / per));
    if (warps == 1)
        residual_norm_kernel<T, NV, true><<<grid, block, 0, st>>>(a);
    else
        residual_norm_kernel<T, NV, false><<<grid, block, 0, st>>>(a);
    return cudaGetLastError();
}

template <class T>
cudaError_t dispatch(const ResidualNormArgs &a, cudaStream_t st)
{
    const int chunks = a.C / 8;
    // rows that do not fill the GPU: one chunk a thread; else up to four, so
    // that a row needs few warps (and few barriers)
    int nv = a.rows <= 2 * device_sm_count() ? 1 : 4;
    while (nv > 1 && chunks <= 32 * (nv / 2)) nv /= 2;
    int warps = (chunks + 32 * nv - 1) / (32 * nv);
    while (warps > kMaxWarps) {
        nv *= 2;
        warps = (chunks + 32 * nv - 1) / (32 * nv);
    }
    if (nv == 1) return launch<T, 1>(a, warps, st);
    return nv == 2 ? launch<T, 2>(a, warps, st) : launch<T, 4>(a, warps, st);
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualNormArgs &a, bool bf16, cudaStream_t st)
{
    return bf16 ? dispatch<__nv_bfloat16>(a, st) : dispatch<float>(a, st);
}

}  // namespace sc
