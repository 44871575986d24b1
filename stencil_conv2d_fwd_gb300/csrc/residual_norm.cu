// The norm behind a block, its gate, the residual stream and the norm before
// the next block, in one pass over the rows:
//
//   t = post(x),  s = scale * residual + gate * t,  sum = s,  y = pre(s)
//
// Bound by memory: x and residual are read once and sum and y written once; a
// row stays in registers, up to 32 elements a thread, from its reading to its
// writing.  A thread's chunks are 16 bytes whatever the type, so that a warp's
// access is 512 bytes in a row (in chunks of eight fp32, whose halves are an access
// each, 65536 rows of 2048 took 497 us; now 357, 6.0 TB/s).  A mean and a variance are a
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

// 16 bytes of a row: E elements.
template <class T>
constexpr int E = 16 / (int)sizeof(T);

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w)); }
template <class T>
__device__ __forceinline__ float element(const uint4 &v, int i)
{
    if constexpr (sizeof(T) == 4) return __uint_as_float(word(v, i));
    return __uint_as_float(i % 2 == 0 ? word(v, i / 2) << 16 : word(v, i / 2) & 0xffff0000u);
}
template <class T>
__device__ __forceinline__ void store_row16(void *p, const float (&v)[E<T>])
{
    uint4 w;
    if constexpr (sizeof(T) == 4)
        w = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    else
        w = make_uint4(tc::pack_bf16(v[0], v[1]), tc::pack_bf16(v[2], v[3]), tc::pack_bf16(v[4], v[5]), tc::pack_bf16(v[6], v[7]));
    *static_cast<uint4 *>(p) = w;
}
template <int N>
__device__ __forceinline__ void vec(const float *p, int at, float (&v)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 a = *reinterpret_cast<const float4 *>(p + at + i);
        v[i] = a.x, v[i + 1] = a.y, v[i + 2] = a.z, v[i + 3] = a.w;
    }
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

// v <- norm(v) of a row whose elements of this thread are v[NV][N]; chunks past
// the row's end are zero and stay out of the sums.
template <int NV, int N, bool ONE>
__device__ __forceinline__ void norm_row(float (&v)[NV][N], const NormArgs &n, int C, int step, int first, float *slot, int W,
                                         int w, int lane)
{
    if (n.kind == 0) return;
    const float inv_c = 1.f / (float)C;
    if (n.kind == 2) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) sum += v[i][j];
        const float mean = row_sum<ONE>(sum, slot, W, w, lane) * inv_c;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (first + i * step < C) {
#pragma unroll
                for (int j = 0; j < N; ++j) v[i][j] -= mean;
            }
    }
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) sq = fmaf(v[i][j], v[i][j], sq);
    const float r = 1.f / sqrtf(row_sum<ONE>(sq, slot + kMaxWarps, W, w, lane) * inv_c + n.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = first + i * step;
        if (at >= C) continue;
        float g[N];
        if (n.weight) {
            vec(n.weight, at, g);
#pragma unroll
            for (int j = 0; j < N; ++j) v[i][j] *= r * g[j];
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) v[i][j] *= r;
        }
        if (n.bias) {
            vec(n.bias, at, g);
#pragma unroll
            for (int j = 0; j < N; ++j) v[i][j] += g[j];
        }
    }
}

// W warps a row, blockDim.y rows a CTA (ONE: W is 1); NV chunks a thread.
template <class T, int NV, bool ONE>
__global__ void __launch_bounds__(32 * kMaxWarps) residual_norm_kernel(const ResidualNormArgs a)
{
    constexpr int N = E<T>;
    __shared__ float slots[ONE ? 1 : 4 * kMaxWarps];   // a row (a CTA has one): four reductions
    const int lane = threadIdx.x & 31, w = ONE ? 0 : threadIdx.x >> 5, W = ONE ? 1 : blockDim.x >> 5;
    const int row = blockIdx.x * blockDim.y + threadIdx.y;
    pdl_trigger();   // the next kernel may be set up; it waits for this grid's end
    pdl_wait();
    if (row >= a.rows) return;   // whole warps; with several warps a row a CTA has one row
    const int first = threadIdx.x * N, step = blockDim.x * N;
    const T *xp = static_cast<const T *>(a.x) + row * a.xs;
    const T *rp = static_cast<const T *>(a.residual) + (a.residual ? row * a.rs : 0);
    uint4 xr[NV], rr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (first + i * step < a.C) xr[i] = ld16_once(xp + first + i * step);
    if (a.residual) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (first + i * step < a.C) rr[i] = ld16_once(rp + first + i * step);
    }
    float v[NV][N];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) v[i][j] = first + i * step < a.C ? element<T>(xr[i], j) : 0.f;
    norm_row<NV, N, ONE>(v, a.post, a.C, step, first, slots, W, w, lane);
    const float *gate = a.gate ? a.gate + (long long)(row / a.gate_rows) * a.C : nullptr;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = first + i * step;
        if (at >= a.C) continue;
        if (gate) {
            float g[N];
            vec(gate, at, g);
#pragma unroll
            for (int j = 0; j < N; ++j) v[i][j] *= g[j];
        }
        if (a.residual) {
#pragma unroll
            for (int j = 0; j < N; ++j) v[i][j] = fmaf(a.scale, element<T>(rr[i], j), v[i][j]);
        }
    }
    if (a.sum) {   // (after all of the gate's loads, which would wait for the stores)
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (first + i * step < a.C) store_row16<T>(static_cast<T *>(a.sum) + row * a.ss + first + i * step, v[i]);
    }
    if (!a.y) return;
    norm_row<NV, N, ONE>(v, a.pre, a.C, step, first, ONE ? slots : slots + 2 * kMaxWarps, W, w, lane);
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (first + i * step < a.C) store_row16<T>(static_cast<T *>(a.y) + row * a.ys + first + i * step, v[i]);
}

template <class T, int NV>
cudaError_t launch(const ResidualNormArgs &a, int warps, cudaStream_t st)
{
    // a warp a row: four rows a CTA, unless the rows are few
    const int per = warps == 1 && a.rows > 4 * device_sm_count() ? 4 : 1;
    const dim3 block(32 * warps, per), grid((unsigned)((a.rows + per - 1) / per));
    return warps == 1 ? launch_behind(residual_norm_kernel<T, NV, true>, grid, block, st, 1, a)
                      : launch_behind(residual_norm_kernel<T, NV, false>, grid, block, st, 1, a);
}

template <class T>
cudaError_t dispatch(const ResidualNormArgs &a, cudaStream_t st)
{
    const int chunks = a.C / E<T>, most = 32 / E<T>;   // chunks of a thread at most: 32 elements
    // rows that do not fill the GPU: one chunk a thread; else up to 32 elements, so
    // that a row needs few warps (and few barriers)
    int nv = a.rows <= 2 * device_sm_count() ? 1 : most;
    while (nv > 1 && chunks <= 32 * (nv / 2)) nv /= 2;
    int warps = (chunks + 32 * nv - 1) / (32 * nv);
    while (warps > kMaxWarps) {
        nv *= 2;
        warps = (chunks + 32 * nv - 1) / (32 * nv);
    }
    if (nv == 1) return launch<T, 1>(a, warps, st);
    if (nv == 2) return launch<T, 2>(a, warps, st);
    if (nv == 4) return launch<T, 4>(a, warps, st);
    if constexpr (E<T> == 4) return launch<T, 8>(a, warps, st);
    return cudaErrorInvalidValue;   // (bf16: 16384 elements are four chunks of 16 warps)
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualNormArgs &a, bool bf16, cudaStream_t st)
{
    return bf16 ? dispatch<__nv_bfloat16>(a, st) : dispatch<float>(a, st);
}

}  // namespace sc
