// y = act(x w^T + b) + residual of up to 16 rows: a decoder's step.  Bound by
// reading w once, so a warp streams rows of w through registers and keeps all
// rows' sums; 1 to 8 warps of a CTA share an output's Cin (more where there are
// few outputs) and add their parts in order through shared memory.
//
// bf16: warp-wide m16n8k16 MMAs with w as the 16-row operand.  The order of
// summation is free, so lane (g, t) takes whole 16-byte chunks of w's rows g and
// g + 8 and the same chunks of x's row g, with no transposition.
// fp32: FMA.  A lane takes four elements of Cin of four outputs and every row of
// x (from L1), and the 32 lanes' sums are added by halves: each exchange leaves a
// lane half as many sums.
#include <cuda_bf16.h>

#include "common.cuh"
#include "launch.h"
#include "layer.h"
#include "linear.cuh"

namespace sc {

namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ uint4 ld_once16(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The CTA's sums: [tile][slice][row][output], outputs of a tile TO, rows R.
template <class T, int TO, int R>
__device__ __forceinline__ void finish_tiles(const LinearArgs &a, const float *sums, int log2_slices)
{
    __syncthreads();
    const int slices = 1 << log2_slices, tiles = kWarps >> log2_slices;
    const long long o0 = (long long)blockIdx.x * tiles * TO;
    for (int e = threadIdx.x; e < tiles * R * TO; e += kWarps * 32) {
        const int tile = e / (R * TO), row = e / TO % R, o = e % TO;
        const long long col = o0 + tile * TO + o;
        if (row >= a.rows || col >= a.Cout) continue;
        const float *p = sums + (tile * slices * R + row) * TO + o;
        float v = 0.f;
        for (int s = 0; s < slices; ++s) v += p[s * R * TO];
        v = activate(a.b ? v + __ldg(a.b + col) : v, a.act);
        if (a.residual) v += to_float(static_cast<const T *>(a.residual)[row * a.rs + col]);
        store_as(static_cast<T *>(a.y) + row * a.ys + col, v);
    }
}

// NT: 8 or 16 rows of x.
template <int NT>
__global__ void __launch_bounds__(kWarps * 32) linear_rows_mma_kernel(const LinearArgs a, int log2_slices)
{
    constexpr int R = 8 * NT, U = 4;
    __shared__ float sums[kWarps * R * 16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int slice = warp & ((1 << log2_slices) - 1);
    const long long tile = (long long)blockIdx.x * (kWarps >> log2_slices) + (warp >> log2_slices);
    const int steps = (a.Cin + 31) / 32;   // of 32 elements: a chunk of 8 for each t
    const int s0 = (int)((long long)steps * slice >> log2_slices), s1 = (int)((long long)steps * (slice + 1) >> log2_slices);
    // rows past the end repeat the last one: their sums are not used
    const __nv_bfloat16 *wp[2], *xp[NT];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const long long o = tile * 16 + g + 8 * i;
        wp[i] = static_cast<const __nv_bfloat16 *>(a.w) + (o < a.Cout ? o : a.Cout - 1LL) * a.ws + t * 8;
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
        xp[i] = static_cast<const __nv_bfloat16 *>(a.x) + min(g + 8 * i, a.rows - 1) * a.xs + t * 8;
    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    for (int s = s0; s < s1; s += U) {
        uint4 w[U][2], x[U][NT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool on = s + u < s1 && (s + u) * 32 + t * 8 < a.Cin;
#pragma unroll
            for (int i = 0; i < 2; ++i) w[u][i] = on ? ld_once16(wp[i] + (s + u) * 32LL) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = 0; i < NT; ++i)
                x[u][i] = on ? __ldg(reinterpret_cast<const uint4 *>(xp[i] + (s + u) * 32LL)) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                mma16816(acc[i], w[u][0].x, w[u][1].x, w[u][0].y, w[u][1].y, x[u][i].x, x[u][i].y);
                mma16816(acc[i], w[u][0].z, w[u][1].z, w[u][0].w, w[u][1].w, x[u][i].z, x[u][i].w);
            }
    }
    // acc: outputs g and g + 8 of rows 2 t and 2 t + 1
    float *mine = sums + warp * R * 16;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) mine[(i * 8 + 2 * t + (j & 1)) * 16 + g + 8 * (j >> 1)] = acc[i][j];
    finish_tiles<__nv_bfloat16, 16, R>(a, sums, log2_slices);
}

// R rows of x, four outputs a warp.
template <int R>
__global__ void __launch_bounds__(kWarps * 32) linear_rows_fma_kernel(const LinearArgs a, int log2_slices)
{
    constexpr int O = 4, U = R <= 4 ? 4 : 2, V = O * R;
    __shared__ float sums[kWarps * R * O];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slice = warp & ((1 << log2_slices) - 1);
    const long long tile = (long long)blockIdx.x * (kWarps >> log2_slices) + (warp >> log2_slices);
    const int steps = (a.Cin + 127) / 128;   // of 128 elements, four a lane
    const int s0 = (int)((long long)steps * slice >> log2_slices), s1 = (int)((long long)steps * (slice + 1) >> log2_slices);
    // rows past the end repeat the last one: their sums are not used
    const float *wp[O];
#pragma unroll
    for (int i = 0; i < O; ++i) {
        const long long o = tile * O + i;
        wp[i] = static_cast<const float *>(a.w) + (o < a.Cout ? o : a.Cout - 1LL) * a.ws + lane * 4;
    }
    const float *xp = static_cast<const float *>(a.x) + lane * 4;
    float v[V];   // [row][output]
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.f;
    for (int s = s0; s < s1; s += U) {
        uint4 w[U][O];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool on = s + u < s1 && (s + u) * 128 + lane * 4 < a.Cin;
#pragma unroll
            for (int i = 0; i < O; ++i) w[u][i] = on ? ld_once16(wp[i] + (s + u) * 128LL) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool on = s + u < s1 && (s + u) * 128 + lane * 4 < a.Cin;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float4 x = on ? __ldg(reinterpret_cast<const float4 *>(xp + min(r, a.rows - 1) * a.xs + (s + u) * 128LL))
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < O; ++i) {
                    float &c = v[r * O + i];
                    c = fmaf(x.x, __uint_as_float(w[u][i].x), c);
                    c = fmaf(x.y, __uint_as_float(w[u][i].y), c);
                    c = fmaf(x.z, __uint_as_float(w[u][i].z), c);
                    c = fmaf(x.w, __uint_as_float(w[u][i].w), c);
                }
            }
        }
    }
    // the lanes' sums, by halves: v[0 .. n) are sums base .. base + n
    int base = 0, n = V;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const bool up = lane & d;
        if (n > 1) {
            n /= 2;
#pragma unroll
            for (int i = 0; i < V / 2; ++i)
                if (i < n) {
                    const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, give, d);
                }
            base += up ? n : 0;
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], d);
        }
    }
    // (with fewer sums than lanes, lanes that differ in the last bits hold the same one)
#pragma unroll
    for (int i = 0; i < (V > 32 ? V / 32 : 1); ++i) sums[warp * V + base + i] = v[i];
    finish_tiles<float, O, R>(a, sums, log2_slices);
}

template <int TO, class K>
cudaError_t launch(K kernel, const LinearArgs &a, int steps, cudaStream_t st)
{
    // Warps that share an output's Cin: as many as give every SM 16, two steps each at least
    const long long tiles = ((long long)a.Cout + TO - 1) / TO, want = 16LL * device_sm_count();
    int log2_slices = 0;
    while (log2_slices < 3 && tiles << log2_slices < want && steps >> log2_slices >= 4) ++log2_slices;
    const int per = kWarps >> log2_slices;
    const long long ctas = (tiles + per - 1) / per;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    kernel<<<(unsigned)ctas, kWarps * 32, 0, st>>>(a, log2_slices);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_rows(const LinearArgs &a, bool bf16, cudaStream_t st)
{
    if (bf16) {
        const int steps = (a.Cin + 31) / 32;
        return a.rows <= 8 ? launch<16>(linear_rows_mma_kernel<1>, a, steps, st) : launch<16>(linear_rows_mma_kernel<2>, a, steps, st);
    }
    const int steps = (a.Cin + 127) / 128;
    if (a.rows <= 1) return launch<4>(linear_rows_fma_kernel<1>, a, steps, st);
    if (a.rows <= 2) return launch<4>(linear_rows_fma_kernel<2>, a, steps, st);
    if (a.rows <= 4) return launch<4>(linear_rows_fma_kernel<4>, a, steps, st);
    if (a.rows <= 8) return launch<4>(linear_rows_fma_kernel<8>, a, steps, st);
    return launch<4>(linear_rows_fma_kernel<16>, a, steps, st);
}

}  // namespace sc
