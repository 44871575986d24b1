// y = act(x w^T + b) + residual of few rows: a decoder's step.  Bound by reading w
// once, so a warp streams rows of w through registers and keeps all rows' sums; 1 to
// 8 warps of a CTA, and where that is not enough 2 to 8 CTAs of a cluster, share an
// output's Cin and add their parts in order through (distributed) shared memory:
// 16 rows of 4096, 512 outputs in bf16 4.4 us, without clusters 8.7.
//
// bf16, up to 16 rows: warp-wide m16n8k16 MMAs with w as the 16-row operand.  The
// order of summation is free, so lane (g, t) takes whole 16-byte chunks of w's rows g
// and g + 8 and the same chunks of x's row g, with no transposition.  (8 rows, w of
// 8192 x 2048: 7.8 us, 4.3 TB/s.)
// fp32, 5 rows and more: the same, both operands in three bf16 planes, blocks of 16 rows
// that read w from L2 but for one.
// fp32, up to 4 rows: FMA.  A lane takes four elements of Cin of four outputs and
// every row of x (from L1), and the 32 lanes' sums are added by halves: each exchange
// leaves a lane half as many sums.  (1 row, w of 32000 x 512: 13.1 us, 5.0 TB/s; 3
// rows 16.1.)
#include <cuda_bf16.h>

#include "attn_rows.cuh"
#include "common.cuh"
#include "launch.h"
#include "layer.h"
#include "linear.cuh"
#include "tc_common.cuh"

namespace sc {

namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct RowsShare {
    int log2_slices;   // warps that share an output's Cin, in a CTA
    int cluster;       // CTAs that do (each with its own slices; log2_slices is 3 then), 1 to 8
};

// This warp's tile of outputs and its part of `steps`.
struct RowsWork {
    long long tile;
    int s0, s1;
    __device__ __forceinline__ RowsWork(const RowsShare &g, int steps, int warp)
    {
        const int slices = g.cluster << g.log2_slices, rank = blockIdx.x % g.cluster;
        const int slice = (rank << g.log2_slices) + (warp & ((1 << g.log2_slices) - 1));
        tile = (long long)(blockIdx.x / g.cluster) * (kWarps >> g.log2_slices) + (warp >> g.log2_slices);
        s0 = (int)((long long)steps * slice / slices);
        s1 = (int)((long long)steps * (slice + 1) / slices);
    }
};

// The CTA's sums: [tile][slice][row][output], outputs of a tile TO, rows R.  In a
// cluster (one tile a CTA) the first CTA adds those of all, in order, from its own
// shared memory.
template <class T, int TO, int R>
__device__ __forceinline__ void finish_tiles(const LinearArgs &a, const float *sums, const RowsShare &g)
{
    __shared__ float shared_sums[8][R * TO];   // of the cluster's CTAs
    __syncthreads();
    const int slices = 1 << g.log2_slices, tiles = kWarps >> g.log2_slices, rank = blockIdx.x % g.cluster;
    auto cta_sum = [&](int tile, int at) {
        const float *p = sums + tile * slices * R * TO + at;
        float v = 0.f;
        for (int s = 0; s < slices; ++s) v += p[s * R * TO];
        return v;
    };
    if (g.cluster > 1) {
        // (every CTA of the cluster has started: its shared memory may be written)
        cluster_wait();
        for (int e = threadIdx.x; e < R * TO; e += kWarps * 32) remote_store(&shared_sums[rank][e], cta_sum(0, e), true);
        cluster_arrive();
        if (rank != 0) return;
        cluster_wait();
    }
    const long long o0 = (long long)(blockIdx.x / g.cluster) * tiles * TO;
    const long long row0 = (long long)blockIdx.y * R;   // a block of rows
    for (int e = threadIdx.x; e < tiles * R * TO; e += kWarps * 32) {
        const int tile = e / (R * TO), row = e / TO % R, o = e % TO;
        const long long col = o0 + tile * TO + o;
        if (row0 + row >= a.rows || col >= a.Cout) continue;
        float v = 0.f;
        if (g.cluster > 1) {
            for (int c = 0; c < g.cluster; ++c) v += shared_sums[c][e];
        } else {
            v = cta_sum(tile, e - tile * R * TO);
        }
        v = activate<sizeof(T) == 2>(a.b ? v + a.b[col] : v, a.act);
        if (a.residual) v += to_float(static_cast<const T *>(a.residual)[(row0 + row) * a.rs + col]);
        store_as(static_cast<T *>(a.y) + (row0 + row) * a.ys + col, v);
    }
}

// NT: 8 or 16 rows of x.
template <int NT>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 4 : 2) linear_rows_mma_kernel(const LinearArgs a, const RowsShare share)
{
    constexpr int R = 8 * NT, U = 4;
    __shared__ float sums[kWarps * R * 16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    pdl_trigger();   // the next kernel may be set up; it waits for this grid's end
    if (share.cluster > 1) cluster_arrive();
    pdl_wait();
    const RowsWork work(share, (a.Cin + 31) / 32, warp);   // steps of 32 elements: a chunk of 8 for each t
    const long long tile = work.tile;
    const int s0 = work.s0, s1 = work.s1;
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
            for (int i = 0; i < 2; ++i) w[u][i] = on ? ld16_once(wp[i] + (s + u) * 32LL) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = 0; i < NT; ++i)
                x[u][i] = on ? *reinterpret_cast<const uint4 *>(xp[i] + (s + u) * 32LL) : make_uint4(0u, 0u, 0u, 0u);
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
    finish_tiles<__nv_bfloat16, 16, R>(a, sums, share);
}

// Two floats as three pairs of bf16, x = x0 + x1 + x2 to 24 bits.  The first two
// planes are at most bf16's largest value M; an infinity is (M, M, infinity), of
// which the last meets the first plane of the other operand only.
__device__ __forceinline__ void split3(float x, float y, uint32_t (&p)[3])
{
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        p[i] = i < 2 ? pack_bf16_finite(x, y) : tc::pack_bf16(x, y);
        x -= __uint_as_float(p[i] << 16);
        y -= __uint_as_float(p[i] & 0xffff0000u);
    }
}

// fp32 rows on the same MMAs: both operands split in registers, a product the six
// of planes i + j <= 2.  The MMAs cut sums short, so large and small products have
// accumulators of their own, which are moved to sums every FLUSH steps.
// 16 rows, w of 8192 x 2048: 22.0 us (67 MB; steps in twos, the next two on their way:
// one at a time 25.1, two blocks of 16 outputs a warp 33.4, FMA 78.9); 8 rows 19.9 (FMA
// 26.3).
template <int NT>
__global__ void __launch_bounds__(kWarps * 32) linear_rows_split_kernel(const LinearArgs a, const RowsShare share)
{
    constexpr int R = 8 * NT, U = 2, FLUSH = 8;
    __shared__ float sums[kWarps * R * 16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3, row0 = blockIdx.y * R;
    pdl_trigger();   // the next kernel may be set up; it waits for this grid's end
    if (share.cluster > 1) cluster_arrive();
    pdl_wait();
    const RowsWork work(share, (a.Cin + 15) / 16, warp);   // steps of 16 elements: a chunk of 4 for each t
    const int s0 = work.s0, s1 = work.s1;
    const float *wp[2], *xp[NT];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const long long o = work.tile * 16 + g + 8 * i;
        wp[i] = static_cast<const float *>(a.w) + (o < a.Cout ? o : a.Cout - 1LL) * a.ws + t * 4;
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) xp[i] = static_cast<const float *>(a.x) + min(row0 + g + 8 * i, a.rows - 1) * a.xs + t * 4;
    float total[NT][4], big[NT][4], small[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) total[i][j] = big[i][j] = small[i][j] = 0.f;
    auto flush = [&]() {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                total[i][j] += big[i][j] + small[i][j];
                big[i][j] = small[i][j] = 0.f;
            }
    };
    uint4 w[U][2], x[U][NT];
    auto load = [&](int s) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool on = s + u < s1 && (s + u) * 16 + t * 4 < a.Cin;
#pragma unroll
            for (int i = 0; i < 2; ++i) w[u][i] = on ? ld16_once(wp[i] + (s + u) * 16LL) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = 0; i < NT; ++i)
                x[u][i] = on ? *reinterpret_cast<const uint4 *>(xp[i] + (s + u) * 16LL) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    load(s0);
    int since = 0;
    for (int s = s0; s < s1; s += U) {
        uint32_t wl[U][2][3], wh[U][2][3], xl[U][NT][3], xh[U][NT][3];   // the chunks' two halves in planes
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                split3(__uint_as_float(w[u][i].x), __uint_as_float(w[u][i].y), wl[u][i]);
                split3(__uint_as_float(w[u][i].z), __uint_as_float(w[u][i].w), wh[u][i]);
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                split3(__uint_as_float(x[u][i].x), __uint_as_float(x[u][i].y), xl[u][i]);
                split3(__uint_as_float(x[u][i].z), __uint_as_float(x[u][i].w), xh[u][i]);
            }
        }
        load(s + U);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 2; k >= 0; --k)
#pragma unroll
                for (int j = 2 - k; j >= 0; --j)
#pragma unroll
                    for (int i = 0; i < NT; ++i)
                        mma16816(k + j == 0 ? big[i] : small[i], wl[u][0][k], wl[u][1][k], wh[u][0][k], wh[u][1][k], xl[u][i][j],
                                 xh[u][i][j]);
        if (++since == FLUSH / U) {
            flush();
            since = 0;
        }
    }
    flush();
    float *mine = sums + warp * R * 16;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) mine[(i * 8 + 2 * t + (j & 1)) * 16 + g + 8 * (j >> 1)] = total[i][j];
    finish_tiles<float, 16, R>(a, sums, share);
}

// R rows of x, four outputs a warp.
template <int R>
__global__ void __launch_bounds__(kWarps * 32, R <= 2 ? 4 : 3) linear_rows_fma_kernel(const LinearArgs a, const RowsShare share)
{
    constexpr int O = 4, U = 2, V = O * R;
    __shared__ float sums[kWarps * R * O];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_trigger();   // the next kernel may be set up; it waits for this grid's end
    if (share.cluster > 1) cluster_arrive();
    pdl_wait();
    const RowsWork work(share, (a.Cin + 127) / 128, warp);   // steps of 128 elements, four a lane
    const long long tile = work.tile;
    const int s0 = work.s0, s1 = work.s1;
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
            for (int i = 0; i < O; ++i) w[u][i] = on ? ld16_once(wp[i] + (s + u) * 128LL) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool on = s + u < s1 && (s + u) * 128 + lane * 4 < a.Cin;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float4 x = on ? *reinterpret_cast<const float4 *>(xp + min(r, a.rows - 1) * a.xs + (s + u) * 128LL)
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
    finish_tiles<float, O, R>(a, sums, share);
}

template <int TO, class K>
cudaError_t launch(K kernel, const LinearArgs &a, int steps, cudaStream_t st, int rows)
{
    // Warps that share an output's Cin: as many as give every SM 16, two steps each
    // at least; more than a CTA's are a cluster's
    const long long blocks = (a.rows + rows - 1) / rows;
    const long long tiles = ((long long)a.Cout + TO - 1) / TO, want = 16LL * device_sm_count();
    RowsShare g{0, 1};
    while (g.log2_slices < 3 && (tiles * blocks) << g.log2_slices < want && steps >> g.log2_slices >= 4) ++g.log2_slices;
    if (g.log2_slices == 3)
        while (g.cluster < 8 && tiles * blocks * 8 * g.cluster < want && steps / (8 * g.cluster) >= 4) g.cluster *= 2;
    const int per = kWarps >> g.log2_slices;
    const long long ctas = (tiles + per - 1) / per * g.cluster;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_behind(kernel, dim3((unsigned)ctas, (unsigned)blocks), dim3(kWarps * 32), st, g.cluster, a, g);
}

}  // namespace

cudaError_t launch_linear_rows(const LinearArgs &a, bool bf16, cudaStream_t st)
{
    if (bf16) {
        const int steps = (a.Cin + 31) / 32;
        return a.rows <= 8 ? launch<16>(linear_rows_mma_kernel<1>, a, steps, st, 8) : launch<16>(linear_rows_mma_kernel<2>, a, steps, st, 16);
    }
    const int steps = (a.Cin + 127) / 128, steps16 = (a.Cin + 15) / 16;
    if (a.rows <= 1) return launch<4>(linear_rows_fma_kernel<1>, a, steps, st, 1);
    if (a.rows <= 2) return launch<4>(linear_rows_fma_kernel<2>, a, steps, st, 2);
    if (a.rows <= 4) return launch<4>(linear_rows_fma_kernel<4>, a, steps, st, 4);
    if (a.rows <= 8) return launch<16>(linear_rows_split_kernel<1>, a, steps16, st, 8);
    return launch<16>(linear_rows_split_kernel<2>, a, steps16, st, 16);
}

}  // namespace sc
