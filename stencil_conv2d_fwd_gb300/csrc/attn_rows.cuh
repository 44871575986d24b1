// The end of the kernels for few rows (attn_rows.cu, attn_mma.cu): joins the
// (m, l, o) of the CTA's warps, then, in the cluster's first CTA, those that
// the others have stored there (distributed shared memory), and writes the
// output, or one partial result a CTA.  Every join is in a fixed order.
#pragma once

#include <cuda_bf16.h>

#include "attn.h"
#include "launch.h"

namespace sc {

constexpr int kRowWarps = 8;
constexpr int kRowThreads = 32 * kRowWarps;
constexpr int kMaxCluster = 8;

struct RowsGeom {
    int splits;      // CTAs per row block
    int cluster;     // splits, or 1
    int row_blocks;
};

// Shared memory of R rows of DP sums: the warps', and, in the cluster's first
// CTA, those of its CTAs.  The other CTAs may write the latter as soon as the
// first has arrived at the cluster's barrier (cluster_arrive).
template <int R, int DP>
struct WarpSums {
    float o[kRowWarps][R][DP];
    float m[kRowWarps][R], l[kRowWarps][R];
};
template <int R, int DP>
struct CtaSums {
    float o[kMaxCluster][R][DP];
    float m[kMaxCluster][R], l[kMaxCluster][R];
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory"); }

// Stores v at p's place in the shared memory of the cluster's first CTA
// (`remote`), or in the CTA's own.
__device__ __forceinline__ void remote_store(float *p, float v, bool remote)
{
    if (!remote) {
        *p = v;
        return;
    }
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;\n" : "=r"(there) : "r"(at));
    asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(there), "f"(v) : "memory");
}

__device__ __forceinline__ uint4 ldg16(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ void store_out(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_out(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// Every thread of the CTA calls this, its warps' sums written (m in units of
// log2) and cluster_arrive called, by when `cs` is no longer used for anything
// else.  Row r of the block is row0 + r of (sequence, key head) nh.
template <class T, int R, int DP>
__device__ __forceinline__ void finish_rows(const WarpSums<R, DP> &sm, CtaSums<R, DP> &cs, const AttnArgs &a, const RowsGeom &g,
                                            const AttnPartials &part, int nh, int row0, int split)
{
    const int tid = threadIdx.x, rows = a.Tq * a.G;
    const int n = nh / a.Hkv, h = nh - n * a.Hkv;
    const int live = min(R, rows - row0);
    const int C = g.cluster, rank = split % C;
    __syncthreads();
    // the CTA's sums, into its place in the shared memory of the cluster's first CTA
    if (C > 1) cluster_wait();
    for (int e = tid; e < live * DP; e += kRowThreads) {
        const int r = e / DP, d = e % DP;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) mm = fmaxf(mm, sm.m[w][r]);
        const float ms = mm == -INFINITY ? 0.f : mm;
        float ls = 0.f, os = 0.f;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) {
            const float f = ex2(sm.m[w][r] - ms);
            ls = fmaf(sm.l[w][r], f, ls);
            os = fmaf(sm.o[w][r][d], f, os);
        }
        remote_store(&cs.o[rank][r][d], os, C > 1);
        if (d == 0) {
            remote_store(&cs.m[rank][r], mm, C > 1);
            remote_store(&cs.l[rank][r], ls, C > 1);
        }
    }
    if (C > 1) {
        // the others are done once their stores are under way: only the first waits for them
        cluster_arrive();
        if (rank != 0) return;
        cluster_wait();
    } else {
        __syncthreads();
    }
    for (int e = tid; e < live * DP; e += kRowThreads) {
        const int r = e / DP, d = e % DP, row = row0 + r;
        float mm = -INFINITY;
        float mc[kMaxCluster], lc[kMaxCluster], oc[kMaxCluster];
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
            if (c < C) {
                mc[c] = cs.m[c][r];
                lc[c] = cs.l[c][r];
                oc[c] = cs.o[c][r][d];
                mm = fmaxf(mm, mc[c]);
            }
        }
        const float ms = mm == -INFINITY ? 0.f : mm;
        float ls = 0.f, os = 0.f;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
            if (c < C) {
                const float f = ex2(mc[c] - ms);
                ls = fmaf(lc[c], f, ls);
                os = fmaf(oc[c], f, os);
            }
        }
        if (d < a.D) {
            const int t = row / a.G, hq = h * a.G + row % a.G;
            if (part.parts > 0) {
                const long long at = ((long long)split * a.N * a.Hkv + nh) * rows + row;
                part.o[at * a.D + d] = os;
                if (d == 0) part.ml[at] = make_float2(mm, ls);
            } else {
                store_out(static_cast<T *>(a.out) + n * a.os.n + t * a.os.t + hq * a.os.h + d, ls == 0.f ? 0.f : os / ls);
                if (d == 0 && a.lse)
                    a.lse[((long long)n * a.Hq + hq) * a.Tq + t] = ls == 0.f ? -INFINITY : mm * kLn2 + logf(ls);
            }
        }
    }
}

// Launches `kernel` over row blocks of R rows with enough CTAs for each that
// there is one for every SM, none with fewer than `step` keys.  Up to 8 CTAs
// of a row block are a cluster, which joins their sums itself; more write
// partial results for a second kernel.  Measured: 32 x 4 key heads over up to
// 3136 bf16 states 18.4 us (two CTAs for every SM 20.7, four 28.4: a CTA's
// start and end cost what it reads in 1 us); one key head over 921600 states
// 45.9 us (two 50.7; in clusters of 8, which leave SMs of a processing cluster
// idle, 67); 8 x 4 fp32 key heads over 16384 states in clusters 26.7 us, as
// partial results 38.9.
template <class K>
cudaError_t launch_rows_kernel(K kernel, const AttnArgs &a, bool bf16, int R, int step, int smem, cudaStream_t st)
{
    const long long rows = (long long)a.Tq * a.G;
    RowsGeom g;
    g.row_blocks = (int)((rows + R - 1) / R);
    const long long blocks = (long long)a.N * a.Hkv * g.row_blocks;
    const long long want = (device_sm_count() + blocks - 1) / blocks;
    const long long most = ((long long)a.Tk + step - 1) / step;
    const long long s = want < most ? want : most;
    if (s <= kMaxCluster) {
        g.cluster = 1;
        while (g.cluster < s) g.cluster *= 2;
        g.splits = g.cluster;
    } else {
        g.cluster = 1;
        g.splits = (int)s;
    }
    if (blocks * g.splits > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    AttnPartials part{nullptr, nullptr, 0};
    void *ws = nullptr;
    if (g.splits > g.cluster) {
        part.parts = g.splits / g.cluster;
        const size_t nrow = (size_t)part.parts * a.N * a.Hkv * rows;
        const cudaError_t e = workspace_alloc(&ws, nrow * ((size_t)a.D * 4 + sizeof(float2)), st);
        if (e != cudaSuccess) return e;
        part.o = static_cast<float *>(ws);   // rows of D floats: 16-byte aligned
        part.ml = reinterpret_cast<float2 *>(part.o + nrow * a.D);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks * g.splits));
    cfg.blockDim = dim3(kRowThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = g.cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = g.cluster > 1 ? 1 : 0;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a, g, part);
    if (e == cudaSuccess && part.parts > 0) e = launch_attn_join(a, bf16, part, st);
    if (ws) {
        const cudaError_t ef = workspace_free(ws, st);
        if (e == cudaSuccess) e = ef;
    }
    return e;
}

}  // namespace sc
