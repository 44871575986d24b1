// What the kernels for few rows have in common (attn_rows.cu, attn_mma.cu): the
// rings that stream the keys and values of the latter, the launch, and the end,
// which joins the (m, l, o) of the CTA's warps, then, in the cluster's first
// CTA, those that the others have stored there (distributed shared memory), and
// writes the output, or one partial result a CTA.  Every join is in a fixed
// order.
#pragma once

#include <cuda_bf16.h>

#include "attn.h"
#include "common.cuh"
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

constexpr int kPiece = 16;   // keys, or values, of a ring entry

// A warp's ring of ENTRIES pieces in shared memory, each kPiece keys or values
// of one (sequence, key head) as rows of DP elements, which its lanes copy there
// asynchronously, 16 bytes each: some 100 to 200 KB are under way on an SM at
// any time without a register held for them and without a barrier between
// warps.  Chunk x of row y lies at chunk x XOR (y mod 8).  States that are not
// valid are not read, and chunks past D neither (their bytes are zero-filled):
// whatever is stored there does not reach a sum.  A warp's pieces are every
// kRowWarps-th of the CTA's share, in the order keys of step 0, values of step
// 0, keys of step 1, ...; ENTRIES - 1 of them are under way.
template <class T, int DP, int ENTRIES>
struct PieceRing {
    static constexpr int EPC = 16 / sizeof(T);              // elements of a chunk
    static constexpr int CH = DP / EPC;                     // chunks of a row
    static constexpr int RPL = 32 / CH;                     // rows of a warp-wide copy
    static constexpr int ENTRY = kPiece * CH;               // in 16-byte units
    static constexpr int LEAD = ENTRIES / 2;                // steps whose keys are under way
    static constexpr int STEP = kRowWarps * kPiece;         // keys from a step to the next
    static_assert(CH <= 32 && LEAD <= 3, "one row at most a copy; a step's valid bits are 16 of a 64-bit word");

    const T *kp, *vp, *kbase, *vbase;   // the lane's part of the next pieces to copy
    long long kst, vst;
    const unsigned char *mb;
    uint4 *ring;
    int len, key0, steps, lane, crow, cch;
    bool cact;
    unsigned long long okq;   // valid bits of the current step and those after it, the current lowest
    int byte;                 // the mask's byte of the step after those
    int entry, fill;          // entries of the piece in use next, and of the next one to be asked for

    __device__ __forceinline__ int mask_byte(int step) const
    {
        const int key = key0 + step * STEP + lane;
        return step < steps && lane < kPiece && key < len ? (mb ? (int)mb[key] : 1) : 0;
    }
    __device__ __forceinline__ void copy(int at, const T *&p, long long pitch, const T *base, uint32_t ok)
    {
        const uint32_t dst = smem_u32(ring + at * ENTRY);
        const T *src = p;
#pragma unroll
        for (int i = 0; i < kPiece / RPL; ++i, src += RPL * pitch) {
            const int row = crow + i * RPL;
            const bool on = cact && (ok >> row & 1u);
            cp_async16(dst + (row * CH + (cch ^ (row & 7))) * 16, on ? src : base, on ? 16 : 0);
        }
        cp_async_commit();
        p += STEP * pitch;
    }
    __device__ __forceinline__ void next_keys(int step)   // of the step LEAD ahead of the current, `step`
    {
        const uint32_t ok = __ballot_sync(0xffffffffu, byte != 0);
        byte = mask_byte(step + LEAD + 1);
        okq |= (unsigned long long)ok << (16 * LEAD);
        copy(fill, kp, kst, kbase, ok);
    }
    __device__ __forceinline__ void next_values()   // of the step (ENTRIES - 1) / 2 ahead
    {
        copy(fill, vp, vst, vbase, (uint32_t)(okq >> (16 * ((ENTRIES - 1) / 2))) & 0xffffu);
    }
    // The CTA's share is the split-th equal part of the sequence's own length.
    __device__ __forceinline__ void begin(uint4 *memory, const AttnArgs &a, int n, int h, int split, int splits, int warp)
    {
        ring = memory;
        lane = threadIdx.x & 31;
        len = a.Tk;
        if (a.k_len) len = max(0, min(len, a.k_len[n]));
        const int pieces = (len + kPiece - 1) / kPiece;
        const int p0 = (int)((long long)pieces * split / splits), p1 = (int)((long long)pieces * (split + 1) / splits);
        steps = p1 - p0 > warp ? (p1 - p0 - warp + kRowWarps - 1) / kRowWarps : 0;
        key0 = (p0 + warp) * kPiece;
        mb = a.key_mask ? a.key_mask + (long long)n * a.Tk : nullptr;
        crow = lane / CH;
        cch = lane % CH;
        cact = cch * EPC < a.D;
        kst = a.ks.t;
        vst = a.vs.t;
        kbase = static_cast<const T *>(a.k);
        vbase = static_cast<const T *>(a.v);
        kp = kbase + n * a.ks.n + h * a.ks.h + (long long)(key0 + crow) * kst + (cact ? cch * EPC : 0);
        vp = vbase + n * a.vs.n + h * a.vs.h + (long long)(key0 + crow) * vst + (cact ? cch * EPC : 0);
        okq = 0;
        entry = 0;
        fill = ENTRIES - 1;
        int b[LEAD];
#pragma unroll
        for (int i = 0; i < LEAD; ++i) b[i] = mask_byte(i);
#pragma unroll
        for (int i = 0; i < LEAD; ++i) {
            const uint32_t ok = __ballot_sync(0xffffffffu, b[i] != 0);
            okq |= (unsigned long long)ok << (16 * i);
            copy(2 * i, kp, kst, kbase, ok);
            if (2 * i + 1 < ENTRIES - 1) copy(2 * i + 1, vp, vst, vbase, ok);
        }
        byte = mask_byte(LEAD);
    }
    // Waits for the next piece, asks for the one ENTRIES - 1 after it (which
    // goes where the piece before it was read: the warp's barrier is behind
    // those reads), and returns it.
    template <bool KEYS>
    __device__ __forceinline__ const uint4 *piece(int step)
    {
        cp_async_wait<ENTRIES - 2>();
        __syncwarp();
        if constexpr (KEYS == (ENTRIES % 2 == 1))
            next_keys(step);
        else
            next_values();
        const uint4 *p = ring + entry * ENTRY;
        entry = entry + 1 == ENTRIES ? 0 : entry + 1;
        fill = fill + 1 == ENTRIES ? 0 : fill + 1;
        return p;
    }
    __device__ __forceinline__ uint32_t valid() const { return (uint32_t)okq & 0xffffu; }
    __device__ __forceinline__ void next_step() { okq >>= 16; }
};

// The rings' memory becomes the warps' sums at the end.  OWN: the cluster's
// sums have their own, so that the first CTA's place is free from the start and
// no CTA waits for another's loop (cluster_arrive at once, else after the loop).
template <class T, int DP, int ENTRIES, int R, bool OWN>
struct RowsShared {
    union {
        uint4 ring[kRowWarps][PieceRing<T, DP, ENTRIES>::ENTRY * ENTRIES];
        struct {
            WarpSums<R, DP> warps;
            CtaSums<OWN ? 1 : R, OWN ? 1 : DP> shared_ctas;
        } sums;
    };
    CtaSums<OWN ? R : 1, OWN ? DP : 1> own_ctas;
    __device__ __forceinline__ CtaSums<R, DP> &ctas()
    {
        if constexpr (OWN)
            return own_ctas;
        else
            return sums.shared_ctas;
    }
};

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
// there is one for every SM, none with less than a step of keys.  Up to 8 CTAs
// of a row block are a cluster, which joins their sums itself; more write
// partial results for a second kernel, unless four steps each of eight CTAs are
// enough.  Measured, calls among others on changing inputs:
//   one key head of 64, one bf16 row over 4000 states: cluster 8.2 us, partial results 10.2
//   8 x 4 of 64, one bf16 row over 16384: 28.6 and 32.5; 8 x 4 of 32, three fp32 rows: 27.1 and 37.9
//   32 x 4 of 64, four bf16 rows over 3136: 23.7 and 26.3; two CTAs for every SM 27.2, four 33.3
//   (a CTA's start and end cost what it reads in 1 us)
//   one of 64, four bf16 rows over 921600: 45.0, two CTAs for every SM 48.1, four 54.9
// behind: the kernel calls pdl_wait before it touches global memory.
template <class K, class A, class... More>
cudaError_t launch_rows_kernel(K kernel, KernelCache &cache, const A &a, bool bf16, int R, int smem, cudaStream_t st, bool behind,
                               const More &...more)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    e = ensure_dynamic_smem(cache, dev, kernel, smem);
    if (e != cudaSuccess) return e;
    constexpr int step = kRowWarps * kPiece;
    const long long rows = (long long)a.Tq * a.G;
    RowsGeom g;
    g.row_blocks = (int)((rows + R - 1) / R);
    const long long blocks = (long long)a.N * a.Hkv * g.row_blocks;
    const long long want = (device_sm_count() + blocks - 1) / blocks;
    const long long most = ((long long)a.Tk + step - 1) / step;
    const long long s = want < most ? want : most;
    if (s <= kMaxCluster || most <= kMaxCluster * 4) {
        g.cluster = 1;
        while (g.cluster < s && g.cluster < kMaxCluster) g.cluster *= 2;
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
        e = workspace_alloc(&ws, nrow * ((size_t)a.D * 4 + sizeof(float2)), st);
        if (e != cudaSuccess) return e;
        part.o = static_cast<float *>(ws);   // rows of D floats: 16-byte aligned
        part.ml = reinterpret_cast<float2 *>(part.o + nrow * a.D);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks * g.splits));
    cfg.blockDim = dim3(kRowThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    int attrs = 0;
    if (g.cluster > 1) {
        at[attrs].id = cudaLaunchAttributeClusterDimension;
        at[attrs].val.clusterDim.x = g.cluster;
        at[attrs].val.clusterDim.y = at[attrs].val.clusterDim.z = 1;
        ++attrs;
    }
    if (behind) {
        at[attrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[attrs].val.programmaticStreamSerializationAllowed = 1;
        ++attrs;
    }
    cfg.attrs = at;
    cfg.numAttrs = attrs;
    e = cudaLaunchKernelEx(&cfg, kernel, a, g, part, more...);
    if (e == cudaSuccess && part.parts > 0) e = launch_attn_join(a, bf16, part, st);
    if (ws) {
        const cudaError_t ef = workspace_free(ws, st);
        if (e == cudaSuccess) e = ef;
    }
    return e;
}

}  // namespace sc
