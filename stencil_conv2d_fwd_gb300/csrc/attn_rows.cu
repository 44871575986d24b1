// Attention of a few query rows over many keys (a decoder's next token, a
// short draft): every key and value is used by R <= 8 rows, so the kernel is
// bound by reading K and V once.
//
//   s_j = scale * q . k_j,  m = max_j s_j,  l = sum_j 2^((s_j - m) log2 e),
//   o = sum_j 2^((s_j - m) log2 e) v_j,     out = o / l
//
// One pass: m, l and o are running values, o and l rescaled when m grows.  A
// key's D elements are held by LPK lanes, 16 bytes each, straight from global
// memory in registers; the dot product is summed over those lanes by
// shuffles, after which all of them have the key's weight for their own slice
// of its value.  Nothing is shared between warps until the end, when (m, l,
// o) of the lane groups, the warps and the CTAs of a cluster (distributed
// shared memory) are joined, in that fixed order.  With more CTAs per row
// than a cluster holds, each cluster writes one partial result and
// attn_join.cu joins them.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "attn.h"
#include "launch.h"

namespace cg = cooperative_groups;

namespace sc {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCluster = 8;

template <class T>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int E = 4;   // elements of 16 bytes
    static __device__ __forceinline__ void unpack(const uint4 &u, float (&f)[4])
    {
        f[0] = __uint_as_float(u.x);
        f[1] = __uint_as_float(u.y);
        f[2] = __uint_as_float(u.z);
        f[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ float from(float v) { return v; }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int E = 8;
    static __device__ __forceinline__ void unpack(const uint4 &u, float (&f)[8])
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ __nv_bfloat16 from(float v) { return __float2bfloat16_rn(v); }
};

struct RowsGeom {
    int splits;      // CTAs per row block (a multiple of the cluster size)
    int cluster;
    int row_blocks;
};

__device__ __forceinline__ uint4 ldg16(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// LPK lanes per key, R rows per CTA, U keys of a lane group in flight.
template <class T, int LPK, int R, int U>
__global__ void __launch_bounds__(kThreads, 2) attn_rows_kernel(const AttnArgs a, const RowsGeom g, const AttnPartials part)
{
    constexpr int E = Elem<T>::E;
    constexpr int KPW = 32 / LPK;   // keys per warp-wide load
    constexpr int DP = LPK * E;
    __shared__ float sm_o[kWarps][R][DP];
    __shared__ float sm_m[kWarps][R], sm_l[kWarps][R];
    __shared__ float cta_o[R][DP], cta_m[R], cta_l[R];

    pdl_trigger();   // the join kernel may be set up; it waits for this grid's end
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int split = blockIdx.x % g.splits;
    const int blk = blockIdx.x / g.splits;
    const int row0 = (blk % g.row_blocks) * R;
    const int nh = blk / g.row_blocks;
    const int n = nh / a.Hkv, h = nh % a.Hkv;
    const int rows = a.Tq * a.G;

    const int dl = lane % LPK, grp = lane / LPK;
    const bool dact = dl * E < a.D;

    // the rows' queries, in units of log2 (a row past the last one stays 0)
    float q[R][E];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = row0 + r;
        float f[E];
#pragma unroll
        for (int i = 0; i < E; ++i) f[i] = 0.f;
        if (row < rows && dact) {
            const int t = row / a.G, hq = h * a.G + row % a.G;
            Elem<T>::unpack(ldg16(static_cast<const T *>(a.q) + n * a.qs.n + t * a.qs.t + hq * a.qs.h + dl * E), f);
        }
#pragma unroll
        for (int i = 0; i < E; ++i) q[r][i] = f[i] * (a.scale * kLog2e);
    }

    // this CTA's keys: an equal share of the sequence's own length
    int len = a.Tk;
    if (a.k_len) len = max(0, min(len, a.k_len[n]));
    const int per = (len + g.splits - 1) / g.splits;   // Tk <= 2^30: no sum here passes 2^31
    const int k0 = (int)min((long long)len, (long long)split * per), k1 = min(len, k0 + per);

    const T *kb = static_cast<const T *>(a.k) + n * a.ks.n + h * a.ks.h + dl * E;
    const T *vb = static_cast<const T *>(a.v) + n * a.vs.n + h * a.vs.h + dl * E;
    const unsigned char *mb = a.key_mask ? a.key_mask + (long long)n * a.Tk : nullptr;

    float m[R], l[R], o[R][E];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) o[r][i] = 0.f;
    }

    constexpr int STEP = kWarps * KPW * U;
    uint4 kr[U], vr[U];
    bool ok[U];
    // keys and values of this lane group's next U keys; invalid ones are not
    // read (whatever is stored there does not reach a sum)
    auto fetch = [&](int base) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int key = base + u * KPW + grp;
            ok[u] = key < k1 && (!mb || mb[key] != 0);
            kr[u] = make_uint4(0u, 0u, 0u, 0u);
            vr[u] = make_uint4(0u, 0u, 0u, 0u);
            if (ok[u] && dact) {
                kr[u] = ldg16(kb + key * a.ks.t);
                vr[u] = ldg16(vb + key * a.vs.t);
            }
        }
    };
    int base = k0 + warp * KPW * U;
    fetch(base);
    for (; base < k1; base += STEP) {
        uint4 kc[U], vc[U];
        bool okc[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            kc[u] = kr[u];
            vc[u] = vr[u];
            okc[u] = ok[u];
        }
        fetch(base + STEP);   // past k1: nothing is read
        float s[U][R];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float kf[E];
            Elem<T>::unpack(kc[u], kf);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float acc = q[r][0] * kf[0];
#pragma unroll
                for (int i = 1; i < E; ++i) acc = fmaf(q[r][i], kf[i], acc);
                s[u][r] = acc;
            }
        }
#pragma unroll
        for (int off = LPK / 2; off > 0; off >>= 1)
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int r = 0; r < R; ++r) s[u][r] += __shfl_xor_sync(0xffffffffu, s[u][r], off);
        float mn[R];
        bool grow = false;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mn[r] = m[r];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                s[u][r] = okc[u] ? s[u][r] : -INFINITY;
                mn[r] = fmaxf(mn[r], s[u][r]);
            }
            grow |= mn[r] > m[r];
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float f = mn[r] == -INFINITY ? 1.f : ex2(m[r] - mn[r]);
                l[r] *= f;
#pragma unroll
                for (int i = 0; i < E; ++i) o[r][i] *= f;
                m[r] = mn[r];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float vf[E];
            Elem<T>::unpack(vc[u], vf);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float p = ex2(s[u][r] - (m[r] == -INFINITY ? 0.f : m[r]));
                l[r] += p;
#pragma unroll
                for (int i = 0; i < E; ++i) o[r][i] = fmaf(p, vf[i], o[r][i]);
            }
        }
    }

    // join the lane groups of the warp ...
#pragma unroll
    for (int off = LPK; off < 32; off <<= 1) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m[r], off), l2 = __shfl_xor_sync(0xffffffffu, l[r], off);
            const float mm = fmaxf(m[r], m2), ms = mm == -INFINITY ? 0.f : mm;
            const float f1 = ex2(m[r] - ms), f2 = ex2(m2 - ms);
            l[r] = l[r] * f1 + l2 * f2;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float o2 = __shfl_xor_sync(0xffffffffu, o[r][i], off);
                o[r][i] = o[r][i] * f1 + o2 * f2;
            }
            m[r] = mm;
        }
    }
    if (grp == 0) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int i = 0; i < E; ++i) sm_o[warp][r][dl * E + i] = o[r][i];
            if (dl == 0) {
                sm_m[warp][r] = m[r];
                sm_l[warp][r] = l[r];
            }
        }
    }
    __syncthreads();
    // ... the warps of the CTA ...
    for (int e = tid; e < R * DP; e += kThreads) {
        const int r = e / DP, d = e % DP;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w][r]);
        const float ms = mm == -INFINITY ? 0.f : mm;
        float ls = 0.f, os = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = ex2(sm_m[w][r] - ms);
            ls = fmaf(sm_l[w][r], f, ls);
            os = fmaf(sm_o[w][r][d], f, os);
        }
        cta_o[r][d] = os;
        if (d == 0) {
            cta_m[r] = mm;
            cta_l[r] = ls;
        }
    }
    // ... and the CTAs of the cluster, each finishing a share of the elements
    cg::cluster_group cl = cg::this_cluster();
    const int C = g.cluster, rank = split % C;
    if (C > 1)
        cl.sync();
    else
        __syncthreads();
    for (int e = rank * kThreads + tid; e < R * DP; e += C * kThreads) {
        const int r = e / DP, d = e % DP, row = row0 + r;
        float mm = -INFINITY;
        float mc[kMaxCluster], lc[kMaxCluster], oc[kMaxCluster];
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
            if (c < C) {
                mc[c] = C > 1 ? *cl.map_shared_rank(&cta_m[r], c) : cta_m[r];
                lc[c] = C > 1 ? *cl.map_shared_rank(&cta_l[r], c) : cta_l[r];
                oc[c] = C > 1 ? *cl.map_shared_rank(&cta_o[r][d], c) : cta_o[r][d];
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
        if (row < rows && d < a.D) {
            const int t = row / a.G, hq = h * a.G + row % a.G;
            if (part.parts > 0) {
                const long long at = ((long long)(split / C) * a.N * a.Hkv + nh) * rows + row;
                part.o[at * a.D + d] = os;
                if (d == 0) part.ml[at] = make_float2(mm, ls);
            } else {
                static_cast<T *>(a.out)[n * a.os.n + t * a.os.t + hq * a.os.h + d] =
                    Elem<T>::from(ls == 0.f ? 0.f : os / ls);
                if (d == 0 && a.lse)
                    a.lse[((long long)n * a.Hq + hq) * a.Tq + t] = ls == 0.f ? -INFINITY : mm * kLn2 + logf(ls);
            }
        }
    }
    if (C > 1) cl.sync();   // no CTA leaves while another reads its shared memory
}

template <class T, int LPK, int R, int U>
cudaError_t launch_rows(const AttnArgs &a, cudaStream_t st)
{
    const long long rows = (long long)a.Tq * a.G;
    RowsGeom g;
    g.row_blocks = (int)((rows + R - 1) / R);
    const long long blocks = (long long)a.N * a.Hkv * g.row_blocks;
    // CTAs per row block: enough to fill the GPU twice over, none with less
    // than one step of keys
    constexpr int STEP = kWarps * (32 / LPK) * U;
    const long long want = (4LL * device_sm_count() + blocks - 1) / blocks;
    const long long most = ((long long)a.Tk + STEP - 1) / STEP;
    long long s = want < most ? want : most;
    if (s <= kMaxCluster) {
        int c = 1;
        while (c < s) c *= 2;
        g.splits = g.cluster = c;
    } else {
        g.cluster = kMaxCluster;
        g.splits = (int)((s + kMaxCluster - 1) / kMaxCluster * kMaxCluster);
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
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = g.cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, attn_rows_kernel<T, LPK, R, U>, a, g, part);
    if (e == cudaSuccess && part.parts > 0) e = launch_attn_join(a, sizeof(T) == 2, part, st);
    if (ws) {
        const cudaError_t ef = workspace_free(ws, st);
        if (e == cudaSuccess) e = ef;
    }
    return e;
}

template <class T, int LPK>
cudaError_t launch_rows_r(const AttnArgs &a, cudaStream_t st)
{
    const long long rows = (long long)a.Tq * a.G;
    if (rows == 1) return launch_rows<T, LPK, 1, 4>(a, st);
    if (rows == 2) return launch_rows<T, LPK, 2, 4>(a, st);
    return launch_rows<T, LPK, 4, 2>(a, st);
}

template <class T>
cudaError_t launch_rows_t(const AttnArgs &a, cudaStream_t st)
{
    const int lanes = a.D / Elem<T>::E;
    if (lanes <= 4) return launch_rows_r<T, 4>(a, st);
    if (lanes <= 8) return launch_rows_r<T, 8>(a, st);
    if (lanes <= 16) return launch_rows_r<T, 16>(a, st);
    return launch_rows_r<T, 32>(a, st);
}

}  // namespace

cudaError_t launch_attn_rows(const AttnArgs &a, bool bf16, cudaStream_t st)
{
    return bf16 ? launch_rows_t<__nv_bfloat16>(a, st) : launch_rows_t<float>(a, st);
}

}  // namespace sc
