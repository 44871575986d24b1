// Attention of up to three fp32 query rows per key head over many keys (a
// decoder's next token, a short draft): every key and value is used by R <= 3
// rows, so the kernel is bound by reading K and V once.  The MMA kernel,
// attn_mma.cu, splits fp32 operands into bf16 planes, which costs the same for
// one row as for eight.  Calls among others on changing inputs, 1, 3 and 4 rows
// (4 in two blocks here):
//   8 x 4 key heads of 32 over 16384 states: 25.5, 27.2, 40.8 us; there 30.8
//   32 x 8 key heads of 64 over 3136:        64.9, 68.2, 110;     there 78.6 to 80.5
//   4 x 8 key heads of 128 over 5000:        30.1, 32.2, 48.8;    there 60.1 to 63.3
// (Asynchronous copies to shared memory, as there, but with FFMA, took one row of
// these a tenth to a third longer.)
//
//   s_j = scale * q . k_j,  m = max_j s_j,  l = sum_j 2^((s_j - m) log2 e),
//   o = sum_j 2^((s_j - m) log2 e) v_j,     out = o / l
//
// One pass: m, l and o are running values, o and l rescaled when m grows.  A
// key's D elements are held by LPK lanes, eight each, straight from global
// memory in registers; the dot product is summed over those lanes by
// shuffles (eight elements a lane, not four, to shuffle half as often), after
// which all of them have the key's weight for their own slice of its value.
// Nothing is shared between warps until the end (attn_rows.cuh).
#include "attn_rows.cuh"
#include "launch.h"

namespace sc {

namespace {

constexpr int E = 8;   // elements of a key per lane

// Eight elements at p.
struct Chunk {
    uint4 w[2];
    __device__ __forceinline__ void zero() { w[0] = w[1] = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void load(const float *p)
    {
        w[0] = ldg16(p);
        w[1] = ldg16(p + 4);
    }
    __device__ __forceinline__ void unpack(float (&f)[E]) const
    {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f[4 * i] = __uint_as_float(w[i].x);
            f[4 * i + 1] = __uint_as_float(w[i].y);
            f[4 * i + 2] = __uint_as_float(w[i].z);
            f[4 * i + 3] = __uint_as_float(w[i].w);
        }
    }
};

// LPK lanes per key, R rows per CTA, U keys of a lane group in flight.
template <int LPK, int R, int U>
__global__ void __launch_bounds__(kRowThreads, 2) attn_rows_kernel(const AttnArgs a, const RowsGeom g, const AttnPartials part)
{
    constexpr int KPW = 32 / LPK;   // keys per warp-wide load
    constexpr int DP = LPK * E;
    __shared__ WarpSums<R, DP> sm;
    __shared__ CtaSums<R, DP> cs;

    pdl_trigger();   // the join kernel may be set up; it waits for this grid's end
    if (g.cluster > 1) cluster_arrive();
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
            Chunk x;
            x.load(static_cast<const float *>(a.q) + n * a.qs.n + t * a.qs.t + hq * a.qs.h + dl * E);
            x.unpack(f);
        }
#pragma unroll
        for (int i = 0; i < E; ++i) q[r][i] = f[i] * (a.scale * kLog2e);
    }

    // this CTA's keys: an equal share of the sequence's own length
    int len = a.Tk;
    if (a.k_len) len = max(0, min(len, a.k_len[n]));
    const int per = (len + g.splits - 1) / g.splits;   // Tk <= 2^30: no sum here passes 2^31
    const int k0 = (int)min((long long)len, (long long)split * per), k1 = min(len, k0 + per);

    const float *kb = static_cast<const float *>(a.k) + n * a.ks.n + h * a.ks.h + dl * E;
    const float *vb = static_cast<const float *>(a.v) + n * a.vs.n + h * a.vs.h + dl * E;
    const unsigned char *mb = a.key_mask ? a.key_mask + (long long)n * a.Tk : nullptr;

    float m[R], l[R], o[R][E];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) o[r][i] = 0.f;
    }

    constexpr int STEP = kRowWarps * KPW * U;
    Chunk kr[U], vr[U];
    bool ok[U];
    // keys and values of this lane group's next U keys; invalid ones are not
    // read (whatever is stored there does not reach a sum)
    auto fetch = [&](int base) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int key = base + u * KPW + grp;
            ok[u] = key < k1 && (!mb || mb[key] != 0);
            kr[u].zero();
            vr[u].zero();
            if (ok[u] && dact) {
                kr[u].load(kb + key * a.ks.t);
                vr[u].load(vb + key * a.vs.t);
            }
        }
    };
    int base = k0 + warp * KPW * U;
    fetch(base);
    for (; base < k1; base += STEP) {
        Chunk kc[U], vc[U];
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
            kc[u].unpack(kf);
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
            vc[u].unpack(vf);
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
            for (int i = 0; i < E; ++i) sm.o[warp][r][dl * E + i] = o[r][i];
            if (dl == 0) {
                sm.m[warp][r] = m[r];
                sm.l[warp][r] = l[r];
            }
        }
    }
    finish_rows<float, R, DP>(sm, cs, a, g, part, nh, row0, split);
}

template <int LPK, int R, int U>
cudaError_t launch_rows(const AttnArgs &a, cudaStream_t st)
{
    static KernelCache cache;
    return launch_rows_kernel(attn_rows_kernel<LPK, R, U>, cache, a, false, R, 0, st);
}

template <int LPK, int U>
cudaError_t launch_rows_r(const AttnArgs &a, cudaStream_t st)
{
    const long long rows = (long long)a.Tq * a.G;
    if (rows == 1) return launch_rows<LPK, 1, U>(a, st);
    return rows == 2 ? launch_rows<LPK, 2, U>(a, st) : launch_rows<LPK, 3, U>(a, st);
}

}  // namespace

cudaError_t launch_attn_rows(const AttnArgs &a, cudaStream_t st)
{
    if (a.D <= 32) return launch_rows_r<4, 2>(a, st);
    if (a.D <= 64) return launch_rows_r<8, 2>(a, st);
    return launch_rows_r<16, 2>(a, st);
}

}  // namespace sc
