// Attention of few rows per key head over many keys: a decoder's next token
// with its group of query heads, a short draft.  Bound by reading K and V
// once; the products run on warp-wide m16n8k16 bf16 MMAs, which take the rows
// as M, so that a block of 8 or 16 rows costs what one row does (bf16: some 35
// instructions per KB of K and V; multiplied out in registers it was 210 for
// four rows, and the issue slots were the bound).
//
//   S = Q K^T,  P = 2^(c S - m),  O = P V,  out = O / sum P,   c = scale log2 e
//
// One pass over the keys, m and the sum running values of a row.  Keys and
// values come through a ring of each warp's own in shared memory (PieceRing),
// and from there to the MMA's registers 16 bytes a lane:
//   * a product's order of summation over d is free, so lane (g, t) of a quad
//     takes its key's 16-byte chunks 4 i + t as its share of k, the same for
//     Q, with no transposition;
//   * the columns of V's product are free as well: lane (g, t) reads one chunk
//     at a time of each of the four keys that its share of P stands for, and
//     pairs two keys' elements.
// Column g of the scores is
// key g / 2 + 4 (g mod 2), and chunk column g of V is chunk g / 2 + 4 (g mod 2),
// so that every quarter-warp's reads fall in eight different bank groups.  The
// scores' registers are P's operand registers as they are.
//
// bf16 tensors: P is rounded to bf16 (a relative error of 2^-8 of single
// terms).  fp32 tensors: Q, K, P and V are split into three bf16 planes in
// registers, x = x0 + x1 + x2 to 24 bits, a product the six of planes
// i + j <= 2: in four MMAs, since rows 8 to 15 of an operand Q or P take its
// second plane.  The MMAs cut sums short instead of rounding them, so the large
// product of the scores and the small ones have accumulators of their own, and
// O is moved to sums outside the MMAs every FLUSH steps.  (At 128 columns these
// accumulators, Q's planes and the sums fill 255 registers, and 48 bytes a
// thread are spilled.)
#include "attn_rows.cuh"
#include "launch.h"
#include "tc_common.cuh"

namespace sc {

namespace {

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w)); }

constexpr int FLUSH = 4;

// Index of column g of a product (see above).
__device__ __forceinline__ int spread(int g) { return (g >> 1) + 4 * (g & 1); }

// Two floats as three pairs of bf16, x = x0 + x1 + x2.  The first two planes
// stay finite: fp32 values above bf16's largest, M, leave the rest to the
// second, and an infinity is (M, M, infinity), of which the last meets the first
// plane of the other operand only, so that 0 times it or a difference of two
// does not arise (attn_split.cu's (0, 0, infinity) would take three more
// instructions an element here).  For the same reason rows 8 to 15 of its
// product are not 0: both halves of the rows take half of that first plane.
__device__ __forceinline__ void split3(float x, float y, uint32_t (&p)[3])
{
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        p[i] = i < 2 ? pack_bf16_finite(x, y) : tc::pack_bf16(x, y);
        x -= __uint_as_float(p[i] << 16);
        y -= __uint_as_float(p[i] & 0xffff0000u);
    }
}

// Half of two bf16.
__device__ __forceinline__ uint32_t half_of(uint32_t x)
{
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&x), __float2bfloat162_rn(0.5f));
    return *reinterpret_cast<const uint32_t *>(&y);
}

// DP: head width rounded up to 64 or 128 (fp32: 32, 64 or 128).  RH: 1 for up
// to 8 rows, 2 for 16 (bf16 only: fp32 has no registers for them, and 16 rows'
// cluster sums no shared memory of their own).
template <class T, int DP>
constexpr int entries() { return sizeof(T) == 4 && DP == 128 ? 3 : 6; }
template <class T, int DP>
constexpr int ctas_per_sm() { return PieceRing<T, DP, entries<T, DP>()>::CH == 8 ? 2 : 1; }
template <class T, int DP, int RH>
using MmaShared = RowsShared<T, DP, entries<T, DP>(), 8 * RH, RH == 1>;

template <class T, int DP, int RH>
__global__ void __launch_bounds__(kRowThreads, ctas_per_sm<T, DP>())
    attn_mma_kernel(const AttnArgs a, const RowsGeom g, const AttnPartials part)
{
    using Ring = PieceRing<T, DP, entries<T, DP>()>;
    constexpr bool F32 = sizeof(T) == 4;
    constexpr int R = 8 * RH;
    constexpr int EPC = Ring::EPC, CH = Ring::CH;
    constexpr int KC = CH / 4;           // chunks of a key per lane
    constexpr int VC = CH / 8;           // of a value per lane
    constexpr int NT = VC * EPC;         // products of 8 columns of O
    static_assert(!F32 || RH == 1, "fp32: 8 rows");
    extern __shared__ __align__(128) unsigned char dyn[];
    MmaShared<T, DP, RH> &sm = *reinterpret_cast<MmaShared<T, DP, RH> *>(dyn);

    pdl_trigger();   // the join kernel may be set up; it waits for this grid's end
    if (RH == 1 && g.cluster > 1) cluster_arrive();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gq = lane >> 2, t = lane & 3;
    const int split = blockIdx.x % g.splits;
    const int blk = blockIdx.x / g.splits;
    const int row0 = (blk % g.row_blocks) * R;
    const int nh = blk / g.row_blocks;
    const int n = nh / a.Hkv, h = nh - n * a.Hkv;
    const int rows = a.Tq * a.G;

    // the rows' queries (a row past the last one is 0), as stored, or in planes:
    // the scale is applied to the fp32 scores
    constexpr int PL = F32 ? 3 : 1, QW = F32 ? 2 : 4;   // planes; words of a chunk's operand
    uint32_t q[RH][PL][KC][QW];
#pragma unroll
    for (int r = 0; r < RH; ++r)
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            const int row = row0 + r * 8 + gq, d = (c * 4 + t) * EPC;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (row < rows && d < a.D) {
                const int tok = row / a.G, hq = h * a.G + row % a.G;
                v = ldg16(static_cast<const T *>(a.q) + n * a.qs.n + tok * a.qs.t + hq * a.qs.h + d);
            }
            if constexpr (F32) {
                uint32_t p0[3], p1[3];
                split3(__uint_as_float(v.x), __uint_as_float(v.y), p0);
                split3(__uint_as_float(v.z), __uint_as_float(v.w), p1);
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    q[r][i][c][0] = p0[i];
                    q[r][i][c][1] = p1[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) q[r][0][c][i] = word(v, i);
            }
        }

    Ring ring;
    ring.begin(sm.ring[warp], a, n, h, split, g.splits, warp);

    const float sc = a.scale * kLog2e;
    float m[RH], l[RH], o[NT][4], sums[F32 ? NT : 1][2];
#pragma unroll
    for (int r = 0; r < RH; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][i] = 0.f;
#pragma unroll
    for (int j = 0; j < (F32 ? NT : 1); ++j) sums[j][0] = sums[j][1] = 0.f;
    auto flush = [&](float f) {
        if constexpr (F32) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                sums[j][0] = (sums[j][0] + (o[j][0] + o[j][2])) * f;
                sums[j][1] = (sums[j][1] + (o[j][1] + o[j][3])) * f;
                o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
            }
        }
    };

    for (int step = 0; step < ring.steps; ++step) {
        const uint32_t ok = ring.valid();
        const uint4 *kt = ring.template piece<true>(step);

        float s[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float lo[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
            const int key = spread(gq);
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const uint4 k = kt[(i * 8 + key) * CH + ((c * 4 + t) ^ key)];
                if constexpr (F32) {
                    uint32_t b0[3], b1[3];
                    split3(__uint_as_float(k.x), __uint_as_float(k.y), b0);
                    split3(__uint_as_float(k.z), __uint_as_float(k.w), b1);
                    const uint32_t h0 = half_of(q[0][0][c][0]), h1 = half_of(q[0][0][c][1]);
                    mma16816(lo, h0, h0, h1, h1, b0[2], b1[2]);
                    mma16816(lo, q[0][2][c][0], 0u, q[0][2][c][1], 0u, b0[0], b1[0]);
                    mma16816(lo, q[0][0][c][0], q[0][1][c][0], q[0][0][c][1], q[0][1][c][1], b0[1], b1[1]);
                    mma16816(s[i], q[0][0][c][0], q[0][1][c][0], q[0][0][c][1], q[0][1][c][1], b0[0], b1[0]);
                } else {
                    mma16816(s[i], q[0][0][c][0], RH == 2 ? q[RH - 1][0][c][0] : 0u, q[0][0][c][1],
                             RH == 2 ? q[RH - 1][0][c][1] : 0u, k.x, k.y);
                    mma16816(s[i], q[0][0][c][2], RH == 2 ? q[RH - 1][0][c][2] : 0u, q[0][0][c][3],
                             RH == 2 ? q[RH - 1][0][c][3] : 0u, k.z, k.w);
                }
            }
            if constexpr (F32) {
                s[i][0] += (lo[0] + lo[2]) + s[i][2];
                s[i][1] += (lo[1] + lo[3]) + s[i][3];
            }
        }
        // scores of row g (and g + 8) for the keys 8 i + t and 8 i + t + 4
        float top[RH];
        bool grow = false;
#pragma unroll
        for (int r = 0; r < RH; ++r) {
            top[r] = m[r];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float &x = s[i][2 * r + e];
                    x = (ok >> (8 * i + t + 4 * e) & 1u) ? x * sc : -INFINITY;
                    top[r] = fmaxf(top[r], x);
                }
            top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
            top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
            grow |= top[r] > m[r];
        }
        const bool any_grow = __any_sync(0xffffffffu, grow);
        if (any_grow) {
#pragma unroll
            for (int r = 0; r < RH; ++r) {
                const float f = top[r] == -INFINITY ? 1.f : ex2(m[r] - top[r]);
                m[r] = top[r];
                l[r] *= f;
                if constexpr (F32) {
                    flush(f);
                } else {
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        o[j][2 * r] *= f;
                        o[j][2 * r + 1] *= f;
                    }
                }
            }
        } else if (F32 && step % FLUSH == FLUSH - 1) {
            flush(1.f);
        }
        uint32_t p[2][RH][PL];
#pragma unroll
        for (int r = 0; r < RH; ++r) {
            const float ms = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float x = ex2(s[i][2 * r] - ms), y = ex2(s[i][2 * r + 1] - ms);
                l[r] += x + y;
                if constexpr (F32)
                    split3(x, y, p[i][r]);
                else
                    p[i][r][0] = tc::pack_bf16(x, y);
            }
        }
        const uint32_t ph[2] = {half_of(p[0][0][0]), half_of(p[1][0][0])};   // fp32
        const uint4 *vt = ring.template piece<false>(step);
#pragma unroll
        for (int c = 0; c < VC; ++c) {
            // keys t, t + 4, t + 8, t + 12
            const int x = c * 8 + spread(gq);
            uint4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = vt[(t + 4 * i) * CH + (x ^ ((t + 4 * i) & 7))];
#pragma unroll
            for (int j = 0; j < EPC; ++j) {
                float(&acc)[4] = o[c * EPC + j];
                if constexpr (F32) {
                    uint32_t b0[3], b1[3];
                    split3(__uint_as_float(word(v[0], j)), __uint_as_float(word(v[1], j)), b0);
                    split3(__uint_as_float(word(v[2], j)), __uint_as_float(word(v[3], j)), b1);
                    mma16816(acc, ph[0], ph[0], ph[1], ph[1], b0[2], b1[2]);
                    mma16816(acc, p[0][0][2], 0u, p[1][0][2], 0u, b0[0], b1[0]);
                    mma16816(acc, p[0][0][0], p[0][0][1], p[1][0][0], p[1][0][1], b0[1], b1[1]);
                    mma16816(acc, p[0][0][0], p[0][0][1], p[1][0][0], p[1][0][1], b0[0], b1[0]);
                } else {
                    const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
                    const uint32_t b0 = __byte_perm(word(v[0], j / 2), word(v[1], j / 2), sel);
                    const uint32_t b1 = __byte_perm(word(v[2], j / 2), word(v[3], j / 2), sel);
                    mma16816(acc, p[0][0][0], RH == 2 ? p[0][RH - 1][0] : 0u, p[1][0][0], RH == 2 ? p[1][RH - 1][0] : 0u, b0, b1);
                }
            }
        }
        ring.next_step();
    }
    flush(1.f);
    cp_async_wait<0>();
    __syncthreads();   // the rings' memory becomes the sums'
    if (RH == 2 && g.cluster > 1) cluster_arrive();

    // the warp's sums: row g (and g + 8); l over the quad
#pragma unroll
    for (int r = 0; r < RH; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        if (t == 0) {
            sm.sums.warps.m[warp][r * 8 + gq] = m[r];
            sm.sums.warps.l[warp][r * 8 + gq] = l[r];
        }
#pragma unroll
        for (int c = 0; c < VC; ++c)
#pragma unroll
            for (int j = 0; j < EPC; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    sm.sums.warps.o[warp][r * 8 + gq][(c * 8 + spread(2 * t + e)) * EPC + j] =
                        F32 ? sums[F32 ? c * EPC + j : 0][e] : o[c * EPC + j][2 * r + e];
    }
    finish_rows<T, R, DP>(sm.sums.warps, sm.ctas(), a, g, part, nh, row0, split);
}

template <class T, int DP, int RH>
cudaError_t launch_mma(const AttnArgs &a, cudaStream_t st)
{
    static KernelCache cache;
    return launch_rows_kernel(attn_mma_kernel<T, DP, RH>, cache, a, sizeof(T) == 2, 8 * RH,
                              (int)sizeof(MmaShared<T, DP, RH>), st, false);
}

}  // namespace

cudaError_t launch_attn_mma(const AttnArgs &a, bool bf16, cudaStream_t st)
{
    if (!bf16) {
        if (a.D <= 32) return launch_mma<float, 32, 1>(a, st);
        return a.D <= 64 ? launch_mma<float, 64, 1>(a, st) : launch_mma<float, 128, 1>(a, st);
    }
    const bool few = (long long)a.Tq * a.G <= 8;
    if (a.D <= 64) return few ? launch_mma<__nv_bfloat16, 64, 1>(a, st) : launch_mma<__nv_bfloat16, 64, 2>(a, st);
    return few ? launch_mma<__nv_bfloat16, 128, 1>(a, st) : launch_mma<__nv_bfloat16, 128, 2>(a, st);
}

}  // namespace sc
