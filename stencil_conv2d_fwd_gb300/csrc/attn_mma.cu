// Attention of up to 16 bf16 rows per key head over many keys: a decoder's
// next token with its group of query heads, a short draft.  Bound by reading
// K and V once; the products run on warp-wide m16n8k16 MMAs, which take the
// rows as M, so that a 16-row block costs what one row does (some 35
// instructions per KB of K and V; multiplied out in registers it was 210 for
// four rows, and the issue slots were the bound).
//
//   S = Q K^T,  P = 2^(c S - m),  O = P V,  out = O / sum P,   c = scale log2 e
//
// One pass, running m and sum of a row, as in attn_rows.cu.  Each warp has a
// ring of its own in shared memory, STAGES pieces of 16 keys and values that
// its lanes copy there asynchronously, 16 bytes each, so that some 100 KB are
// under way on an SM at any time without a register held for them and without
// a barrier between warps.  States that are not valid are not read (their
// bytes are zero-filled): whatever is stored there does not reach a sum.
// Operands go from there to the MMA's registers 16 bytes a lane:
//   * a product's order of summation over d is free, so lane (g, t) of a quad
//     takes its key's elements 8 (4 c + t) .. + 8 as its share of k, the same
//     for Q, with no transposition;
//   * the columns of V's product are free as well: lane (g, t) reads one chunk
//     of 8 elements of each of the four keys that its share of P stands for,
//     and pairs two keys' elements with one byte permutation each.
// 16-byte chunk x of a row y lies at chunk x XOR (y mod 8).  Column g of the
// scores is key g / 2 + 4 (g mod 2), and chunk column g of V is chunk
// g / 2 + 4 (g mod 2), so that every quarter-warp's reads fall in eight
// different bank groups.  The scores' registers are P's operand registers as
// they are; P is rounded to bf16 (a relative error of 2^-8 of single terms).
// A warp's pieces are every 8th of the CTA's share.
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

constexpr int KEYS = 16;   // keys of a step

// Index of column g of a product (see above).
__device__ __forceinline__ int spread(int g) { return (g >> 1) + 4 * (g & 1); }

// DP: head width rounded up to 64 or 128.  RH: 1 for up to 8 rows, 2 for 16.
constexpr int STAGES = 3;   // of 16 + 16 rows; a step's valid bits are 16 of a 64-bit word: at most 4

// The rings' memory becomes the sums' at the end.  With 8 rows the cluster's
// sums have their own: the first CTA's place is then free from the start, and
// no CTA waits for another's loop.  With 16 there is no room.
template <int DP, int RH>
struct MmaShared {
    union {
        uint4 ring[kRowWarps][STAGES][2][KEYS][DP / 8];   // K, V
        struct {
            WarpSums<8 * RH, DP> warps;
            CtaSums<RH == 1 ? 1 : 8 * RH, RH == 1 ? 1 : DP> shared_ctas;
        } sums;
    };
    CtaSums<RH == 1 ? 8 : 1, RH == 1 ? DP : 1> own_ctas;
    __device__ __forceinline__ CtaSums<8 * RH, DP> &ctas()
    {
        if constexpr (RH == 1)
            return own_ctas;
        else
            return sums.shared_ctas;
    }
};

template <int DP, int RH>
__global__ void __launch_bounds__(kRowThreads, DP == 64 ? 2 : 1)
    attn_mma_kernel(const AttnArgs a, const RowsGeom g, const AttnPartials part)
{
    constexpr int R = 8 * RH;
    constexpr int ST = STAGES;
    constexpr int KC = DP / 32;          // 16-byte chunks of a key per lane
    constexpr int VC = DP / 64;          // of a value per lane
    constexpr int CH = DP / 8;           // chunks of a row
    constexpr int RPL = 32 / CH;         // rows of a warp-wide copy
    constexpr int COPIES = KEYS / RPL;
    extern __shared__ __align__(128) unsigned char dyn[];
    MmaShared<DP, RH> &sm = *reinterpret_cast<MmaShared<DP, RH> *>(dyn);

    pdl_trigger();   // the join kernel may be set up; it waits for this grid's end
    if (RH == 1 && g.cluster > 1) cluster_arrive();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gq = lane >> 2, t = lane & 3;
    const int split = blockIdx.x % g.splits;
    const int blk = blockIdx.x / g.splits;
    const int row0 = (blk % g.row_blocks) * R;
    const int nh = blk / g.row_blocks;
    const int n = nh / a.Hkv, h = nh - n * a.Hkv;
    const int rows = a.Tq * a.G;

    // the rows' queries (a row past the last one is 0), as stored: the scale
    // is applied to the fp32 scores
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    uint4 q[RH][KC];
#pragma unroll
    for (int r = 0; r < RH; ++r)
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            const int row = row0 + r * 8 + gq, d = (c * 4 + t) * 8;
            q[r][c] = zero;
            if (row < rows && d < a.D) {
                const int tok = row / a.G, hq = h * a.G + row % a.G;
                q[r][c] = ldg16(static_cast<const __nv_bfloat16 *>(a.q) + n * a.qs.n + tok * a.qs.t + hq * a.qs.h + d);
            }
        }

    int len = a.Tk;
    if (a.k_len) len = max(0, min(len, a.k_len[n]));
    // this CTA's keys: an equal share of the sequence's own length, in pieces
    const int pieces = (len + KEYS - 1) / KEYS;
    const int p0 = (int)((long long)pieces * split / g.splits), p1 = (int)((long long)pieces * (split + 1) / g.splits);
    const int steps = p1 - p0 > warp ? (p1 - p0 - warp + kRowWarps - 1) / kRowWarps : 0;   // of this warp
    const int key0 = (p0 + warp) * KEYS;
    constexpr int STEP = kRowWarps * KEYS;
    const unsigned char *mb = a.key_mask ? a.key_mask + (long long)n * a.Tk : nullptr;

    // the lane's part of a step's copies: row crow + RPL i, chunk cch
    const int crow = lane / CH, cch = lane % CH;
    const bool cact = cch * 8 < a.D;   // chunks past D are zero-filled
    const __nv_bfloat16 *kp = static_cast<const __nv_bfloat16 *>(a.k) + n * a.ks.n + h * a.ks.h +
                              (long long)(key0 + crow) * a.ks.t + (cact ? cch * 8 : 0);
    const __nv_bfloat16 *vp = static_cast<const __nv_bfloat16 *>(a.v) + n * a.vs.n + h * a.vs.h +
                              (long long)(key0 + crow) * a.vs.t + (cact ? cch * 8 : 0);
    const __nv_bfloat16 *kbase = static_cast<const __nv_bfloat16 *>(a.k), *vbase = static_cast<const __nv_bfloat16 *>(a.v);
    uint4 *ring = &sm.ring[warp][0][0][0][0];
    constexpr int STAGE = 2 * KEYS * CH;   // in 16-byte units
    uint32_t dst[COPIES];
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
        const int row = crow + i * RPL;
        dst[i] = smem_u32(ring + row * CH + (cch ^ (row & 7)));
    }

    // Valid bits of a step's keys.  The mask's byte is read two steps ahead of
    // its copies.
    auto mask_byte = [&](int step) -> int {
        const int key = key0 + step * STEP + lane;
        return step < steps && lane < KEYS && key < len ? (mb ? (int)mb[key] : 1) : 0;
    };
    auto copy = [&](int stage, uint32_t ok) {
        const uint32_t at = stage * STAGE * 16;
        const __nv_bfloat16 *k = kp, *v = vp;
#pragma unroll
        for (int i = 0; i < COPIES; ++i, k += RPL * a.ks.t, v += RPL * a.vs.t) {
            const bool on = cact && (ok >> (crow + i * RPL) & 1u);
            cp_async16(dst[i] + at, on ? k : kbase, on ? 16 : 0);
            cp_async16(dst[i] + at + KEYS * CH * 16, on ? v : vbase, on ? 16 : 0);
        }
        cp_async_commit();
        kp += STEP * a.ks.t;
        vp += STEP * a.vs.t;
    };
    // steps 0 .. ST - 2 under way; their valid bits, 16 each, the oldest lowest
    unsigned long long okq = 0;
    {
        int byte[ST - 1];
#pragma unroll
        for (int i = 0; i < ST - 1; ++i) byte[i] = mask_byte(i);
#pragma unroll
        for (int i = 0; i < ST - 1; ++i) {
            const uint32_t ok = __ballot_sync(0xffffffffu, byte[i] != 0);
            okq |= (unsigned long long)ok << (16 * i);
            copy(i, ok);
        }
    }
    int byte = mask_byte(ST - 1);

    const float sc = a.scale * kLog2e;
    float m[RH], l[RH], o[VC * 8][4];
#pragma unroll
    for (int r = 0; r < RH; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < VC * 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][i] = 0.f;

    int stage = 0, fill = ST - 1;
    for (int step = 0; step < steps; ++step) {
        cp_async_wait<ST - 2>();
        __syncwarp();
        // the step ST - 1 ahead goes where the last step was read (the barrier
        // above is behind those reads)
        {
            const uint32_t ok = __ballot_sync(0xffffffffu, byte != 0);
            byte = mask_byte(step + ST);
            okq |= (unsigned long long)ok << (16 * (ST - 1));
            copy(fill, ok);
            fill = fill + 1 == ST ? 0 : fill + 1;
        }
        const uint32_t ok = (uint32_t)okq & 0xffffu;
        okq >>= 16;
        const uint4 *kt = ring + stage * STAGE, *vt = kt + KEYS * CH;
        stage = stage + 1 == ST ? 0 : stage + 1;

        float s[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const int key = spread(gq);
                const uint4 k = kt[(i * 8 + key) * CH + ((c * 4 + t) ^ key)];
                mma16816(s[i], q[0][c].x, RH == 2 ? q[RH - 1][c].x : 0u, q[0][c].y, RH == 2 ? q[RH - 1][c].y : 0u, k.x, k.y);
                mma16816(s[i], q[0][c].z, RH == 2 ? q[RH - 1][c].z : 0u, q[0][c].w, RH == 2 ? q[RH - 1][c].w : 0u, k.z, k.w);
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
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int r = 0; r < RH; ++r) {
                const float f = top[r] == -INFINITY ? 1.f : ex2(m[r] - top[r]);
                m[r] = top[r];
                l[r] *= f;
#pragma unroll
                for (int j = 0; j < VC * 8; ++j) {
                    o[j][2 * r] *= f;
                    o[j][2 * r + 1] *= f;
                }
            }
        }
        uint32_t p[2][RH];
#pragma unroll
        for (int r = 0; r < RH; ++r) {
            const float ms = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float x = ex2(s[i][2 * r] - ms), y = ex2(s[i][2 * r + 1] - ms);
                l[r] += x + y;
                p[i][r] = tc::pack_bf16(x, y);
            }
        }
#pragma unroll
        for (int c = 0; c < VC; ++c) {
            // keys t, t + 4, t + 8, t + 12
            const int x = c * 8 + spread(gq);
            uint4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = vt[(t + 4 * i) * CH + (x ^ ((t + 4 * i) & 7))];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
                const uint32_t b0 = __byte_perm(word(v[0], j / 2), word(v[1], j / 2), sel);
                const uint32_t b1 = __byte_perm(word(v[2], j / 2), word(v[3], j / 2), sel);
                mma16816(o[c * 8 + j], p[0][0], RH == 2 ? p[0][RH - 1] : 0u, p[1][0], RH == 2 ? p[1][RH - 1] : 0u, b0, b1);
            }
        }
    }
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
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    sm.sums.warps.o[warp][r * 8 + gq][(c * 8 + spread(2 * t + e)) * 8 + j] = o[c * 8 + j][2 * r + e];
    }
    finish_rows<__nv_bfloat16, R, DP>(sm.sums.warps, sm.ctas(), a, g, part, nh, row0, split);
}

template <int DP, int RH>
cudaError_t launch_mma(const AttnArgs &a, cudaStream_t st)
{
    const int smem = (int)sizeof(MmaShared<DP, RH>);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    static KernelCache cache;
    e = ensure_dynamic_smem(cache, dev, attn_mma_kernel<DP, RH>, smem);
    if (e != cudaSuccess) return e;
    return launch_rows_kernel(attn_mma_kernel<DP, RH>, a, true, 8 * RH, kRowWarps * KEYS, smem, st);
}

}  // namespace

cudaError_t launch_attn_mma(const AttnArgs &a, cudaStream_t st)
{
    const bool few = (long long)a.Tq * a.G <= 8;
    if (a.D <= 64) return few ? launch_mma<64, 1>(a, st) : launch_mma<64, 2>(a, st);
    return few ? launch_mma<128, 1>(a, st) : launch_mma<128, 2>(a, st);
}

}  // namespace sc
