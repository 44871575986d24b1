// Attention of few rows per key head over states held as 8-bit codes with a
// scale for each block of states and head: a decoder's next token with its group
// of query heads, a short draft; more rows come in blocks of 8 or 16.
//
//   S = scale ks (Q Kc^T),  P = 2^(log2e S - top),  O = sum_groups vs 2^(top - m) (P Vc),
//   l = sum_groups 2^(top - m) sum P,  out = O / l
//
// over groups of 16 keys (32 where they share a scale), top the group's largest
// score and m the largest so far.
//
// Bound by reading the codes once.  The products run on warp-wide m16n8k16 fp16
// MMAs: a code, integer or e4m3, is exact in fp16, so neither the codes nor their
// scales are rounded.  Queries are fp16 times a power of two for each row (a bf16
// query is exact; an fp32 one has two planes of 11 bits, the second as rows 8 to
// 15 of the operand).  Weights are 2^14 P, so that fp16 holds them to 2^-11 of
// themselves down to 2^-28 of the group's largest (fp32 tensors: two planes, 22 bits
// of that largest); a group has one scale, so a small weight cannot meet a larger
// one's scale.  A group's products start from zero and enter the sums in fp32 with
// its scale, so that the MMAs' cut-off sums stay short.
//
// Keys and values come through a ring of each warp's own in shared memory, copied
// there by TMA, one instruction for 16 or 32 rows (by 16-byte copies of the lanes
// their addresses took a fifth of all instructions), and go to the operands in
// registers 8 or 16 bytes at a time:
//   * the order of summation over d is free, so lane (g, t) takes whole 16-byte
//     chunks of its key as its share of k, and Q is laid out to match;
//   * the columns of V's product are free too: lane (g, t) takes the g-th eighth
//     of the head of each of the four keys that its share of P stands for.
// Integer codes become fp16 in 2.5 (K) or 3 (V) instructions for two: a byte
// with its sign bit turned is the low byte of 1024 + 128 + x in fp16, from which
// 1152 is taken.
//
// Measured (in a graph): one bf16 token, 4 heads on one key head of 64, over 921600
// e4m3 states 30.6 us (118 MB; 9 us of launch, ring start and join, the rest at 5.6
// TB/s); 32 tokens, 16 heads on 4, over up to 3136 int8 states 17.1.  A warp's chain of
// products, maximum and weights is what a step waits for (issue slots 49% busy); two
// CTAs an SM took as long on one sequence and a third longer on a batch.  Heads of 128,
// whose registers spill (8 rows): 32 tokens, 16 heads on 4, over 3136 int8 states 46 us in
// bf16 (heads of 64 20), 40 in fp32 (20); 4 heads on one over 921600 states 74 and 65.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstring>
#include <mutex>

#include "attn_rows.cuh"
#include "launch.h"
#include "layer.h"
#include "tc_common.cuh"

namespace sc {

namespace {

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t y;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t x)
{
    float2 y;
    asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\ncvt.f32.f16 %0, l;\ncvt.f32.f16 %1, h;\n}\n" : "=f"(y.x), "=f"(y.y) : "r"(x));
    return y;
}

// Four codes -> two pairs of fp16.  Integers: (bytes 0, 2) and (1, 3); e4m3:
// (0, 1) and (2, 3).
template <bool E4M3>
__device__ __forceinline__ void to_f16(uint32_t w, uint32_t &p0, uint32_t &p1)
{
    if constexpr (E4M3) {
        asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\ncvt.rn.f16x2.e4m3x2 %0, l;\ncvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
            : "=r"(p0), "=r"(p1)
            : "r"(w));
    } else {
        // (w & 0x00ff00ff) ^ 0x64806480 is 1024 + (x + 128) in each half
        uint32_t e, o;
        asm("lop3.b32 %0, %1, 0x00ff00ff, %2, 0x6a;" : "=r"(e) : "r"(w), "r"(0x64806480u));
        asm("lop3.b32 %0, %1, 0x00ff00ff, %2, 0x6a;" : "=r"(o) : "r"(w >> 8), "r"(0x64806480u));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p0) : "r"(e), "r"(0x64806480u));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p1) : "r"(o), "r"(0x64806480u));
    }
}
// Which byte of four is element i of the pairs (p0.lo, p0.hi, p1.lo, p1.hi).
template <bool E4M3>
__host__ __device__ constexpr int byte_of(int i) { return E4M3 ? i : (i == 1 ? 2 : (i == 2 ? 1 : i)); }
// The selector that gathers bytes 2 i and 2 i + 1 of two words so that the pairs
// of to_f16 are (word 0, word 1) of byte 2 i, and of byte 2 i + 1.
template <bool E4M3>
__host__ __device__ constexpr uint32_t gather(int i) { return E4M3 ? (i ? 0x7362u : 0x5140u) : (i ? 0x7632u : 0x5410u); }

// Tensor maps of the codes, [n][h][t][D], boxes of DP bytes of a step's rows,
// swizzled; n_axis and h_axis are 0 where all share one (stride 0).
struct Q8Maps {
    CUtensorMap k, v;
};
struct Q8Axes {
    int k_n, k_h, v_n, v_h;
    int *status;
};

__device__ __forceinline__ void load_states(uint32_t dst, const CUtensorMap *m, int t, int h, int n, uint32_t bar)
{
    tma_load_4d(dst, m, 0, t, h, n, bar);
}

// A warp's ring: STAGES steps of KP keys and as many values, rows of DP bytes
// swizzled by the copy: 16-byte chunk c of row r lies at c XOR (r / 2 mod 4) of a
// 64-byte row, at c XOR (r mod 8) of a 128-byte one.
template <int DP>
struct Q8Ring {
    static constexpr int KP = DP == 64 ? 32 : 16;
    static constexpr int GROUPS = KP / 16;              // of 16 keys, each with one scale
    static constexpr int CH = DP / 16;                  // chunks of a row
    static constexpr int STAGES = 3;
    static constexpr int TILE = KP * DP;                // bytes
    static constexpr int STEP = kRowWarps * KP;         // keys from a step to the next
    static constexpr uint32_t FULL = KP == 32 ? 0xffffffffu : 0xffffu;

    const float *ks, *vs;
    const unsigned char *mb;
    uint64_t *bars;
    unsigned char *ring;
    int len, key0, steps, lane, log2_block, byte, kn, kh, vn, vh, drop_copy;
    unsigned long long timeout_ns;
    float scales[2 * GROUPS];   // of the step after the current one

    __device__ __forceinline__ int mask_byte(int step) const
    {
        const int key = key0 + step * STEP + lane;
        return step < steps && lane < KP && key < len ? (int)mb[key] : 0;
    }
    static __device__ __forceinline__ int chunk_at(int r, int c) { return r * CH + (CH == 8 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)); }
    __device__ __forceinline__ void copy(int step, const Q8Maps &m)
    {
        if (step >= steps || lane != 0) return;
        const int slot = step % STAGES, t = key0 + step * STEP;
        const uint32_t bar = smem_u32(bars + slot), at = smem_u32(ring + slot * 2 * TILE);
        if (step == drop_copy) return;
        mbar_arrive_expect_tx(bar, 2 * TILE);
        load_states(at, &m.k, t, kh, kn, bar);
        load_states(at + TILE, &m.v, t, vh, vn, bar);
    }
    // The scales of a step's groups: a group past the valid length takes the last
    // valid state's, which is not used.
    __device__ __forceinline__ void next_scales(int step)
    {
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
            const int at = step < steps ? min(key0 + step * STEP + 16 * i, len - 1) >> log2_block : 0;
            scales[i] = ks[at];
            scales[GROUPS + i] = vs[at];
        }
    }
    __device__ __forceinline__ void begin(unsigned char *memory, uint64_t *barriers, const AttnQ8Args &a, const Q8Maps &m,
                                          const Q8Axes &ax, const TcTest &test, int n, int h, int split, int splits, int warp)
    {
        drop_copy = test.drop_copy;
        timeout_ns = test.timeout_ns;
        ring = memory;
        bars = barriers;
        lane = threadIdx.x & 31;
        if (lane < 2)   // the maps come beside the length
            asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<unsigned long long>(lane ? &m.v : &m.k)) : "memory");
        pdl_wait();
        len = a.Tk;
        if (a.k_len) len = max(0, min(len, a.k_len[n]));
        const int pieces = (len + KP - 1) / KP;
        const int p0 = (int)((long long)pieces * split / splits), p1 = (int)((long long)pieces * (split + 1) / splits);
        steps = p1 - p0 > warp ? (p1 - p0 - warp + kRowWarps - 1) / kRowWarps : 0;
        key0 = (p0 + warp) * KP;
        mb = a.key_mask ? a.key_mask + (long long)n * a.Tk : nullptr;
        kn = n * ax.k_n, kh = h * ax.k_h, vn = n * ax.v_n, vh = h * ax.v_h;
        if (lane == 0) {
            for (int i = 0; i < STAGES; ++i) mbar_init(smem_u32(bars + i), 1);
            fence_mbar_init();
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < STAGES; ++i) copy(i, m);
        log2_block = a.log2_block;
        ks = a.k_scale + ((long long)n * a.Hkv + h) * a.blocks;
        vs = a.v_scale + ((long long)n * a.Hkv + h) * a.blocks;
        next_scales(0);
        byte = mb ? mask_byte(0) : 0;
    }
    // Waits for a step's stage; valid: its states' bits, sc: its scales, late: it did not
    // come in time.
    __device__ __forceinline__ unsigned char *next(int step, uint32_t &valid, float (&sc)[2 * GROUPS], bool &late)
    {
#pragma unroll
        for (int i = 0; i < 2 * GROUPS; ++i) sc[i] = scales[i];
        next_scales(step + 1);
        if (mb) {
            valid = __ballot_sync(0xffffffffu, byte != 0);
            byte = mask_byte(step + 1);
        } else {
            const int left = len - (key0 + step * STEP);
            valid = left >= KP ? FULL : (1u << left) - 1u;
        }
        const int slot = step % STAGES;
        late = !mbar_wait_bounded(smem_u32(bars + slot), (step / STAGES) & 1, timeout_ns);
        return ring + slot * 2 * TILE;
    }
    // Behind a step that was late: the copies that are on their way get their time, a
    // thousand times what they take at least.
    __device__ __forceinline__ void drain(int step)
    {
        const unsigned long long limit = timeout_ns > 1000000ull ? timeout_ns : 1000000ull;
        for (int s = step; s < min(step + STAGES, steps); ++s)
            (void)mbar_wait_bounded(smem_u32(bars + s % STAGES), (s / STAGES) & 1, limit);
        __syncwarp();
    }
};

// The rings' memory becomes the warps' sums at the end; the cluster's sums have
// their own.
template <int DP, int R>
struct Q8Shared {
    union {
        unsigned char ring[kRowWarps][2 * Q8Ring<DP>::TILE * Q8Ring<DP>::STAGES];
        WarpSums<R, DP> warps;
    };
    CtaSums<R, DP> ctas;
    uint64_t bars[kRowWarps][Q8Ring<DP>::STAGES];
};

constexpr float kWeightLog2 = 14.f;   // weights are 2^14 P

// T: float or bf16 queries; R: 8 rows, or with bf16 16.
template <class T, int DP, bool E4M3, int R>
__global__ void __launch_bounds__(kRowThreads, R == 8 ? 2 : 1)
    attn_q8_kernel(const AttnQ8Args a, const RowsGeom g, const AttnPartials part, const __grid_constant__ Q8Maps maps, const Q8Axes axes,
                   const TcTest test)
{
    using Ring = Q8Ring<DP>;
    constexpr bool F32 = sizeof(T) == 4;
    constexpr int RH = R / 8;
    constexpr int KC = Ring::CH / 4;     // chunks of a key per lane
    constexpr int NT = DP / 8;           // products of 8 columns of O, one for each of the lane's bytes of a value
    static_assert(!F32 || RH == 1, "fp32: rows 8 to 15 are the second plane");
    extern __shared__ __align__(1024) unsigned char dyn[];
    Q8Shared<DP, R> &sm = *reinterpret_cast<Q8Shared<DP, R> *>(dyn);

    if (smem_u32(dyn) & 1023u) {   // the swizzled tiles need it; there is no static shared memory before them
        if (threadIdx.x == 0) atomicExch(axes.status, kDeviceTimeout);
        return;
    }
    pdl_trigger();   // the join kernel, or the next, may be set up; it waits for this grid's end
    if (g.cluster > 1) cluster_arrive();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gq = lane >> 2, t = lane & 3;
    const int split = blockIdx.x % g.splits;
    const int blk = blockIdx.x / g.splits;
    const int row0 = (blk % g.row_blocks) * R;
    const int nh = blk / g.row_blocks;
    const int n = nh / a.Hkv, h = nh - n * a.Hkv;
    const int rows = a.Tq * a.G;

    Ring ring;
    ring.begin(sm.ring[warp], sm.bars[warp], a, maps, axes, test, n, h, split, g.splits, warp);

    // the rows' queries times a power of two that puts a row's largest element in
    // [2^12, 2^13); back[] undoes it and carries scale log2 e
    uint32_t q[KC * 4][4];
    float back[RH];
    {
        float f[RH][KC][16];
#pragma unroll
        for (int r = 0; r < RH; ++r) {
            const int row = row0 + r * 8 + gq;
            const int tok = row / a.G, hq = h * a.G + row % a.G;
            float mx = 0.f;
            bool odd = false;
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const int d = (c * 4 + t) * 16;
#pragma unroll
                for (int i = 0; i < 16; ++i) f[r][c][i] = 0.f;
                if (row < rows && d < a.D) {
                    const T *p = static_cast<const T *>(a.q) + n * a.qs.n + tok * a.qs.t + hq * a.qs.h + d;
#pragma unroll
                    for (int i = 0; i < 16; i += 16 / (int)sizeof(T)) {
                        const uint4 v = ld16_once(p + i);
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if constexpr (F32) {
                                f[r][c][i + j] = __uint_as_float(w[j]);
                            } else {
                                f[r][c][i + 2 * j] = __uint_as_float(w[j] << 16);
                                f[r][c][i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
                            }
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    mx = fmaxf(mx, fabsf(f[r][c][i]));
                    odd |= !(fabsf(f[r][c][i]) < INFINITY);
                }
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const uint32_t odd_quad = __ballot_sync(0xffffffffu, odd) >> (lane & ~3) & 0xfu;
            // 2^(12 - exponent), in two steps where a row is tiny
            const int e = max((int)(__float_as_uint(mx) >> 23) - 127, -126);
            const int up = mx > 0.f ? 12 - e : 0;
            const float u0 = __uint_as_float((uint32_t)(127 + up / 2) << 23), u1 = __uint_as_float((uint32_t)(127 + up - up / 2) << 23);
            const float d0 = __uint_as_float((uint32_t)(127 - up / 2) << 23), d1 = __uint_as_float((uint32_t)(127 - (up - up / 2)) << 23);
            // an infinity or NaN makes the row NaN
            back[r] = odd_quad ? __uint_as_float(0x7fffffffu) : a.scale * kLog2e * d0 * d1;
#pragma unroll
            for (int c = 0; c < KC; ++c)
#pragma unroll
                for (int i = 0; i < 16; ++i) f[r][c][i] = odd_quad ? 0.f : f[r][c][i] * u0 * u1;
        }
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
            for (int w = 0; w < 4; ++w)
#pragma unroll
                for (int p = 0; p < 2; ++p) {   // operand registers (0, 1), (2, 3): the two pairs of a word of codes
                    const int i0 = 4 * w + byte_of<E4M3>(2 * p), i1 = 4 * w + byte_of<E4M3>(2 * p + 1);
                    const uint32_t hi = pack_f16(f[0][c][i0], f[0][c][i1]);
                    q[c * 4 + w][2 * p] = hi;
                    if constexpr (F32) {
                        const float2 x = unpack_f16(hi);
                        q[c * 4 + w][2 * p + 1] = pack_f16(f[0][c][i0] - x.x, f[0][c][i1] - x.y);
                    } else {
                        q[c * 4 + w][2 * p + 1] = RH == 2 ? pack_f16(f[RH - 1][c][i0], f[RH - 1][c][i1]) : 0u;
                    }
                }
    }

    float m[RH], l[RH], o[NT][2 * RH];   // m: the largest top, to which l and o are relative
#pragma unroll
    for (int r = 0; r < RH; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 2 * RH; ++i) o[j][i] = 0.f;

    for (int step = 0; step < ring.steps; ++step) {
        uint32_t ok;
        float sc[2 * Ring::GROUPS];
        bool late;
        unsigned char *tile = ring.next(step, ok, sc, late);
        const uint4 *kt = reinterpret_cast<const uint4 *>(tile), *vt = reinterpret_cast<const uint4 *>(tile + Ring::TILE);
        const bool full = ok == Ring::FULL;
        if (E4M3 && !full) {
            // values that are not valid: 0, as their weight times NaN is not
            if (lane < Ring::KP && !(ok >> lane & 1u)) {
                uint4 *row = reinterpret_cast<uint4 *>(tile + Ring::TILE) + lane * Ring::CH;
#pragma unroll
                for (int i = 0; i < Ring::CH; ++i) row[i] = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();   // before the next copy to this place
            __syncwarp();
        }

        float s[2 * Ring::GROUPS][4];
#pragma unroll
        for (int i = 0; i < 2 * Ring::GROUPS; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
            // column g of the scores is key 8 i + g
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const uint4 k = kt[Ring::chunk_at(8 * i + gq, c * 4 + t)];
                const uint32_t w[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint32_t b0, b1;
                    to_f16<E4M3>(w[x], b0, b1);
                    mma_f16(s[i], q[c * 4 + x], b0, b1);
                }
            }
        }
        // scores of row g (and g + 8) for the keys 8 i + 2 t and 8 i + 2 t + 1; top: what
        // a group's weights are relative to, its largest score less 14
        const bool joint = Ring::GROUPS == 2 && a.log2_block > 4 && (ok >> 16) != 0 && (ok & 0xffffu) != 0;   // one scale
        float top[Ring::GROUPS][RH];
        bool grow = false;
#pragma unroll
        for (int r = 0; r < RH; ++r) {
#pragma unroll
            for (int i = 0; i < Ring::GROUPS; ++i) {
                const float f = back[r] * sc[i];
                float mx = -INFINITY;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float &x = s[2 * i + e / 2][2 * r + e % 2];
                    if constexpr (F32) x += s[2 * i + e / 2][2 + e % 2];
                    x *= f;
                    if (!full) x = (ok >> (16 * i + 8 * (e / 2) + 2 * t + e % 2) & 1u) ? x : -INFINITY;
                    mx = fmaxf(mx, x);
                }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                top[i][r] = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) - kWeightLog2;
                grow |= top[i][r] > m[r];
            }
            if (joint) top[0][r] = top[Ring::GROUPS - 1][r] = fmaxf(top[0][r], top[Ring::GROUPS - 1][r]);
        }
        if (__any_sync(0xffffffffu, grow || late)) {
            if (__any_sync(0xffffffffu, late)) {   // the scores are of whatever was there: the warp's sums end here
                if (lane == 0) atomicExch(axes.status, kDeviceTimeout);
                ring.drain(step);
                break;
            }
#pragma unroll
            for (int r = 0; r < RH; ++r) {
                const float mm = fmaxf(m[r], fmaxf(top[0][r], top[Ring::GROUPS - 1][r]));
                const float f = mm == -INFINITY ? 1.f : ex2(m[r] - mm);
                m[r] = mm;
                l[r] *= f;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    o[j][2 * r] *= f;
                    o[j][2 * r + 1] *= f;
                }
            }
        }
        uint32_t p[Ring::GROUPS][4];
        float vs[Ring::GROUPS][RH];   // a group's factor: its scale, and its weights relative to m
#pragma unroll
        for (int r = 0; r < RH; ++r) {
            const float mr = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
            for (int i = 0; i < Ring::GROUPS; ++i) {
                const float f = ex2(top[i][r] - mr), ms = top[i][r] == -INFINITY ? 0.f : top[i][r];
                vs[i][r] = sc[Ring::GROUPS + i] * f;
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float x = ex2(s[2 * i + e][2 * r] - ms), y = ex2(s[2 * i + e][2 * r + 1] - ms);
                    sum += x + y;
                    const uint32_t hi = pack_f16(x, y);
                    p[i][2 * e + r] = hi;
                    if constexpr (F32) {
                        const float2 z = unpack_f16(hi);
                        p[i][2 * e + 1] = pack_f16(x - z.x, y - z.y);
                    } else if constexpr (RH == 1) {
                        p[i][2 * e + 1] = 0u;
                    }
                }
                l[r] = fmaf(sum, f, l[r]);
            }
        }
#pragma unroll
        for (int c = 0; c < NT / 8; ++c) {
            // the lane's eight bytes (half a chunk of 128-wide heads, whose 16 bytes come as two) of four keys a group
            uint2 v[Ring::GROUPS][4];
#pragma unroll
            for (int i = 0; i < Ring::GROUPS; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = 16 * i + 8 * (e / 2) + 2 * t + e % 2;
                    if constexpr (DP == 64)
                        v[i][e] = reinterpret_cast<const uint2 *>(vt + Ring::chunk_at(r, gq >> 1))[gq & 1];
                    else
                        v[i][e] = reinterpret_cast<const uint2 *>(vt + Ring::chunk_at(r, gq))[c];
                }
#pragma unroll
            for (int x = 0; x < 4; ++x) {   // bytes 2 x and 2 x + 1
                uint32_t b[Ring::GROUPS][2][2];
#pragma unroll
                for (int i = 0; i < Ring::GROUPS; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint2 &u0 = v[i][2 * e], &u1 = v[i][2 * e + 1];
                        const uint32_t w = x < 2 ? __byte_perm(u0.x, u1.x, gather<E4M3>(x)) : __byte_perm(u0.y, u1.y, gather<E4M3>(x - 2));
                        to_f16<E4M3>(w, b[i][0][e], b[i][1][e]);
                    }
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    float(&sum)[2 * RH] = o[c * 8 + 2 * x + y];
                    auto add = [&](const float (&acc)[4], const float (&f)[RH]) {
                        if constexpr (F32) {
                            sum[0] = fmaf(acc[0] + acc[2], f[0], sum[0]);
                            sum[1] = fmaf(acc[1] + acc[3], f[0], sum[1]);
                        } else {
#pragma unroll
                            for (int k = 0; k < 2 * RH; ++k) sum[k] = fmaf(acc[k], f[k / 2], sum[k]);
                        }
                    };
                    float acc[4] = {0.f, 0.f, 0.f, 0.f};
                    mma_f16(acc, p[0], b[0][y][0], b[0][y][1]);
                    if constexpr (Ring::GROUPS == 2) {
                        if (!joint) {
                            if (ok & 0xffffu) add(acc, vs[0]);
                            acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
                        }
                        mma_f16(acc, p[Ring::GROUPS - 1], b[Ring::GROUPS - 1][y][0], b[Ring::GROUPS - 1][y][1]);
                        if (joint || (ok >> 16)) add(acc, vs[Ring::GROUPS - 1]);
                    } else if (ok) {
                        add(acc, vs[0]);
                    }
                }
            }
        }
        __syncwarp();   // the stage has been read
        ring.copy(step + Ring::STAGES, maps);
    }
    __syncthreads();   // the rings' memory becomes the sums': every copy has been waited for

    // the warp's sums: row g (and g + 8); l over the quad
#pragma unroll
    for (int r = 0; r < RH; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        if (t == 0) {
            sm.warps.m[warp][r * 8 + gq] = m[r];
            sm.warps.l[warp][r * 8 + gq] = l[r];
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)   // column 2 t + e of product j is byte j of that lane group's part of the head
                sm.warps.o[warp][r * 8 + gq][(2 * t + e) * (DP / 8) + j] = o[j][2 * r + e];
    }
    finish_rows<T, R, DP>(sm.warps, sm.ctas, a, g, part, nh, row0, split);
}

PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

template <int DP>
bool encode_map(CUtensorMap *m, const void *p, const HeadStrides &s, const AttnQ8Args &a)
{
    // an axis of one element may come with any stride, one of stride 0 has one: the map wants a multiple of 16 above zero
    const cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)a.Tk, (cuuint64_t)(s.h ? a.Hkv : 1), (cuuint64_t)(s.n ? a.N : 1)};
    const cuuint64_t strides[3] = {a.Tk > 1 ? (cuuint64_t)s.t : 16, dims[2] > 1 ? (cuuint64_t)s.h : 16, dims[3] > 1 ? (cuuint64_t)s.n : 16};
    const cuuint32_t box[4] = {DP, Q8Ring<DP>::KP, 1, 1}, one[4] = {1, 1, 1, 1};
    return encoder()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     DP == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T, int DP, bool E4M3, int R>
cudaError_t launch_q8(const AttnQ8Args &a, cudaStream_t st, const TcTest &test)
{
    static KernelCache cache;
    Q8Axes ax{a.ks.n != 0, a.ks.h != 0, a.vs.n != 0, a.vs.h != 0, device_status_ptr()};
    if (!ax.status) return cudaErrorInvalidDevice;
    Q8Maps m;
    std::memset(&m, 0, sizeof(m));
    if (!encode_map<DP>(&m.k, a.k, a.ks, a) || !encode_map<DP>(&m.v, a.v, a.vs, a)) return cudaErrorInvalidValue;
    return launch_rows_kernel(attn_q8_kernel<T, DP, E4M3, R>, cache, a, sizeof(T) == 2, R, (int)sizeof(Q8Shared<DP, R>), st, true, m, ax,
                              test);
}

template <class T, bool E4M3>
cudaError_t dispatch(const AttnQ8Args &a, cudaStream_t st, const TcTest &test)
{
    if constexpr (sizeof(T) == 2) {
        if ((long long)a.Tq * a.G > 8) return a.D <= 64 ? launch_q8<T, 64, E4M3, 16>(a, st, test) : launch_q8<T, 128, E4M3, 16>(a, st, test);
    }
    return a.D <= 64 ? launch_q8<T, 64, E4M3, 8>(a, st, test) : launch_q8<T, 128, E4M3, 8>(a, st, test);
}

}  // namespace

cudaError_t launch_attn_q8(const AttnQ8Args &a, bool bf16, bool e4m3, cudaStream_t st, const TcTest &test)
{
    if (!encoder()) return cudaErrorNotSupported;
    if (bf16) return e4m3 ? dispatch<__nv_bfloat16, true>(a, st, test) : dispatch<__nv_bfloat16, false>(a, st, test);
    return e4m3 ? dispatch<float, true>(a, st, test) : dispatch<float, false>(a, st, test);
}

}  // namespace sc
