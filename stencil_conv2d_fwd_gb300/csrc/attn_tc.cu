// Attention of many query rows on the tensor cores (tcgen05, accumulators in
// tensor memory).
//
//   S = Q K^T,  P = 2^(c S - m),  O = P V,  out = O / sum_j P_j,   c = scale log2 e
//
// over tiles of 128 rows and 128 keys, in one pass over the keys: m and the
// sum are running values of a row.  A row is a (token, head of the group)
// pair, so the query heads that share a key head share its tiles.
//
// A CTA works on two streams, each with its S tile and its O accumulator in
// tensor memory; while one stream's softmax runs, the tensor cores work on
// the other.
//   * Two row tiles (PAIR): stream i is row tile i, and every key tile is used
//     by both.
//   * One row tile: stream i takes every other key tile; the two (m, sum, O)
//     are joined at the end.  Where every row tile has an SM of its own.
// P is handed over in two halves of the key tile, so that the first half's
// products run while the second half is made.
// Warps 0-3 and 4-7 are the streams' softmax, one thread per row (a warp
// reads the quadrant of tensor memory that it may address): scores from
// tensor memory, masked, 2^x, and P back to tensor memory as the second
// product's A operand, over the scores' columns.  With bf16 tensors O is
// rescaled only when a row's maximum has grown by more than 2^8 since the last
// rescaling (P then stays below 256); the division at the end cancels the
// common factor.  Warp 8 issues the TMA copies, warp 9 the MMAs.
// Warps 10 and 11 clear the value rows of states that a length or a mask
// leaves out (their weight is 0, but 0 times an infinity would not be).  Key
// tiles without a valid state are neither read nor computed with: the CTA
// first looks through its share of the mask and lists the others.  (To gather
// the valid states' rows alone, so that every tile is dense, cost more than
// the states left out: 32 x 77 queries over padded 56 x 56 maps, half of whose
// states are valid, 118 us by TMA gathers of four rows, 60 us by 16-byte
// copies, 45 us in place.)
//
// Accumulators, softmax and sums are fp32.  bf16 tensors: P is rounded to bf16
// for the second product (a relative error of 2^-8 of single terms, the size
// of the output's own rounding), and O stays in tensor memory.  fp32 tensors:
// Q, K, V (attn_split.cu) and P are three bf16 planes each, a product the six
// of planes i + j <= 2, the small ones first.  The tensor cores cut each sum
// short instead of rounding it, and over hundreds of products into one
// accumulator that adds up (1e-5 of the result at 3136 keys); so there O holds
// one key tile's product at a time, which the softmax threads add to sums of
// their own in registers.
//
// Bound (4 x 16384 queries over 3600 states, 16 heads of 128 bf16: 1.27 to 1.31
// ms, 1.50 PFLOP/s, 0.77 of the 1.94 that a large library product reaches here): the
// products' reads of shared memory.  A 128 x 128 x 16 product takes 64 clocks
// and reads 8 KB for S (the row and the key tile's slices), 4 KB for O, and the
// copies write 64 KB a pair of tiles, together what 128 bytes a clock allow;
// a pair of 128 x 128 tiles takes some 2800 clocks against 2048 of products
// alone, and starting and ending a CTA 6 of 85 thousand.  Two threads a row
// (20 warps) made it 6% slower: the softmax is not what is waited for.  With 64
// columns or fewer a product takes the same 64 clocks, so the O products of
// 64-wide heads run at half rate (the same queries over 16 heads of 64 bf16:
// 1.06 ms, 0.91 PFLOP/s): fp32 prompts (2 x 1001 queries over 3136 states, 8
// heads of 64: 80 us, 162 TFLOP/s of the formula, 6 times that in products) are
// bound by them.  fp32 heads of more than 64 have key tiles of 64, and it is the
// S products that run at half rate (8 heads of 128: 142 us, 182 TFLOP/s; 4 x
// 2048 queries over 3600 states, 16 heads: 1.03 ms, 235).  The two-row-tile
// form of the planes (PAIR) spills 80 bytes a softmax thread, the others less
// than 32.  Few row tiles are bound by reading keys and
// values (6.7 TB/s while the tiles run) and by a CTA's start and end, 4 us.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <cstring>
#include <mutex>

#include "attn.h"
#include "launch.h"
#include "tc_common.cuh"

namespace sc {

namespace at {

constexpr int TILE = 128;              // rows of a row tile
constexpr int BLK = TILE * 128;        // bytes of 128 rows of 64 bf16 (one 128-byte swizzled row each)
// Keys of a key tile.  Tensor memory of a stream (256 columns): the scores from
// 0, the first plane of P over them, the second from keys on; the third over
// the scores' second half (64 columns of O: read before it is written) or
// from 3/2 keys on; O the last DP.
template <int DP, int PL>
constexpr int key_tile() { return PL == 3 && DP == 128 ? 64 : 128; }
// Registers of the softmax warps and of the others, out of the 168 a thread
// that the block is launched with (launch() checks): 8 x 216 + 4 x 72 = 12 x 168.
constexpr int REGS_LAUNCH = 168, REGS_SOFTMAX = 216, REGS_OTHER = 72;
constexpr int THREADS = 384;
constexpr int MAX_SLOTS = 12;
constexpr int VC = 8;                  // barriers of cleared value tiles: more than the ring holds
constexpr int LIST = 512;              // key tiles of a share that are looked through; a longer share keeps all
constexpr int GRID_Y = 32768;          // (sequence, key head) pairs of a grid's y axis
constexpr float GROW = 8.f;            // log2 growth of a row's maximum that rescales O
constexpr size_t SMEM_CAP = 227 * 1024;

struct Geom {
    int row_tiles;        // row tiles of a (sequence, key head)
    int units;            // CTAs' row units of it: pairs of row tiles, or row tiles
    int tb, gb, gblocks;  // tokens and group heads of a row tile; blocks of gb heads
    int splits;           // CTAs that share a row unit's keys
    bool packed;          // q, k and v are the workspace's copies (attn_split.cu)
    int k_axes[2], v_axes[2];        // whether the maps' (h, n) are axes (1), or shared by all (0)
};

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void *tmap, int c0, int c1, int c2, int c3, int c4,
                                            uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];\n" ::
            "r"(dst),
        "l"(reinterpret_cast<unsigned long long>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
        : "memory");
}

// One thread of the warp (elect.sync).  The MMA warp runs its loops whole and
// predicates each instruction on this, so that the descriptors stay in uniform
// registers: issued from a branch of one lane, each product took some 130
// clocks to issue, twice what it takes to run.
__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t one;
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "elect.sync _|p, 0xffffffff;\n"
        "selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(one));
    return one;
}

// D[tmem] (+)= A[smem] B[smem] and D[tmem] (+)= A[tmem] B[smem], bf16 operands
__device__ __forceinline__ void mma_ss(uint32_t one, uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                       uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n"
        ".reg .pred p, q;\n"
        ".reg .b64 da, db;\n"
        "setp.ne.b32 p, %6, 0;\n"
        "setp.ne.b32 q, %7, 0;\n"
        "mov.b64 da, {%1, %2};\n"
        "mov.b64 db, {%3, %4};\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n"
        "}\n" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc), "r"(one)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t one, uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                       uint32_t acc)
{
    asm volatile(
        "{\n"
        ".reg .pred p, q;\n"
        ".reg .b64 db;\n"
        "setp.ne.b32 p, %5, 0;\n"
        "setp.ne.b32 q, %6, 0;\n"
        "mov.b64 db, {%2, %3};\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n"
        "}\n" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc), "r"(one)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t one, uint32_t bar)
{
    asm volatile(
        "{\n"
        ".reg .pred q;\n"
        "setp.ne.b32 q, %1, 0;\n"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n"
        "}\n" ::"r"(bar),
        "r"(one)
        : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// The largest of three, one instruction at the rate of a maximum of two.
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

template <int ID, int N>
__device__ __forceinline__ void named_sync()
{
    asm volatile("bar.sync %0, %1;\n" ::"n"(ID), "n"(N) : "memory");
}
template <int ID, int N>
__device__ __forceinline__ void named_arrive()
{
    asm volatile("bar.arrive %0, %1;\n" ::"n"(ID), "n"(N) : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *m)
{
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<unsigned long long>(m)) : "memory");
}

// Matrix descriptors' high words: 128-byte swizzle, 8-row groups 1024 bytes
// apart.  Low words: the start address; the second operand V is N-major, its
// 64-column blocks one block of key rows apart (desc_lo_v).
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t DESC_LO_K = 1u << 16;
constexpr uint32_t desc_lo_v(int key_tile) { return (uint32_t)(key_tile * 128 >> 4) << 16; }

template <bool PAIR>
struct Shared {
    // barriers of one arrival (`empty`: of the MMA warp and, where value rows
    // are cleared, the two clearing warps), of the two clearing warps, and of a
    // stream's four
    uint64_t full[MAX_SLOTS], empty[MAX_SLOTS], q_full, s_full[2], o_full[2], drain;
    uint64_t vclean[VC];
    uint64_t p_full[2][2];
    uint32_t words[2][2][4];           // valid bits of a key tile, per stream, two tiles deep
    float m[PAIR ? 1 : TILE], l[PAIR ? 1 : TILE];   // stream 1's, at the end
    uint16_t tiles[LIST];              // the share's key tiles that have a valid state
    uint8_t any[LIST];                 // whether a tile has one
    int count;
    uint32_t tmem;
    int abort;
};
constexpr int BARS_ONE = 2 * MAX_SLOTS + 6, BARS_TWO = BARS_ONE + VC, BARS = BARS_TWO + 4;

// Shared memory: row tiles (of one row tile at least the room of its 128 x DP
// fp32 sums, which the streams' join uses), the ring, then Shared.
template <int DP, int PL, bool PAIR>
constexpr int q_region()
{
    return (PAIR ? 2 * PL : (PL > 2 ? PL : 2)) * (DP / 64) * BLK;   // a multiple of 1024
}

template <int DP, int PL, bool PAIR>
constexpr int ring_slots()
{
    const int n = ((int)SMEM_CAP - q_region<DP, PL, PAIR>() - (int)sizeof(Shared<PAIR>)) / (DP / 64 * key_tile<DP, PL>() * 128);
    return n < MAX_SLOTS ? n : MAX_SLOTS;
}

template <bool B>
struct Bool {
    static constexpr bool value = B;
};

// PL operand planes: 1 (bf16 tensors), or 3 (fp32 tensors split into three
// bf16 planes, see attn_split.cu).
template <int DP, int PL, bool PAIR>
__global__ void __launch_bounds__(THREADS, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo, const AttnArgs a,
                   const Geom g, const AttnPartials part, int *status, const TcTest test)
{
    constexpr int DB = DP / 64;                 // 64-column blocks of a head
    constexpr int QT = PAIR ? 2 : 1;            // row tiles
    constexpr int KT = key_tile<DP, PL>();
    constexpr int KBLK = KT * 128;              // bytes of a key tile's rows of 64 bf16
    constexpr int SLOT = DB * KBLK;
    constexpr int SLOTS = ring_slots<DP, PL, PAIR>();
    extern __shared__ __align__(1024) unsigned char dyn[];
    Shared<PAIR> &sh = *reinterpret_cast<Shared<PAIR> *>(dyn + q_region<DP, PL, PAIR>() + SLOTS * SLOT);

    // (the shuffle makes the warp's number, and all that follows from it, uniform)
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t q_smem = smem_u32(dyn), ring = q_smem + q_region<DP, PL, PAIR>();
    if (q_smem & 1023u) {   // the swizzled tiles need it; there is no static shared memory before them
        if (tid == 0) atomicExch(status, kDeviceTimeout);
        return;
    }

    // what this CTA does
    const int nh = blockIdx.y + blockIdx.z * GRID_Y;
    if (nh >= a.N * a.Hkv) return;
    const int unit = g.splits == 1 ? blockIdx.x : blockIdx.x / g.splits;
    const int split = blockIdx.x - unit * g.splits;
    const int n = nh / a.Hkv, h = nh - n * a.Hkv;
    if (warp == 8 && lane < 4) prefetch_map(lane == 0 ? &mq : (lane == 1 ? &mk : (lane == 2 ? &mv : &mo)));
    int len = a.Tk;
    if (a.k_len) len = max(0, min(len, a.k_len[n]));
    const int tiles_all = (len + KT - 1) / KT;
    const int t_begin = (int)((long long)tiles_all * split / g.splits);
    const int t_end = (int)((long long)tiles_all * (split + 1) / g.splits);
    const int key_begin = t_begin * KT, key_end = min(len, t_end * KT);   // this CTA's share
    const unsigned char *mb = a.key_mask ? a.key_mask + (long long)n * a.Tk : nullptr;
    int nt = max(0, (key_end - key_begin + KT - 1) / KT);   // its key tiles, then those with a valid state
    const bool look = mb && nt <= LIST;
    auto tile_key = [&](int j) -> int { return key_begin + (look ? (int)sh.tiles[j] : j) * KT; };

    // A wait that runs out marks the CTA: every later wait returns at once and
    // all loops, which are finite, run to their end.
    volatile int *abort_flag = &sh.abort;
    auto wait = [&](uint64_t &bar, uint32_t parity) {
        const uint32_t b = smem_u32(&bar);
        if (mbar_try_wait(b, parity)) return;
        const unsigned long long t0 = global_ns();
        while (!mbar_try_wait(b, parity)) {
            if (*abort_flag) return;
            if (global_ns() - t0 > test.timeout_ns) {
                *abort_flag = 1;
                return;
            }
        }
    };

    // Order of the ring's tiles, the order in which the MMAs use them: the
    // first LAG key tiles, then value tile j and key tile j + LAG in turn.
    constexpr int LAG = PAIR ? 1 : 2;
    uint32_t issued = 0;          // ring entries whose copies have been issued
    // The copies of the seq-th tile.
    auto load_tile = [&](int seq) {
        const int l0 = min(LAG, nt), both = 2 * (nt - l0), s = seq - l0;
        const bool value = seq >= l0 && (s >= both || (s & 1) == 0);
        const int tile = seq < l0 ? seq : (s >= both ? nt - l0 + s - both : (value ? s / 2 : l0 + s / 2));
        const int *ax = value ? g.v_axes : g.k_axes;
        const int key0 = tile_key(tile);
        for (int p = PL - 1; p >= 0; --p, ++issued) {   // the smallest plane first
            const uint32_t slot = issued % SLOTS, round = issued / SLOTS;
            const uint32_t bar = smem_u32(&sh.full[slot]);
            if (round > 0) wait(sh.empty[slot], (round - 1) & 1);
            if (*abort_flag) return;
            if ((int)issued == test.drop_copy) continue;
            mbar_arrive_expect_tx(bar, SLOT);
            for (int d = 0; d < DB; ++d)
                tma_load_5d(ring + slot * SLOT + d * KBLK, value ? &mv : &mk, d * 64, key0, h * ax[0], n * ax[1], p, bar);
        }
    };

    if (warp == 8) {
        const int release = mb || len < a.Tk ? 3 : 1;   // arrivals of `empty`: 3 where value rows are cleared (`ragged` below)
        for (int i = lane; i < BARS; i += 32)
            mbar_init(smem_u32(&sh.full[0]) + 8 * i,
                      i < BARS_ONE ? (i >= MAX_SLOTS && i < 2 * MAX_SLOTS ? release : 1) : (i < BARS_TWO ? 2 : 4));
        if (lane == 0) sh.abort = 0;
        fence_mbar_init();
        __syncwarp();
        if (g.packed) pdl_wait();   // the copies read what the launch before has written
        if (lane == 0 && nt > 0) {
            // row tiles: tokens and heads past the end read as zero
            mbar_arrive_expect_tx(smem_u32(&sh.q_full), (uint32_t)(QT * PL * DB * g.gb * g.tb * 128));
            for (int i = 0; i < QT; ++i) {
                const int rt = unit * QT + i;
                const int tok = rt / g.gblocks * g.tb, gh = rt % g.gblocks * g.gb;
                for (int p = 0; p < PL; ++p)
                    for (int d = 0; d < DB; ++d)
                        tma_load_5d(q_smem + ((i * PL + p) * DB + d) * BLK, &mq, d * 64, gh, tok, g.packed ? nh : h,
                                    g.packed ? p : n, smem_u32(&sh.q_full));
            }
        }
        __syncwarp();
    } else if (warp == 9) {
        tc::tmem_alloc(smem_u32(&sh.tmem), 512);
    }
    if (look) {
#pragma unroll 2
        for (int j = warp; j < nt; j += THREADS / 32) {
            int any = 0;
#pragma unroll
            for (int i = 0; i < KT / 32; ++i) {
                const int key = key_begin + j * KT + 32 * i + lane;
                any |= key < key_end ? (int)mb[key] : 0;
            }
            any = __any_sync(0xffffffffu, any != 0);
            if (lane == 0) sh.any[j] = (uint8_t)any;
        }
    }
    tc::fence_before_sync();
    // the copying warp goes on: the first copies' latency runs beside the
    // allocation, and the others do not wait until it has issued them
    if (warp == 8 && !look)
        named_arrive<4, THREADS>();
    else
        named_sync<4, THREADS>();
    tc::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem, 0);
    const int q_tiles = nt;   // the row tiles have been asked for
    if (look) {
        if (warp == 8) {
            int count = 0;
            for (int j0 = 0; j0 < nt; j0 += 32) {
                const uint32_t on = __ballot_sync(0xffffffffu, j0 + lane < nt && sh.any[j0 + lane] != 0);
                if (on >> lane & 1u) sh.tiles[count + __popc(on & ((1u << lane) - 1u))] = (uint16_t)(j0 + lane);
                count += __popc(on);
            }
            if (lane == 0) sh.count = count;
        }
        __syncthreads();
        nt = sh.count;
    }
    const bool ragged = mb || len < a.Tk;
    constexpr int P1 = KT, P2 = DP == 64 ? KT / 2 : KT + KT / 2, TO = 256 - DP;   // columns of a stream
    auto p_plane = [](int p) { return p == 0 ? 0 : (p == 1 ? P1 : P2); };

    if (warp >= 8) {
        // one instruction for the four warps, as its form asks
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(REGS_OTHER));
        if (warp == 8) {
            if (lane == 0) {
                for (int seq = 0; seq < 2 * nt; ++seq) load_tile(seq);
                // a mask that leaves nothing: no one else waits for the row tiles
                if (nt == 0 && q_tiles > 0) wait(sh.q_full, 0);
            }
            __syncwarp();
        } else if (warp == 9) {
            if (nt > 0) {
                const uint32_t one = elect_one();
                const uint32_t idesc_s = tc::idesc_mma(1, KT), idesc_v = tc::idesc_mma(1, (a.D + 15) / 16 * 16) | (1u << 16);
                wait(sh.q_full, 0);
                // S of stream i from the key tile whose first plane is ring entry c
                auto mma_s = [&](int i, uint32_t c, bool release) {
#pragma unroll
                    for (int pk = PL - 1; pk >= 0; --pk, ++c) {
                        const uint32_t slot = c % SLOTS;
                        wait(sh.full[slot], (c / SLOTS) & 1);
                        tc::fence_after_sync();
                        const uint32_t kb = ((ring + slot * SLOT) >> 4) | DESC_LO_K;
#pragma unroll
                        for (int pq = PL - 1 - pk; pq >= 0; --pq) {
                            const uint32_t qb = ((q_smem + ((PAIR ? i : 0) * PL + pq) * DB * BLK) >> 4) | DESC_LO_K;
#pragma unroll
                            for (int k = 0; k < DP / 16; ++k)
                                if (k * 16 < a.D)
                                    mma_ss(one, tmem + i * 256, qb + ((k >> 2) * BLK + (k & 3) * 32) / 16, DESC_HI,
                                           kb + ((k >> 2) * KBLK + (k & 3) * 32) / 16, DESC_HI, idesc_s,
                                           pk != PL - 1 || pq != PL - 1 - pk || k > 0);
                        }
                        if (release) mma_commit(one, smem_u32(&sh.empty[slot]));
                    }
                    mma_commit(one, smem_u32(&sh.s_full[i]));
                };
                // O of stream i = P V (fp32 tensors), or += P V; use = the stream's count of P tiles so far
                // P comes in two halves of the key tile: the first half's products run while the second is made
                auto mma_v = [&](int i, uint32_t c, int j, uint32_t use, bool release, bool last) {
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        wait(sh.p_full[i][part], use & 1);
                        if (part == 0 && ragged) wait(sh.vclean[j % VC], (j / VC) & 1);
                        tc::fence_after_sync();
#pragma unroll
                        for (int pv = PL - 1; pv >= 0; --pv) {
                            const uint32_t e = c + (PL - 1 - pv), slot = e % SLOTS;
                            if (part == 0) {
                                wait(sh.full[slot], (e / SLOTS) & 1);
                                tc::fence_after_sync();
                            }
                            const uint32_t vb = ((ring + slot * SLOT) >> 4) | desc_lo_v(KT);
#pragma unroll
                            for (int pp = PL - 1 - pv; pp >= 0; --pp)
#pragma unroll
                                for (int k = part * KT / 32; k < (part + 1) * KT / 32; ++k)
                                    mma_ts(one, tmem + i * 256 + TO, tmem + i * 256 + p_plane(pp) + k * 8, vb + k * 128,
                                           DESC_HI, idesc_v,
                                           pv != PL - 1 || pp != PL - 1 - pv || k > 0 || (PL == 1 && use > 0));
                            if (part == 1 && release) mma_commit(one, smem_u32(&sh.empty[slot]));
                        }
                    }
                    if (last) mma_commit(one, smem_u32(&sh.o_full[i]));
                };
                if constexpr (PAIR) {
                    mma_s(0, 0, false);
                    mma_s(1, 0, true);
                    uint32_t c = PL;
                    for (int j = 0; j < nt; ++j) {
                        const bool more = j + 1 < nt;
                        mma_v(0, c, j, j, false, !more);
                        if (more) mma_s(0, c + PL, false);
                        mma_v(1, c, j, j, true, !more);
                        if (more) mma_s(1, c + PL, true);
                        c += more ? 2 * PL : PL;
                    }
                } else {
                    mma_s(0, 0, true);
                    if (nt > 1) mma_s(1, PL, true);
                    uint32_t c = nt > 1 ? 2 * PL : PL;
                    for (int j = 0; j < nt; ++j) {
                        const bool more = j + 2 < nt;
                        mma_v(j & 1, c, j, j >> 1, true, !more);
                        c += PL;
                        if (more) {
                            mma_s(j & 1, c, true);
                            c += PL;
                        }
                    }
                }
            }
            __syncwarp();
        } else if (ragged) {
            // value rows that are not valid: zero, in every plane and block.
            // A barrier's parity tells a round only from its neighbours, so these
            // warps wait for every entry of the ring in turn, the key tiles' too,
            // and each entry's release waits for them: a slot's next copy is not
            // asked for before both have seen this one, however late they are.
            uint32_t c = 0;
            auto seen = [&]() {   // the next entry's copy
                if (test.clear_delay_ns > 0)
                    for (const unsigned long long t0 = global_ns(); global_ns() - t0 < test.clear_delay_ns;) {}
                wait(sh.full[c % SLOTS], (c / SLOTS) & 1);
            };
            auto release = [&](uint32_t entry) { mbar_arrive(smem_u32(&sh.empty[entry % SLOTS])); };
            auto pass = [&]() {   // a key tile
#pragma unroll 1   // (unrolled, these loops cost the softmax warps of the three-plane pairs 300 bytes of spills)
                for (int p = 0; p < PL; ++p, ++c) {
                    seen();
                    __syncwarp();
                    if (lane == 0) release(c);
                }
            };
            for (int j = 0; j < LAG && j < nt; ++j) pass();
            constexpr int KL = KT / 64;   // keys of a lane: two warps share the tile
            const int row0 = (warp - 10) * 32 * KL + lane;
            for (int j = 0; j < nt; ++j) {
                const int key0 = tile_key(j);
                bool bad[KL];
#pragma unroll
                for (int i = 0; i < KL; ++i) {
                    const int key = key0 + row0 + i * 32;
                    // states past Tk are not in the tensor and read as zero
                    bad[i] = key < a.Tk && (key >= len || (mb && mb[key] == 0));
                }
#pragma unroll 1
                for (int p = 0; p < PL; ++p, ++c) {
                    const uint32_t slot = c % SLOTS;
                    seen();
#pragma unroll
                    for (int i = 0; i < KL; ++i) {
                        if (!bad[i]) continue;
                        const uint32_t at = ring + slot * SLOT + (row0 + i * 32) * 128;
                        for (int d = 0; d < DB; ++d)
#pragma unroll
                            for (int e = 0; e < 8; ++e)   // from chunk `lane` on: no two lanes in one bank
                                tc::st_shared_v4(at + d * KBLK + ((e + lane) & 7) * 16, 0u, 0u, 0u, 0u);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&sh.vclean[j % VC]));
#pragma unroll 1
                    for (int p = 1; p <= PL; ++p) release(c - p);
                }
                if (j + LAG < nt) pass();
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(REGS_SOFTMAX));
        const int i = warp >> 2;                   // stream
        const int row = (warp & 3) * 32 + lane;    // row of the tile
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + i * 256 + lanes, to = ts + TO;
        const int step = PAIR ? 1 : 2;
        const float c = a.scale * kLog2e;
        float m = -INFINITY, l = 0.f;   // m: maximum that P is relative to, in units of log2
        float acc[PL == 3 ? DP : 1];    // fp32 tensors: the row's sums, relative to m
#pragma unroll
        for (int d = 0; d < (PL == 3 ? DP : 1); ++d) acc[d] = 0.f;
        constexpr int KW = KT / 32;     // words of a tile's valid bits
        int use = 0;
        // this thread's byte of key tile j: 0 where the state is not valid
        auto mask_byte = [&](int j) {
            if (j >= nt || row >= KT) return 0;
            const int key = tile_key(j) + row;
            return key < len ? (int)mb[key] : 0;
        };
        int next = mb ? mask_byte(PAIR ? 0 : i) : 0;
        // half of a key tile's P is in tensor memory
        auto hand_over = [&](int part) {
            tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.p_full[i][part]));
        };
        // 32 scores from column 32 e; those that are not valid become -infinity
        auto load_scores = [&](int e, uint32_t (&s)[32], uint32_t w, bool masked) {
            tc::tmem_ld<32>(ts + e * 32, s);
            tc::tmem_wait_ld();
            if (masked) {
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    if (!((w >> k) & 1u)) s[k] = 0xff800000u;
            }
        };
        for (int j = PAIR ? 0 : i; j < nt; j += step, ++use) {
            const int key0 = tile_key(j);
            uint32_t w[KW];
            bool masked = key0 + KT > len;
            if (mb) {
                // one key per thread, a word per warp; the next tile's byte is
                // read a tile ahead (its latency was a third of a masked tile's time)
                const uint32_t word = __ballot_sync(0xffffffffu, next != 0);
                next = mask_byte(j + step);
                if (lane == 0) sh.words[i][use & 1][warp & 3] = word;
                if (i == 0)
                    named_sync<1, 128>();
                else
                    named_sync<2, 128>();
                uint32_t all = ~0u;
#pragma unroll
                for (int e = 0; e < KW; ++e) {
                    w[e] = sh.words[i][use & 1][e];
                    all &= w[e];
                }
                masked = all != ~0u;
            } else {
#pragma unroll
                for (int e = 0; e < KW; ++e) {
                    const int left = len - key0 - 32 * e;
                    w[e] = left >= 32 ? ~0u : (left <= 0 ? 0u : (1u << left) - 1u);
                }
            }
            wait(sh.s_full[i], use & 1);
            tc::fence_after_sync();
            if constexpr (PL == 1) {
                uint32_t s[4][32];
#pragma unroll
                for (int e = 0; e < 4; ++e) tc::tmem_ld<32>(ts + e * 32, s[e]);
                tc::tmem_wait_ld();
                if (masked) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (!((w[e] >> k) & 1u)) s[e][k] = 0xff800000u;
                }
                float mx[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    mx[e] = __uint_as_float(s[e][0]);
#pragma unroll
                    for (int k = 1; k < 31; k += 2)
                        mx[e] = max3(mx[e], __uint_as_float(s[e][k]), __uint_as_float(s[e][k + 1]));
                    mx[e] = fmaxf(mx[e], __uint_as_float(s[e][31]));
                }
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
                const bool grow = top - m > GROW;   // false where both are -infinity
                float f = 1.f;
                if (grow) {
                    f = ex2(m - top);
                    m = top;
                    l *= f;
                }
                if (use > 0 && __any_sync(0xffffffffu, grow)) {
                    // the stream's last product is complete: it was issued before this S
                    for (int d = 0; d < DP; d += 32) {
                        if (d >= a.D) break;
                        uint32_t o[32];
                        tc::tmem_ld<32>(to + d, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                        tmem_st32(to + d, o);
                    }
                }
                const float mc = m == -INFINITY ? 0.f : m;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    uint32_t p[32];
#pragma unroll
                    for (int k = 0; k < 64; k += 2) {
                        const float x = ex2(fmaf(__uint_as_float(s[e + k / 32][k % 32]), c, -mc));
                        const float y = ex2(fmaf(__uint_as_float(s[e + k / 32][k % 32 + 1]), c, -mc));
                        sum[e + k / 32] += x;
                        sum[(e + k / 32) ^ 1] += y;
                        p[k / 2] = tc::pack_bf16(x, y);
                    }
                    tmem_st32(ts + e * 16, p);
                    hand_over(e / 2);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            } else {
                // the scores' second half stays in registers where P's third
                // plane is written over it
                constexpr int HOLD = DP == 64 ? KW / 2 : 0;
                uint32_t hold[HOLD > 0 ? HOLD : 1][32];
                float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < KW; ++e) {
                    uint32_t s[32];
                    load_scores(e, s, w[e], masked);
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        mx[k / 2 & 1] = max3(mx[k / 2 & 1], __uint_as_float(s[k]), __uint_as_float(s[k + 1]));
                        if (e >= KW - HOLD) {
                            hold[e - (KW - HOLD)][k] = s[k];
                            hold[e - (KW - HOLD)][k + 1] = s[k + 1];
                        }
                    }
                }
                const float top = fmaxf(fmaxf(mx[0], mx[1]) * c, m);
                const float mc = top == -INFINITY ? 0.f : top, f = ex2(m - mc);   // 1 or less; 0 at the first scores
                m = top;
                // the last tile's product, relative to the last maximum; it is
                // complete: it was issued before this S
                if (use > 0) {
#pragma unroll
                    for (int d = 0; d < DP; d += 16) {
                        if (d < a.D) {
                            uint32_t o[16];
                            tc::tmem_ld<16>(to + d, o);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; ++k) acc[d + k] = (acc[d + k] + __uint_as_float(o[k])) * f;
                        }
                    }
                }
                float sum[2] = {0.f, 0.f};
#pragma unroll
                for (int e = 0; e < KW; ++e) {
                    uint32_t s[32];
                    if (e < KW - HOLD) {
                        load_scores(e, s, w[e], masked);
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k) s[k] = hold[HOLD > 0 ? e - (KW - HOLD) : 0][k];
                    }
#pragma unroll
                    for (int q = 0; q < 32; q += 16) {
                        uint32_t p0[8], p1[8], p2[8];
#pragma unroll
                        for (int k = 0; k < 16; k += 2) {
                            float x = ex2(fmaf(__uint_as_float(s[q + k]), c, -mc));
                            float y = ex2(fmaf(__uint_as_float(s[q + k + 1]), c, -mc));
                            sum[0] += x;
                            sum[1] += y;
                            p0[k / 2] = tc::pack_bf16(x, y);
                            x -= __uint_as_float(p0[k / 2] << 16);
                            y -= __uint_as_float(p0[k / 2] & 0xffff0000u);
                            p1[k / 2] = tc::pack_bf16(x, y);
                            p2[k / 2] = tc::pack_bf16(x - __uint_as_float(p1[k / 2] << 16),
                                                      y - __uint_as_float(p1[k / 2] & 0xffff0000u));
                        }
                        tmem_st8(ts + (32 * e + q) / 2, p0);
                        tmem_st8(ts + P1 + (32 * e + q) / 2, p1);
                        tmem_st8(ts + P2 + (32 * e + q) / 2, p2);
                    }
                    if (e == KW / 2 - 1) hand_over(0);
                    if (e == KW - 1) hand_over(1);
                }
                l = l * f + (sum[0] + sum[1]);
            }
        }
        if (use > 0) {
            wait(sh.o_full[i], 0);
            tc::fence_after_sync();
        }
        // 32 of the row's sums, from column d
        auto row_sums = [&](int d, float (&y)[32]) {
            uint32_t o[32];
            tc::tmem_ld<32>(to + d, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) y[k] = __uint_as_float(o[k]) + (PL == 3 ? acc[PL == 3 ? d + k : 0] : 0.f);
        };
        // this thread's row
        const int rt = PAIR ? unit * 2 + i : unit;
        const int tok = rt / g.gblocks * g.tb + row / g.gb, gh = rt % g.gblocks * g.gb + row % g.gb;
        const bool live = rt < g.row_tiles && row < g.gb * g.tb && tok < a.Tq && gh < a.G;
        const int hq = h * a.G + gh;
        // the joined (m, l) and the factors of the streams' O
        float f0 = 1.f, f1 = 0.f;
        float *stage = reinterpret_cast<float *>(dyn);
        if constexpr (!PAIR) {
            // stream 1 hands its sums over in the row tile's shared memory (the
            // scores' products are complete once either stream's O is), one
            // column of 128 rows after the other
            if (i == 1) {
                sh.m[row] = m;
                sh.l[row] = l;
                if (use > 0) {
#pragma unroll
                    for (int d = 0; d < DP; d += 32) {
                        if (d < a.D) {
                            float y[32];
                            row_sums(d, y);
#pragma unroll
                            for (int k = 0; k < 32; ++k) stage[(d + k) * TILE + row] = y[k];
                        }
                    }
                }
                named_sync<3, 256>();
            } else {
                named_sync<3, 256>();
                const float m1 = sh.m[row], l1 = sh.l[row];
                const float mm = fmaxf(m, m1), ms = mm == -INFINITY ? 0.f : mm;
                f0 = ex2(m - ms);
                f1 = ex2(m1 - ms);
                l = l * f0 + l1 * f1;
                m = mm;
            }
        }
        if (PAIR || i == 0) {
            const bool any = nt > 0, two = !PAIR && nt > 1;
            const bool final_out = part.parts == 0;
            const float inv = final_out ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
            // The row tile goes to memory by TMA (rows and columns past the
            // tensor's end are left out), from shared memory that is free by
            // now: the stream's own row tile of Q (its scores' products are
            // complete), or with one row tile the ring.  (16-byte stores of 128
            // rows to 128 lines each took 2 us of a CTA's 22.)
            if (nt == 0 && q_tiles > 0) wait(sh.q_full, 0);
            unsigned char *tile = dyn + (PAIR ? i * PL * DB * BLK : q_region<DP, PL, PAIR>());
            constexpr int ROOM = PAIR ? PL * DB : SLOTS * SLOT / BLK;   // blocks of 128 rows of 128 bytes
            auto store = [&](auto out_bf16) {
                constexpr bool OB = decltype(out_bf16)::value;
                constexpr int CB = OB ? 64 : 32, NB = DP / CB;   // columns of a block, blocks
                constexpr int GRP = NB < ROOM ? NB : ROOM;       // blocks at a time
#pragma unroll
                for (int b0 = 0; b0 < NB; b0 += GRP) {
#pragma unroll
                    for (int d = b0 * CB; d < (b0 + GRP) * CB; d += 32) {
                        if (d >= a.D) continue;
                        float y[32];
                        if (any) {
                            row_sums(d, y);
                        } else {
#pragma unroll
                            for (int k = 0; k < 32; ++k) y[k] = 0.f;
                        }
                        uint32_t w[OB ? 16 : 32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            float v = y[k] * f0;
                            if (two) v = fmaf(stage[(d + k) * TILE + row], f1, v);
                            y[k] = l == 0.f ? 0.f : v * inv;
                        }
#pragma unroll
                        for (int k = 0; k < (OB ? 16 : 32); ++k)
                            w[k] = OB ? tc::pack_bf16(y[OB ? 2 * k : k], y[OB ? 2 * k + 1 : k]) : __float_as_uint(y[k]);
                        const uint32_t at = smem_u32(tile) + (d / CB - b0) * BLK + row * 128;
                        const int c0 = d % CB * (OB ? 2 : 4) / 16;   // 16-byte chunks, swizzled as the copies expect
#pragma unroll
                        for (int k = 0; k < (OB ? 4 : 8); ++k)
                            tc::st_shared_v4(at + (((c0 + k) ^ (row & 7)) << 4), w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                    }
                    fence_proxy_async_smem();
                    if (i == 0)
                        named_sync<1, 128>();
                    else
                        named_sync<2, 128>();
                    if (row == 0 && rt < g.row_tiles) {
                        const int tok0 = rt / g.gblocks * g.tb, gh0 = rt % g.gblocks * g.gb;
                        for (int b = b0; b < b0 + GRP && b * CB < a.D; ++b)
                            tma_store_5d(&mo, smem_u32(tile) + (b - b0) * BLK, b * CB, gh0, tok0, final_out ? h : nh,
                                         final_out ? n : split);
                        bulk_commit();
                        bulk_wait_read<0>();   // the writes end with the grid, the reads of shared memory before the CTA
                    }
                    if (b0 + GRP < NB) {   // the blocks are written over
                        if (i == 0)
                            named_sync<1, 128>();
                        else
                            named_sync<2, 128>();
                    }
                }
            };
            if (PL == 1 && final_out)
                store(Bool<PL == 1>{});
            else
                store(Bool<false>{});
            if (live) {
                if (!final_out)
                    part.ml[((long long)split * a.N * a.Hkv + nh) * ((long long)a.Tq * a.G) + (long long)tok * a.G + gh] =
                        make_float2(m, l);
                else if (a.lse)
                    a.lse[((long long)n * a.Hq + hq) * a.Tq + tok] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
            }
        }
        tc::fence_before_sync();
    }
    __syncthreads();
    if (sh.abort) {
        // give the copies and products in flight their time to end before the
        // shared and tensor memory are given back
        if (tid == 0) atomicExch(status, kDeviceTimeout);
        if (warp == 8 && lane == 0) {
            if (q_tiles > 0) (void)mbar_wait_bounded(smem_u32(&sh.q_full), 0, test.timeout_ns);
            for (uint32_t e = issued > (uint32_t)SLOTS ? issued - SLOTS : 0; e < issued; ++e)
                (void)mbar_wait_bounded(smem_u32(&sh.full[e % SLOTS]), (e / SLOTS) & 1, test.timeout_ns);
        }
        if (warp == 9) {
            mma_commit(elect_one(), smem_u32(&sh.drain));   // by the thread that issued the products
            (void)mbar_wait_bounded(smem_u32(&sh.drain), 0, test.timeout_ns);
            __syncwarp();
        }
        __syncthreads();
    }
    if (warp == 9) tc::tmem_dealloc(tmem, 512);
}

PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// A map of rows of D elements with four outer axes (strides in bytes), boxes of
// 128 bytes of box1 x box2 rows.
bool encode_map(CUtensorMap *m, bool bf16, const void *base, int D, const long long (&size)[4], const long long (&stride)[4],
                int box1, int box2)
{
    cuuint64_t dims[5] = {(cuuint64_t)D}, strides[4];
    for (int i = 0; i < 4; ++i) {
        dims[i + 1] = (cuuint64_t)size[i];
        // an axis of one element may come with any stride: the map wants a
        // multiple of 16 above zero
        strides[i] = size[i] == 1 ? 16 : (cuuint64_t)stride[i];
    }
    const cuuint32_t box[5] = {bf16 ? 64u : 32u, (cuuint32_t)box1, (cuuint32_t)box2, 1, 1};
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    return encoder()(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 5,
                     const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Maps {
    CUtensorMap q, k, v, out;
};

template <int DP, int PL, bool PAIR>
cudaError_t launch(const AttnArgs &a, const Geom &g, const Maps &m, const AttnPartials &part, cudaStream_t st,
                   const TcTest &test)
{
    constexpr int SMEM = q_region<DP, PL, PAIR>() + ring_slots<DP, PL, PAIR>() * (DP / 64 * key_tile<DP, PL>() * 128) +
                         (int)sizeof(Shared<PAIR>);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    static KernelCache cache;
    e = ensure_dynamic_smem(cache, dev, attn_tc_kernel<DP, PL, PAIR>, SMEM);
    if (e != cudaSuccess) return e;
    // the register split is of REGS_LAUNCH a thread: with fewer, a warp would wait for registers that never come
    static const int regs = [] {
        cudaFuncAttributes fa = {};
        return cudaFuncGetAttributes(&fa, attn_tc_kernel<DP, PL, PAIR>) == cudaSuccess ? fa.numRegs : 0;
    }();
    if (regs != REGS_LAUNCH) return cudaErrorNotSupported;
    int *status = device_status_ptr();
    if (!status) return cudaErrorInvalidDevice;
    const long long x = (long long)g.units * g.splits, nh = (long long)a.N * a.Hkv;
    if (x > 0x7fffffffLL || nh > (long long)GRID_Y * 65535) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)x, (unsigned)(nh < GRID_Y ? nh : GRID_Y), (unsigned)((nh + GRID_Y - 1) / GRID_Y));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = g.packed ? 1 : 0;   // behind attn_split's launch
    return cudaLaunchKernelEx(&cfg, attn_tc_kernel<DP, PL, PAIR>, m.q, m.k, m.v, m.out, a, g, part, status, test);
}

}  // namespace at

cudaError_t launch_attn_tc(const AttnArgs &a, bool bf16, cudaStream_t st, const TcTest &test)
{
    if (!at::encoder()) return cudaErrorNotSupported;
    at::Geom g = {};
    g.gb = a.G < at::TILE ? a.G : at::TILE;
    g.tb = at::TILE / g.gb;
    g.gblocks = (a.G + g.gb - 1) / g.gb;
    const long long rt = (long long)((a.Tq + g.tb - 1) / g.tb) * g.gblocks;
    if (rt > 0x3fffffffLL) return cudaErrorInvalidConfiguration;
    g.row_tiles = (int)rt;
    // two row tiles of three planes of 128 columns do not fit in shared memory
    // (nor is there a reason to pair them where each has an SM of its own)
    const bool pair = (bf16 || a.D <= 64) && g.row_tiles > 1 &&
                      (long long)a.N * a.Hkv * g.row_tiles > device_sm_count();
    g.units = pair ? (g.row_tiles + 1) / 2 : g.row_tiles;
    // CTAs per row unit: fill the GPU, at least four key tiles each (2 x 8 key
    // heads, 77 rows, 25 tiles: 14.4 us, at least eight 16.4, sixteen 24.6; two of
    // 9000 keys, 17 rows: 14.3, 16.4, 22.5), and none for fewer than
    // twelve tiles, whose join costs what it saves
    const long long blocks = (long long)a.N * a.Hkv * g.units;
    const int kt = bf16 ? at::key_tile<64, 1>() : (a.D <= 64 ? at::key_tile<64, 3>() : at::key_tile<128, 3>());
    const long long tiles = (a.Tk + kt - 1) / kt;
    long long splits = device_sm_count() / blocks;
    if (splits > tiles / 4) splits = tiles / 4;
    if (splits < 1 || tiles < 12) splits = 1;
    g.splits = (int)splits;

    // fp32 tensors are split into planes; bf16 ones are used as they lie where
    // the TMA copies can address them: axes of the row and key tiles that are
    // not shared
    g.packed = !bf16 || (a.G > 1 && a.qs.h == 0) || (a.Tq > 1 && a.qs.t == 0) || (a.Hkv > 1 && a.qs.h == 0) ||
               (a.N > 1 && a.qs.n == 0) || (a.Tk > 1 && (a.ks.t == 0 || a.vs.t == 0));
    const int planes = bf16 ? 1 : 3;
    const long long rows = (long long)a.N * a.Hq * a.Tq, keys = (long long)a.N * a.Hkv * a.Tk;
    g.k_axes[0] = g.packed || a.ks.h != 0;
    g.k_axes[1] = g.packed || a.ks.n != 0;
    g.v_axes[0] = g.packed || a.vs.h != 0;
    g.v_axes[1] = g.packed || a.vs.n != 0;

    // workspace: partial results, and the packed tensors
    auto pad = [](size_t b) { return (b + 255) & ~(size_t)255; };
    const size_t po = g.splits > 1 ? pad((size_t)g.splits * rows * a.D * 4) : 0;
    const size_t pml = g.splits > 1 ? pad((size_t)g.splits * rows * sizeof(float2)) : 0;
    const size_t pq = g.packed ? pad((size_t)rows * a.D * 2 * planes) : 0;
    const size_t pk = g.packed ? pad((size_t)keys * a.D * 2 * planes) : 0;
    char *ws = nullptr;
    if (po + pml + pq + pk > 0) {
        const cudaError_t e = workspace_alloc(reinterpret_cast<void **>(&ws), po + pml + pq + 2 * pk, st);
        if (e != cudaSuccess) return e;
    }
    AttnPartials part{nullptr, nullptr, 0};
    if (g.splits > 1) part = AttnPartials{reinterpret_cast<float *>(ws), reinterpret_cast<float2 *>(ws + po), g.splits};
    void *const plane[3] = {ws + po + pml, ws + po + pml + pq, ws + po + pml + pq + pk};

    at::Maps m;
    std::memset(&m, 0, sizeof(m));
    bool ok;
    const void *k = g.packed ? plane[1] : a.k, *v = g.packed ? plane[2] : a.v;
    if (g.packed) {
        const long long size[4] = {a.G, a.Tq, (long long)a.N * a.Hkv, planes}, d = a.D * 2LL;
        const long long stride[4] = {d, d * a.G, d * a.G * a.Tq, d * rows};
        ok = at::encode_map(&m.q, true, plane[0], a.D, size, stride, g.gb, g.tb);
        const long long ksize[4] = {a.Tk, a.Hkv, a.N, planes};
        const long long kstride[4] = {d, d * a.Tk, d * a.Tk * a.Hkv, d * keys};
        ok = ok && at::encode_map(&m.k, true, k, a.D, ksize, kstride, kt, 1) &&
             at::encode_map(&m.v, true, v, a.D, ksize, kstride, kt, 1);
    } else {
        const long long size[4] = {a.G, a.Tq, a.Hkv, a.N};
        const long long stride[4] = {a.qs.h * 2, a.qs.t * 2, a.qs.h * a.G * 2, a.qs.n * 2};
        ok = at::encode_map(&m.q, true, a.q, a.D, size, stride, g.gb, g.tb);
        // a shared axis (stride 0) of the keys or values is one coordinate of the map
        for (int i = 0; i < 2; ++i) {
            const HeadStrides &s = i ? a.vs : a.ks;
            const long long ksize[4] = {a.Tk, s.h ? a.Hkv : 1, s.n ? a.N : 1, 1};
            const long long kstride[4] = {s.t * 2, s.h * 2, s.n * 2, 16};
            ok = ok && at::encode_map(i ? &m.v : &m.k, true, i ? v : k, a.D, ksize, kstride, kt, 1);
        }
    }
    if (part.parts > 0) {
        const long long size[4] = {a.G, a.Tq, (long long)a.N * a.Hkv, g.splits}, d = a.D * 4LL;
        const long long stride[4] = {d, d * a.G, d * a.G * a.Tq, d * rows};
        ok = ok && at::encode_map(&m.out, false, part.o, a.D, size, stride, g.gb, g.tb);
    } else {
        const int es = bf16 ? 2 : 4;
        const long long size[4] = {a.G, a.Tq, a.Hkv, a.N};
        const long long stride[4] = {a.os.h * es, a.os.t * es, a.os.h * a.G * es, a.os.n * es};
        ok = ok && at::encode_map(&m.out, bf16, a.out, a.D, size, stride, g.gb, g.tb);
    }
    cudaError_t e = ok ? cudaSuccess : cudaErrorInvalidValue;
    if (e == cudaSuccess && g.packed) e = launch_attn_split(a, bf16, plane, st);
    if (e == cudaSuccess) {
        if (bf16 && a.D <= 64)
            e = pair ? at::launch<64, 1, true>(a, g, m, part, st, test) : at::launch<64, 1, false>(a, g, m, part, st, test);
        else if (bf16)
            e = pair ? at::launch<128, 1, true>(a, g, m, part, st, test) : at::launch<128, 1, false>(a, g, m, part, st, test);
        else if (a.D <= 64)
            e = pair ? at::launch<64, 3, true>(a, g, m, part, st, test) : at::launch<64, 3, false>(a, g, m, part, st, test);
        else
            e = at::launch<128, 3, false>(a, g, m, part, st, test);
    }
    if (e == cudaSuccess && part.parts > 0) e = launch_attn_join(a, bf16, part, st);
    if (ws) {
        const cudaError_t ef = workspace_free(ws, st);
        if (e == cudaSuccess) e = ef;
    }
    return e;
}

}  // namespace sc
