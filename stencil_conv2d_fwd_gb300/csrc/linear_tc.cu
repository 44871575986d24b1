// y = act(x w^T + b) + residual on the tensor cores (tcgen05, accumulators in
// tensor memory), for more rows than linear_rows.cu takes.
//
// A CTA, or a pair of CTAs on two SMs (cta_group::2: each holds half of both
// operands, and the pair's product reads both), computes tiles of 128 rows a CTA
// and BN outputs, one after the other (a persistent grid).  Rows of x and w are
// copied by TMA in steps of 64 elements of Cin through a ring of swizzled
// stages; two accumulators in tensor memory let the epilogue of one tile run
// beside the products of the next.
// Warps 0-7 are the epilogue: a warp reads the quadrant of tensor memory that it
// may address and half of the columns, adds bias, activation and residual in
// fp32, rounds once and hands 32 rows of 128 bytes at a time to a TMA store
// (the residual comes the same way); y or a residual that TMA cannot address (odd
// pitches, rows that end inside a 16-byte unit) is written and read a row at a time
// by the warp.  Warp 8 issues the copies, warp 9 the products.
//
// fp32 tensors: x and w are three bf16 planes each (linear_split below), a
// product the six of planes i + j <= 2, the small ones first.  The tensor cores
// cut each sum short instead of rounding it, so an accumulator takes no more than
// KCHUNK stages of Cin (256 elements); the epilogue's threads add those up in registers.
//
// Measured: 8192 x 8192 x 8192 bf16 616 us (1.78 PFLOP/s; the measured library product
// 1.73 sustained, 1.94 in a burst), 65536 x 2048 x 8192 1180 to 1308 (tensor cores 86%
// active), with gelu 1429 to 1508 (73%: the activation's instructions and energy);
// 14401 x 1024 x 4096 fp32 410 to 469 us, 258 to 294 TFLOP/s of the formula, six times
// that in products.
//
// The tiles after the last full turn of the SMs may be split along Cin (`splits`):
// each part writes fp32 sums, which a second kernel adds in order and finishes.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <cstring>
#include <mutex>

#include "divisor.cuh"
#include "launch.h"
#include "layer.h"
#include "linear.cuh"
#include "tc_common.cuh"

namespace sc {

namespace lt {

constexpr int TILE = 128;                // rows of a CTA's tile
constexpr int KB = 64;                   // elements of Cin a stage: one 128-byte swizzled row
constexpr int KCHUNK = 4;                // stages of Cin that an accumulator takes (fp32 tensors)
constexpr int THREADS = 384;
constexpr int EPI_WARPS = 8;
constexpr int STG = 32 * 128;            // bytes of a warp's staging: 32 rows of 128
// registers of the epilogue warps and of the others, out of what the block is launched with
constexpr int REGS_LAUNCH = 168, REGS_EPI = 216, REGS_OTHER = 72;
constexpr int MAX_STAGES = 8;
constexpr int GROUP_M = 8;               // row tiles that share a pass over w

template <int CG, int BN>
constexpr int stage_bytes() { return TILE * 128 + BN / CG * 128; }

struct Shared {
    uint64_t full[MAX_STAGES], empty[MAX_STAGES], acc_full[2], acc_empty[2], residual[EPI_WARPS], drain;
    uint32_t tmem;
    int abort;         // a wait of this CTA has expired
    int other_abort;   // one of the pair's other CTA, which writes it before the last barrier of the two
};
template <int CG, int BN>
constexpr int stages()
{
    constexpr int n = (227 * 1024 - EPI_WARPS * STG - (int)sizeof(Shared)) / stage_bytes<CG, BN>();
    return n < MAX_STAGES ? n : MAX_STAGES;
}
template <int CG, int BN>
constexpr int smem_bytes() { return stages<CG, BN>() * stage_bytes<CG, BN>() + EPI_WARPS * STG + (int)sizeof(Shared); }

struct Geom {
    int tiles_m, tiles_n;
    int whole, splits;  // tiles before the first one that is split along Cin; parts of those from there on
    int steps;          // stages of Cin: ceil(Cin / 64)
    int items;          // whole + (tiles - whole) * splits
    Divisor per_group, tail_rows, parts;   // tiles of a group; row tiles of the last group; splits
    int box;            // columns of y that a TMA store takes: 64 (bf16) or 32; 0: rows by the warp
    bool residual_tma;
    float *part;        // splits > 1: [splits][split tile][row][BN]
};

// The place of tile t: row tiles in groups that go over w together.  (By
// multiplications: with divisions the products waited 3 us for each tile.)
__device__ __forceinline__ void tile_at(const Geom &g, int t, int &m, int &n)
{
    const int grp = (int)g.per_group.quotient(t), in = t - grp * (int)g.per_group.d;
    const bool tail = (grp + 1) * GROUP_M > g.tiles_m;
    n = tail ? (int)g.tail_rows.quotient(in) : in / GROUP_M;
    m = grp * GROUP_M + in - n * (tail ? (int)g.tail_rows.d : GROUP_M);
}

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

// The address of `p` in the cluster's first CTA.
__device__ __forceinline__ uint32_t in_leader(uint32_t p)
{
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;\n" : "=r"(there) : "r"(p));
    return there;
}

// A box at (x, y, z) to this CTA's shared memory; a pair's copies count on the
// leader's barrier (`bar` is its address there).
template <int CG>
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap *m, int x, int y, int z, uint32_t bar)
{
    if constexpr (CG == 2)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(
                dst),
            "l"(reinterpret_cast<unsigned long long>(m)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(
                dst),
            "l"(reinterpret_cast<unsigned long long>(m)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
}
__device__ __forceinline__ void store_3d(const CUtensorMap *m, uint32_t src, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];\n" ::"l"(
                     reinterpret_cast<unsigned long long>(m)),
                 "r"(x), "r"(y), "r"(z), "r"(src)
                 : "memory");
}

template <int CG>
__device__ __forceinline__ void mma(uint32_t one, uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t acc)
{
    if constexpr (CG == 2)
        asm volatile(
            "{\n"
            ".reg .pred p, q;\n"
            ".reg .b64 da, db;\n"
            "setp.ne.b32 p, %5, 0;\n"
            "setp.ne.b32 q, %6, 0;\n"
            "mov.b64 da, {%1, %3};\n"
            "mov.b64 db, {%2, %3};\n"
            "@q tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %4, p;\n"
            "}\n" ::"r"(d),
            "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(acc), "r"(one)
            : "memory");
    else
        asm volatile(
            "{\n"
            ".reg .pred p, q;\n"
            ".reg .b64 da, db;\n"
            "setp.ne.b32 p, %5, 0;\n"
            "setp.ne.b32 q, %6, 0;\n"
            "mov.b64 da, {%1, %3};\n"
            "mov.b64 db, {%2, %3};\n"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n"
            "}\n" ::"r"(d),
            "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(acc), "r"(one)
            : "memory");
}
// Arrives on the barrier, in both CTAs of a pair, once the products so far are complete.
template <int CG>
__device__ __forceinline__ void commit(uint32_t one, uint32_t bar)
{
    if constexpr (CG == 2)
        asm volatile(
            "{\n"
            ".reg .pred q;\n"
            ".reg .b16 both;\n"
            "setp.ne.b32 q, %1, 0;\n"
            "mov.b16 both, 3;\n"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], both;\n"
            "}\n" ::"r"(bar),
            "r"(one)
            : "memory");
    else
        asm volatile(
            "{\n"
            ".reg .pred q;\n"
            "setp.ne.b32 q, %1, 0;\n"
            "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n"
            "}\n" ::"r"(bar),
            "r"(one)
            : "memory");
}
__device__ __forceinline__ void arrive_leader(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(in_leader(bar)) : "memory");
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
template <int CG>
__device__ __forceinline__ void alloc(uint32_t dst, uint32_t cols)
{
    if constexpr (CG == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(dst), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
    } else {
        tc::tmem_alloc(dst, cols);
    }
}
template <int CG>
__device__ __forceinline__ void dealloc(uint32_t at, uint32_t cols)
{
    if constexpr (CG == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(at), "r"(cols) : "memory");
    else
        tc::tmem_dealloc(at, cols);
}

// 128-byte swizzle, K-major, 8-row groups 1024 bytes apart.
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t DESC_LO = 1u << 16;

template <int CG, int BN>
constexpr uint32_t idesc()   // D fp32, A and B bf16, both K-major
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(TILE * CG >> 4) << 24);
}

// F32: planes of fp32 tensors; else bf16 tensors.
template <int CG, int BN, bool F32>
__global__ void __launch_bounds__(THREADS, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
                     const __grid_constant__ CUtensorMap my, const __grid_constant__ CUtensorMap mr,
                     const __grid_constant__ CUtensorMap mp, const LinearArgs a, const Geom g, int *status, const LinearTest test)
{
    constexpr int STAGES = stages<CG, BN>(), STAGE = stage_bytes<CG, BN>();
    constexpr int COLS = BN >= 128 ? BN / 2 : BN;      // columns of an epilogue warp
    constexpr uint32_t TMEM_COLS = 2 * BN < 32 ? 32 : 2 * BN;
    extern __shared__ __align__(1024) unsigned char dyn[];
    Shared &sh = *reinterpret_cast<Shared *>(dyn + STAGES * STAGE + EPI_WARPS * STG);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t base = smem_u32(dyn);
    if (base & 1023u) {   // the same in every CTA
        if (tid == 0) atomicExch(status, kDeviceTimeout);
        return;
    }
    const int rank = CG == 2 ? (int)(blockIdx.x & 1) : 0;
    const int first = blockIdx.x / CG, stride = gridDim.x / CG;

    // Whether the barrier's phase is complete: not if it took too long, or if another
    // wait of this CTA did (the lanes of a warp may see that flag at different times).
    volatile int *abort_flag = &sh.abort;
    auto wait = [&](uint64_t &bar, uint32_t parity) {
        const uint32_t b = smem_u32(&bar);
        if (mbar_try_wait(b, parity)) return true;
        const unsigned long long t0 = global_ns();
        while (!mbar_try_wait(b, parity)) {
            if (*abort_flag) return false;
            if (global_ns() - t0 > test.timeout_ns) {
                *abort_flag = 1;
                return false;
            }
        }
        return true;
    };
    // Work item: a tile, or a part of Cin of one of the last tiles.
    struct Item {
        int m, n, k0, k1, split, part;   // part: the split tile's number, -1: a whole one
    };
    auto item = [&](int i) {
        Item r;
        r.part = -1;
        r.split = 0;
        int t = i;
        if (i >= g.whole && g.splits > 1) {
            r.part = (int)g.parts.quotient(i - g.whole);
            r.split = i - g.whole - r.part * g.splits;
            t = g.whole + r.part;
        }
        tile_at(g, t, r.m, r.n);
        r.k0 = r.part < 0 ? 0 : (int)g.parts.quotient(g.steps * r.split);
        r.k1 = r.part < 0 ? g.steps : (int)g.parts.quotient(g.steps * (r.split + 1));
        return r;
    };
    constexpr int PRODUCTS = F32 ? 6 : 1;
    // The planes of a product, the small ones first: (x, w) = (2,0) (1,1) (0,2) (1,0) (0,1) (0,0)
    auto plane_x = [](int p) { return F32 ? (p == 0 ? 2 : (p == 1 || p == 3 ? 1 : 0)) : 0; };
    auto plane_w = [](int p) { return F32 ? (p == 2 ? 2 : (p == 1 || p == 4 ? 1 : 0)) : 0; };

    if (warp == 8) {
        if (lane == 0) {
            for (int i = 0; i < STAGES; ++i) {
                mbar_init(smem_u32(&sh.full[i]), 1);
                mbar_init(smem_u32(&sh.empty[i]), 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(smem_u32(&sh.acc_full[i]), 1);
                mbar_init(smem_u32(&sh.acc_empty[i]), CG * EPI_WARPS);
            }
            for (int i = 0; i < EPI_WARPS; ++i) mbar_init(smem_u32(&sh.residual[i]), 1);
            mbar_init(smem_u32(&sh.drain), 1);
            sh.abort = sh.other_abort = 0;
            fence_mbar_init();
        }
        __syncwarp();
    } else if (warp == 9) {
        alloc<CG>(smem_u32(&sh.tmem), TMEM_COLS);
    }
    pdl_wait();   // what comes before touches no global memory
    tc::fence_before_sync();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();
    tc::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem, 0);
    uint32_t issued = 0;   // stages asked for
    uint32_t loads = 0;    // of the residual, by this warp

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(REGS_OTHER));
        if (warp == 8) {
            if (lane == 0) {
                for (int i = first; i < g.items && !*abort_flag; i += stride) {
                    const Item it = item(i);
                    const int row = (it.m * CG + rank) * TILE, col = it.n * BN + rank * (BN / CG);
                    for (int c0 = it.k0; c0 < it.k1; c0 += F32 ? KCHUNK : it.k1) {
                        const int c1 = F32 ? min(c0 + KCHUNK, it.k1) : it.k1;
                        for (int p = 0; p < PRODUCTS; ++p)
                            for (int k = c0; k < c1; ++k, ++issued) {
                                const uint32_t slot = issued % STAGES, round = issued / STAGES;
                                const uint32_t bar = CG == 2 ? in_leader(smem_u32(&sh.full[slot])) : smem_u32(&sh.full[slot]);
                                if (round > 0) (void)wait(sh.empty[slot], (round - 1) & 1);
                                if (*abort_flag) break;
                                if (rank == 0) mbar_arrive_expect_tx(smem_u32(&sh.full[slot]), CG * STAGE);
                                const uint32_t at = base + slot * STAGE;
                                if ((int)issued == test.drop_copy) continue;
                                load_3d<CG>(at, &mx, k * KB, row, plane_x(p), bar);
                                load_3d<CG>(at + TILE * 128, &mw, k * KB, col, plane_w(p), bar);
                            }
                    }
                }
            }
            __syncwarp();
        } else if (warp == 9 && rank == 0) {
            const uint32_t one = elect_one();
            uint32_t c = 0, use = 0;   // stages and accumulators used
            // An expired wait ends the products, for the whole warp: each one more would
            // give stages back that the pair's second CTA would fill, with no one to expect
            // the bytes.
            bool on = true;
            for (int i = first; i < g.items && on; i += stride) {
                const Item it = item(i);
                for (int c0 = it.k0; c0 < it.k1 && on; c0 += F32 ? KCHUNK : it.k1, ++use) {
                    const int n = (F32 ? min(c0 + KCHUNK, it.k1) - c0 : it.k1 - c0) * PRODUCTS;
                    const uint32_t buf = use & 1;
                    if (use > 1) on = __all_sync(0xffffffffu, wait(sh.acc_empty[buf], ((use >> 1) - 1) & 1));
                    tc::fence_after_sync();
                    for (int k = 0; k < n && on; ++k, ++c) {
                        const uint32_t slot = c % STAGES;
                        on = __all_sync(0xffffffffu, wait(sh.full[slot], (c / STAGES) & 1));
                        if (!on) break;
                        tc::fence_after_sync();
                        const uint32_t xa = ((base + slot * STAGE) >> 4) | DESC_LO;
                        const uint32_t wa = ((base + slot * STAGE + TILE * 128) >> 4) | DESC_LO;
#pragma unroll
                        for (int j = 0; j < KB / 16; ++j)
                            mma<CG>(one, tmem + buf * BN, xa + 2 * j, wa + 2 * j, DESC_HI, idesc<CG, BN>(), k > 0 || j > 0);
                        commit<CG>(one, smem_u32(&sh.empty[slot]));
                    }
                    if (on) commit<CG>(one, smem_u32(&sh.acc_full[buf]));
                }
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(REGS_EPI));
        const int quad = warp & 3, part = warp >> 2;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t stg = base + STAGES * STAGE + warp * STG, stg_row = stg + lane * 128;
        const int col_part = COLS == BN ? 0 : part * COLS;
        const bool active = COLS < BN || part == 0;   // tiles of 64 columns: the first four warps
        uint32_t use = 0;
        for (int i = first; i < g.items; i += stride) {
            const Item it = item(i);
            const int row0 = (it.m * CG + rank) * TILE + quad * 32, row = row0 + lane;
            const int col0 = it.n * BN + col_part;
            // the columns' biases, a lane's each
            float bias[COLS / 32];
#pragma unroll
            for (int j = 0; j < COLS / 32; ++j) {
                const int col = col0 + j * 32 + lane;
                bias[j] = a.b && col < a.Cout ? a.b[col] : 0.f;
            }
            float acc[F32 ? COLS : 1];
            auto columns = [&](int at, float (&v)[32]) {   // this row's 32 columns from col0 + at
                if constexpr (F32) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = acc[F32 ? at + j : 0];
                } else {
                    uint32_t o[32];
                    tc::tmem_ld<32>(tmem + (use & 1) * BN + col_part + at + lanes, o);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(o[j]);
                }
            };
            auto release = [&]() {
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 2)
                        arrive_leader(smem_u32(&sh.acc_empty[use & 1]));
                    else
                        mbar_arrive(smem_u32(&sh.acc_empty[use & 1]));
                }
                ++use;
            };
            if constexpr (F32) {
                for (int c0 = it.k0; c0 < it.k1; c0 += KCHUNK) {
                    (void)wait(sh.acc_full[use & 1], (use >> 1) & 1);
                    __syncwarp();
                    tc::fence_after_sync();
                    if (active) {
#pragma unroll
                        for (int d = 0; d < COLS; d += 32) {
                            uint32_t o[32];
                            tc::tmem_ld<32>(tmem + (use & 1) * BN + col_part + d + lanes, o);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j) acc[F32 ? d + j : 0] = (c0 == it.k0 ? 0.f : acc[F32 ? d + j : 0]) + __uint_as_float(o[j]);
                        }
                    }
                    release();
                }
            } else {
                (void)wait(sh.acc_full[use & 1], (use >> 1) & 1);
                __syncwarp();
                tc::fence_after_sync();
            }
            // bias, activation (32 columns from col0 + d)
            auto finish = [&](float (&v)[32], int d) {
                if (a.b) {
                    const float mine = bias[d / 32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] += __shfl_sync(0xffffffffu, mine, j);
                }
                activate32<!F32>(v, a.act);
            };
            auto finish_at = [&](float (&v)[32], int d) {   // (d not a constant)
                float mine = bias[0];
#pragma unroll
                for (int j = 1; j < COLS / 32; ++j) mine = d == 32 * j ? bias[j] : mine;
                if (a.b) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] += __shfl_sync(0xffffffffu, mine, j);
                }
                activate32<!F32>(v, a.act);
            };
            bool held = !F32;   // the accumulator is not yet released
            // (one answer for the warp: what follows is for all of its lanes)
            if (active && row0 < a.rows && !__any_sync(0xffffffffu, *abort_flag)) {
                if (it.part >= 0) {
                    // fp32 sums of this part of Cin
#pragma unroll
                    for (int d = 0; d < COLS; d += 32) {
                        float v[32];
                        columns(d, v);
                        if (lane == 0) bulk_wait_read<0>();
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            tc::st_shared_v4(stg_row + ((j ^ (lane & 7)) << 4), __float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                                             __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3]));
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            store_3d(&mp, stg, col_part + d, (it.part * CG + rank) * TILE + quad * 32, it.split);
                            bulk_commit();
                        }
                    }
                } else if (g.box) {
                    // 128 bytes of 32 rows at a time; the last store's reading of the
                    // staging, or the residual's way there, is beside the arithmetic
                    constexpr int BOX = F32 ? 32 : 64;
#pragma unroll
                    for (int d = 0; d < COLS; d += BOX) {
                        if (col0 + d >= a.Cout) break;
                        if (lane == 0 && g.residual_tma) {
                            bulk_wait_read<0>();
                            mbar_arrive_expect_tx(smem_u32(&sh.residual[warp]), STG);
                            load_3d<1>(stg, &mr, col0 + d, row0, 0, smem_u32(&sh.residual[warp]));
                        }
                        float v[BOX / 32][32];
                        if constexpr (F32) {
                            columns(d, v[0]);
                        } else {
                            uint32_t o[2][32];
#pragma unroll
                            for (int e = 0; e < 2; ++e) tc::tmem_ld<32>(tmem + (use & 1) * BN + col_part + d + 32 * e + lanes, o[e]);
                            tc::tmem_wait_ld();
                            if (d + BOX >= COLS) {   // the last of the accumulator
                                release();
                                held = false;
                            }
#pragma unroll
                            for (int e = 0; e < 2; ++e)
#pragma unroll
                                for (int j = 0; j < 32; ++j) v[BOX / 32 - 1 ? e : 0][j] = __uint_as_float(o[e][j]);
                        }
#pragma unroll
                        for (int e = 0; e < BOX / 32; ++e) finish(v[e], d + 32 * e);
                        if (lane == 0 && !g.residual_tma) bulk_wait_read<0>();
                        __syncwarp();
                        // (no further copy behind one that has not come)
                        if (g.residual_tma && !__all_sync(0xffffffffu, wait(sh.residual[warp], loads++ & 1))) break;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {   // 16-byte chunks of the row
                            const uint32_t at = stg_row + ((j ^ (lane & 7)) << 4);
                            if constexpr (F32) {
                                float *y = v[0] + 4 * j;
                                if (g.residual_tma) {
                                    const uint4 r = ld_shared_v4(at);
                                    y[0] += __uint_as_float(r.x);
                                    y[1] += __uint_as_float(r.y);
                                    y[2] += __uint_as_float(r.z);
                                    y[3] += __uint_as_float(r.w);
                                }
                                tc::st_shared_v4(at, __float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3]));
                            } else {
                                float *y = v[BOX / 32 - 1 ? j / 4 : 0] + j % 4 * 8;
                                if (g.residual_tma) {
                                    const uint4 r = ld_shared_v4(at);
                                    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                                    for (int k = 0; k < 4; ++k) {
                                        y[2 * k] += __uint_as_float(w[k] << 16);
                                        y[2 * k + 1] += __uint_as_float(w[k] & 0xffff0000u);
                                    }
                                }
                                tc::st_shared_v4(at, tc::pack_bf16(y[0], y[1]), tc::pack_bf16(y[2], y[3]), tc::pack_bf16(y[4], y[5]),
                                                 tc::pack_bf16(y[6], y[7]));
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            store_3d(&my, stg, col0 + d, row0, 0);
                            bulk_commit();
                        }
                    }
                } else {
                    // rows by the warp: fp32 through the staging, lane = column
                    using T = typename std::conditional<F32, float, __nv_bfloat16>::type;
#pragma unroll 1
                    for (int d = 0; d < COLS; d += 32) {
                        if (col0 + d >= a.Cout) break;
                        float v[32];
                        if constexpr (F32) {
#pragma unroll
                            for (int e = 0; e < COLS; e += 32)
                                if (e == d) columns(e, v);
                        } else {
                            columns(d, v);
                        }
                        finish_at(v, d);
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            tc::st_shared_v4(stg_row + ((j ^ (lane & 7)) << 4), __float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                                             __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3]));
                        __syncwarp();
                        const int col = col0 + d + lane, live = min(32, a.rows - row0);
                        if (col < a.Cout) {
                            const T *rp = static_cast<const T *>(a.residual) + (a.residual ? row0 * a.rs + col : 0);
                            T *yp = static_cast<T *>(a.y) + row0 * a.ys + col;
#pragma unroll 8
                            for (int r = 0; r < live; ++r) {
                                float s = ld_shared_f32(stg + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
                                if (a.residual) s += to_float(rp[r * a.rs]);
                                store_as(yp + r * a.ys, s);
                            }
                        }
                    }
                }
            }
            if (held) release();
        }
        if (lane == 0) bulk_wait_read<0>();
        tc::fence_before_sync();
    }
    // One answer for the CTA: its threads part ways below, and meet at barriers.
    const bool expired = __syncthreads_or(*abort_flag);
    if (expired) {
        // give the copies and products in flight their time to end before the shared
        // and tensor memory are given back: a thousand times what they take, however short
        // the limit of the waits is
        const unsigned long long limit = test.timeout_ns > 1000000ull ? test.timeout_ns : 1000000ull;
        if (tid == 0) atomicExch(status, kDeviceTimeout);
        if (warp == 8 && lane == 0 && rank == 0)
            for (uint32_t e = issued > (uint32_t)STAGES ? issued - STAGES : 0; e < issued; ++e)
                (void)mbar_wait_bounded(smem_u32(&sh.full[e % STAGES]), (e / STAGES) & 1, limit);
        if (warp < EPI_WARPS && loads > 0) (void)mbar_wait_bounded(smem_u32(&sh.residual[warp]), (loads - 1) & 1, limit);
        if (warp == 9 && rank == 0) {
            commit<CG>(elect_one(), smem_u32(&sh.drain));
            (void)mbar_wait_bounded(smem_u32(&sh.drain), 0, limit);
            __syncwarp();
        }
        __syncthreads();
    }
    if constexpr (CG == 2) {
        // neither leaves while the other's copies and products use its memory; after
        // an expired wait the second CTA's last copies may have no one who waits for
        // them, so both stay for a thousand times as long as a copy takes.  Each tells the
        // other in a word of its own, which is read behind the barrier that orders it.
        if (tid == 0 && expired) {
            uint32_t there;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(there) : "r"(smem_u32(&sh.other_abort)), "r"(rank ^ 1));
            asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(there), "r"(1) : "memory");
        }
        __syncwarp();
        cluster_sync();
        if (expired || *static_cast<volatile int *>(&sh.other_abort)) {
            for (const unsigned long long t0 = global_ns(); global_ns() - t0 < 1000000ull;) __nanosleep(1000);
            __syncwarp();
            cluster_sync();
        }
    }
    if (warp == 9) dealloc<CG>(tmem, TMEM_COLS);
}

// Adds the parts of Cin of the split tiles in order and finishes: y = act(sum + b) +
// residual.  Tiles of rows x BN elements; a thread has four columns of a row.
template <class T>
__global__ void __launch_bounds__(256) linear_join_kernel(const LinearArgs a, const Geom g, int rows, int bn)
{
    pdl_wait();
    const int e = blockIdx.x * 256 + threadIdx.x, quads = bn / 4;   // of the tile blockIdx.y
    const int row = e / quads, c = (e - row * quads) * 4;
    int m, n;
    tile_at(g, g.whole + blockIdx.y, m, n);
    const long long r = (long long)m * rows + row;
    const int col = n * bn + c;
    if (row >= rows || r >= a.rows || col >= a.Cout) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    const float *p = g.part + ((long long)blockIdx.y * rows + row) * bn + c;
#pragma unroll 4
    for (int i = 0; i < g.splits; ++i, p += (long long)gridDim.y * rows * bn) {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (col + j >= a.Cout) break;
        float x = activate<sizeof(T) == 2>(v[j] + (a.b ? a.b[col + j] : 0.f), a.act);
        if (a.residual) x += to_float(static_cast<const T *>(a.residual)[r * a.rs + col + j]);
        store_as(static_cast<T *>(a.y) + r * a.ys + col + j, x);
    }
}

// fp32 rows as three bf16 planes, x = x0 + x1 + x2 to 24 bits (attn_split.cu has
// the formats' ends: x0 is finite, an infinity sits in the last plane).  Bound by
// memory: 4 bytes read and 6 written an element.
struct SplitPart {
    const float *x;
    __nv_bfloat16 *y;   // planes rows * cols apart
    long long rows, stride;
};
__global__ void __launch_bounds__(256) linear_split_kernel(const SplitPart p0, const SplitPart p1, int cols8)
{
    pdl_trigger();   // the product's kernel may be set up; its copies wait for this grid's end
    pdl_wait();
    const SplitPart &p = blockIdx.y ? p1 : p0;
    const long long chunks = p.rows * cols8, plane = chunks * 8;
    for (long long e = (long long)blockIdx.x * 256 + threadIdx.x; e < chunks; e += (long long)gridDim.x * 256) {
        const long long row = e / cols8;
        const int c = (int)(e - row * cols8);
        const float4 *src = reinterpret_cast<const float4 *>(p.x + row * p.stride + c * 8);
        const float4 v0 = src[0], v1 = src[1];
        const float x[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = fabsf(x[i]) < INFINITY ? x[i] : 0.f;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (k == 2) {
                    f[2 * i] = fabsf(x[2 * i]) < INFINITY ? f[2 * i] : x[2 * i];
                    f[2 * i + 1] = fabsf(x[2 * i + 1]) < INFINITY ? f[2 * i + 1] : x[2 * i + 1];
                }
                w[i] = k == 0 ? pack_bf16_finite(f[2 * i], f[2 * i + 1]) : tc::pack_bf16(f[2 * i], f[2 * i + 1]);
                f[2 * i] -= __uint_as_float(w[i] << 16);
                f[2 * i + 1] -= __uint_as_float(w[i] & 0xffff0000u);
            }
            *reinterpret_cast<uint4 *>(p.y + k * plane + e * 8) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
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

// [planes][rows][cols], boxes of 128 bytes of box_rows rows.
bool encode_map(CUtensorMap *m, bool bf16, const void *base, long long cols, long long rows, long long planes, long long stride,
                long long plane, int box_rows)
{
    const int es = bf16 ? 2 : 4;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)planes};
    const cuuint64_t strides[2] = {(cuuint64_t)(stride * es), planes > 1 ? (cuuint64_t)(plane * es) : 16};
    const cuuint32_t box[3] = {128u / es, (cuuint32_t)box_rows, 1}, one[3] = {1, 1, 1};
    return encoder()(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void *>(base), dims,
                     strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Maps {
    CUtensorMap x, w, y, r, part;
};

template <int CG, int BN, bool F32>
cudaError_t launch(const LinearArgs &a, const Geom &g, const Maps &m, cudaStream_t st, const LinearTest &test)
{
    constexpr int SMEM = smem_bytes<CG, BN>();
    static_assert(SMEM <= 227 * 1024, "shared memory");
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    static KernelCache cache;
    e = ensure_dynamic_smem(cache, dev, linear_tc_kernel<CG, BN, F32>, SMEM);
    if (e != cudaSuccess) return e;
    // the register split is of REGS_LAUNCH a thread: with fewer, a warp would wait for registers that never come
    static const int regs = [] {
        cudaFuncAttributes fa = {};
        return cudaFuncGetAttributes(&fa, linear_tc_kernel<CG, BN, F32>) == cudaSuccess ? fa.numRegs : 0;
    }();
    if (regs != REGS_LAUNCH) return cudaErrorNotSupported;
    int *status = device_status_ptr();
    if (!status) return cudaErrorInvalidDevice;
    const int slots = device_sm_count() / CG;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(CG * (g.items < slots ? g.items : slots)));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    int n = 0;
    if (CG == 2) {
        at[n].id = cudaLaunchAttributeClusterDimension;
        at[n].val.clusterDim.x = CG;
        at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
        ++n;
    }
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
    cfg.attrs = at;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, linear_tc_kernel<CG, BN, F32>, m.x, m.w, m.y, m.r, m.part, a, g, status, test);
}

}  // namespace lt

cudaError_t launch_linear_tc(const LinearArgs &a, bool bf16, cudaStream_t st, const LinearTest &test)
{
    if (!lt::encoder()) return cudaErrorNotSupported;
    const int es = bf16 ? 2 : 4, products = bf16 ? 1 : 6;
    lt::Geom g = {};
    g.steps = (a.Cin + lt::KB - 1) / lt::KB;
    const int sms = device_sm_count();
    // Tile and parts.  Estimated clocks: a tile's stages (of which one in four more
    // waits for copies where a CTA is alone, or the pair's tile narrow), 1500 for a tile's
    // turn, 4000 for the start and the last epilogue.  The tiles after the last full turn
    // of the SMs, or all where there are few, are split along Cin into as many parts as
    // fill a turn, for a second launch (6000) that reads them.  2464 x 2048 x 2048 bf16
    // (80 tiles on 76 pairs): 28.2 us with whole tiles, 23.4 with the last four split.
    static const struct {
        int cg, bn;
        double step;    // clocks of a stage
    } shape[4] = {{2, 256, 540.}, {2, 128, 400.}, {1, 128, 520.}, {1, 64, 420.}};
    int best = 0, splits = 1;
    long long whole = 0;
    double least = 1e300;
    for (int i = 0; i < 4; ++i) {
        const long long tm = (a.rows + 128LL * shape[i].cg - 1) / (128 * shape[i].cg), tn = (a.Cout + (long long)shape[i].bn - 1) / shape[i].bn;
        const long long slots = sms / shape[i].cg, tiles = tm * tn, rest = tiles % slots;
        const double tile = (double)g.steps * products * shape[i].step;
        const double t1 = (double)((tiles + slots - 1) / slots) * (tile + 1500.);
        if (t1 + 4000. < least) {
            least = t1 + 4000.;
            best = i;
            splits = 1;
            whole = tiles;
        }
        for (int s = 2; s <= 16 && s <= (g.steps + 3) / 4 && rest * s <= slots; ++s) {
            const double join = 6000. + (double)rest * 128 * shape[i].cg * shape[i].bn * 4 * (s + 1) / 3000.;
            const double t = (double)(tiles / slots) * (tile + 1500.) + tile / s + 1500. + 4000. + join;
            if (rest > 0 && t < least) {
                least = t;
                best = i;
                splits = s;
                whole = tiles - rest;
            }
        }
    }
    const int cg = shape[best].cg, bn = shape[best].bn;
    const long long tm = (a.rows + 128LL * cg - 1) / (128 * cg), tn = (a.Cout + (long long)bn - 1) / bn;
    if (tm * tn > 0x3fffffffLL || tn > 0x3fffffffLL / lt::GROUP_M) return cudaErrorInvalidConfiguration;
    g.tiles_m = (int)tm;
    g.tiles_n = (int)tn;
    g.splits = splits;
    g.whole = (int)whole;
    const int split_tiles = (int)(tm * tn - whole);
    g.items = g.whole + split_tiles * splits;
    g.per_group = make_divisor((int)(tn * lt::GROUP_M));
    g.tail_rows = make_divisor(g.tiles_m % lt::GROUP_M ? g.tiles_m % lt::GROUP_M : lt::GROUP_M);
    g.parts = make_divisor(splits);

    auto pad = [](size_t b) { return (b + 255) & ~(size_t)255; };
    const int tile_rows = lt::TILE * cg;
    const size_t pp = pad((size_t)splits * split_tiles * tile_rows * bn * 4);
    const size_t px = bf16 ? 0 : pad((size_t)a.rows * a.Cin * 6), pw = bf16 ? 0 : pad((size_t)a.Cout * a.Cin * 6);
    char *ws = nullptr;
    if (pp + px + pw > 0) {
        const cudaError_t e = workspace_alloc(reinterpret_cast<void **>(&ws), pp + px + pw, st);
        if (e != cudaSuccess) return e;
    }
    g.part = split_tiles > 0 ? reinterpret_cast<float *>(ws) : nullptr;
    auto tma_rows = [&](const void *p, long long stride) {
        return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && stride * es % 16 == 0 && stride > 0;
    };
    // (a TMA store leaves out whole 16-byte units past the row's end, but not a part of one)
    const bool y_tma = tma_rows(a.y, a.ys) && (long long)a.Cout * es % 16 == 0 && (!a.residual || tma_rows(a.residual, a.rs));
    g.box = y_tma ? (bf16 ? 64 : 32) : 0;
    g.residual_tma = y_tma && a.residual;

    lt::Maps m;
    std::memset(&m, 0, sizeof(m));
    bool ok;
    if (bf16) {
        ok = lt::encode_map(&m.x, true, a.x, a.Cin, a.rows, 1, a.xs, 0, lt::TILE) &&
             lt::encode_map(&m.w, true, a.w, a.Cin, a.Cout, 1, a.ws, 0, bn / cg);
    } else {
        ok = lt::encode_map(&m.x, true, ws + pp, a.Cin, a.rows, 3, a.Cin, (long long)a.rows * a.Cin, lt::TILE) &&
             lt::encode_map(&m.w, true, ws + pp + px, a.Cin, a.Cout, 3, a.Cin, (long long)a.Cout * a.Cin, bn / cg);
    }
    if (g.part) {
        const long long rows = (long long)split_tiles * tile_rows;
        ok = ok && lt::encode_map(&m.part, false, g.part, bn, rows, splits, bn, rows * bn, 32);
    }
    if (g.box) ok = ok && lt::encode_map(&m.y, bf16, a.y, a.Cout, a.rows, 1, a.ys, 0, 32);
    if (g.residual_tma) ok = ok && lt::encode_map(&m.r, bf16, a.residual, a.Cout, a.rows, 1, a.rs, 0, 32);
    cudaError_t e = ok ? cudaSuccess : cudaErrorInvalidValue;
    if (e == cudaSuccess && !bf16) {
        const lt::SplitPart p0{static_cast<const float *>(a.x), reinterpret_cast<__nv_bfloat16 *>(ws + pp), a.rows, a.xs};
        const lt::SplitPart p1{static_cast<const float *>(a.w), reinterpret_cast<__nv_bfloat16 *>(ws + pp + px), a.Cout, a.ws};
        const long long most = (a.rows > a.Cout ? a.rows : a.Cout) * (a.Cin / 8LL);
        long long blocks = (most + 255) / 256;
        if (blocks > 16LL * sms) blocks = 16LL * sms;
        e = launch_behind(lt::linear_split_kernel, dim3((unsigned)blocks, 2), dim3(256), st, 1, p0, p1, a.Cin / 8);
    }
    if (e == cudaSuccess) {
        switch (best * 2 + (bf16 ? 0 : 1)) {
        case 0: e = lt::launch<2, 256, false>(a, g, m, st, test); break;
        case 1: e = lt::launch<2, 256, true>(a, g, m, st, test); break;
        case 2: e = lt::launch<2, 128, false>(a, g, m, st, test); break;
        case 3: e = lt::launch<2, 128, true>(a, g, m, st, test); break;
        case 4: e = lt::launch<1, 128, false>(a, g, m, st, test); break;
        case 5: e = lt::launch<1, 128, true>(a, g, m, st, test); break;
        case 6: e = lt::launch<1, 64, false>(a, g, m, st, test); break;
        default: e = lt::launch<1, 64, true>(a, g, m, st, test); break;
        }
    }
    if (e == cudaSuccess && g.part) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(tile_rows * (bn / 4) / 256), (unsigned)split_tiles);
        cfg.blockDim = dim3(256);
        cfg.stream = st;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        e = bf16 ? cudaLaunchKernelEx(&cfg, lt::linear_join_kernel<__nv_bfloat16>, a, g, tile_rows, bn)
                 : cudaLaunchKernelEx(&cfg, lt::linear_join_kernel<float>, a, g, tile_rows, bn);
    }
    if (ws) {
        const cudaError_t ef = workspace_free(ws, st);
        if (e == cudaSuccess) e = ef;
    }
    return e;
}

}  // namespace sc
