// States as 8-bit codes with one scale for each block of states and head:
//
//   a = max |x| over the block's valid states,  scale = a / top,  code = nearest(top x / a)
//
// Bound by memory: 2 or 4 bytes read and one written an element.  A block is
// read once into registers, 16 or 32 elements a thread, its largest value
// found as the largest of the magnitudes' bits (so that an infinity or NaN is
// above every number), and the codes written from the registers.
// The quotient is x times top / a in fp32, off by less than 2^-22 of itself; where
// that leaves the code open (a value next to a border between two codes, every
// 2^13th or so of fp32 values, and many bf16 ones, which lie on borders), top x is
// compared with border times a in exact arithmetic made of fp32 FMAs (in 64 bits,
// whose rate is 1/64 here, bf16 states took 794 us where they now take 90).
// 32 x 3136 states, 8 heads of 64, keys and values: fp32 88 to 89 us (5.8 TB/s, either
// code), bf16 92 (e4m3) and 96 (int8; 3.3 TB/s: some 27 instructions an element of both,
// issued 82% of the time).  Lengths from 1600 to 3136: fp32 75 us (5.0 TB/s), bf16 76 to 78.
#include <cuda_bf16.h>

#include "common.cuh"
#include "divisor.cuh"
#include "launch.h"
#include "layer.h"

namespace sc {

namespace {

constexpr int kQuantThreads = 256;
template <class T>
constexpr int E = 16 / (int)sizeof(T);           // elements of a 16-byte chunk

// (a warp's access is 512 bytes in a row whatever the type)
__device__ __forceinline__ void load_chunk(const float *p, float (&v)[4])
{
    const uint4 a = ld16_once(p);
    v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
}
__device__ __forceinline__ void load_chunk(const __nv_bfloat16 *p, float (&v)[8])
{
    const uint4 a = ld16_once(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// The values of two positive e4m3 codes, added.
__device__ __forceinline__ float e4m3_sum(uint32_t a, uint32_t b)
{
    float x, y;
    asm("{\n.reg .b16 c, l, h;\n.reg .b32 p;\nmov.b32 {c, l}, %2;\ncvt.rn.f16x2.e4m3x2 p, c;\nmov.b32 {l, h}, p;\n"
        "cvt.f32.f16 %0, l;\ncvt.f32.f16 %1, h;\n}\n"
        : "=f"(x), "=f"(y)
        : "r"(a | b << 8));
    return x + y;
}

// Two floats -> two e4m3 codes (nearest, ties to even), `lo` in the low byte.
__device__ __forceinline__ uint32_t to_e4m3(float lo, float hi)
{
    uint16_t y;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(y) : "f"(hi), "f"(lo));
    return y;
}

// The largest of m, |x| and |y|; NaN if one is.
__device__ __forceinline__ float max_nan(float m, float x, float y)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(x)), "f"(fabsf(y)));
    return r;
}

// The sign of n |x| - m a in exact arithmetic, for integers n and m of up to 10 bits
// and nearly equal products: a product's rounding error is one more FMA, the large
// parts' difference is exact, and so is that of the errors, which have fewer than
// ten bits between them.  a is in [1, 2).
__device__ __forceinline__ float exact_difference(float n, float x, float m, float a)
{
    const float p = n * x, q = m * a;
    return (p - q) + (fmaf(n, x, -p) - fmaf(m, a, -q));
}

// The N codes of x / scale, a byte each; inv = top / a.  The quotient's two
// ends are rounded; where they differ, the border between the two codes decides.
template <bool E4M3, int N>
__device__ __forceinline__ uint2 codes(const float (&x)[N], float a, float inv)
{
    constexpr float magic = 12582912.f;   // 1.5 * 2^23: the sum with it rounds to an integer, its low byte
    const float inv0 = inv * (1.f - 0x1p-21f), inv1 = inv * (1.f + 0x1p-21f);
    uint32_t w[2] = {0u, 0u}, v[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < N; j += 4) {
        if constexpr (E4M3) {
            w[j / 4] = __byte_perm(to_e4m3(x[j] * inv0, x[j + 1] * inv0), to_e4m3(x[j + 2] * inv0, x[j + 3] * inv0), 0x5410);
            v[j / 4] = __byte_perm(to_e4m3(x[j] * inv1, x[j + 1] * inv1), to_e4m3(x[j + 2] * inv1, x[j + 3] * inv1), 0x5410);
        } else {
            uint32_t m[4], k[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                m[i] = __float_as_uint(fmaf(x[j + i], inv0, magic));
                k[i] = __float_as_uint(fmaf(x[j + i], inv1, magic));
            }
            w[j / 4] = __byte_perm(__byte_perm(m[0], m[1], 0x0040), __byte_perm(m[2], m[3], 0x0040), 0x5410);
            v[j / 4] = __byte_perm(__byte_perm(k[0], k[1], 0x0040), __byte_perm(k[2], k[3], 0x0040), 0x5410);
        }
    }
    uint32_t open[2] = {w[0] ^ v[0], w[1] ^ v[1]};
    if (open[0] | open[1]) {
        const float unit = __uint_as_float((254u << 23) - (__float_as_uint(a) & 0x7f800000u)), an = a * unit;
        // one open code after the other: there is mostly one
        do {
            const int half = open[0] ? 0 : 1;
            const uint32_t shift = (uint32_t)(__ffs((int)(half ? open[1] : open[0])) - 1) & ~7u;
            const int j = half * 4 + (int)(shift >> 3);
            float xj = x[0];
#pragma unroll
            for (int i = 1; i < N; ++i) xj = i == j ? x[i] : xj;
            uint32_t &word = half ? w[1] : w[0];
            const uint32_t code = word >> shift & 0xffu, up = (half ? v[1] : v[0]) >> shift & 0xffu;
            // w's code is the one nearer to zero, c of the magnitude; the border to the
            // next one is half the sum of the two
            const int c = E4M3 ? (int)(code & 0x7fu) : abs((int)(signed char)code);
            const float sum = E4M3 ? e4m3_sum(c, c + 1) : 2.f * (float)c + 1.f;
            const float d = exact_difference(E4M3 ? 896.f : 254.f, fabsf(xj) * unit, sum, an);
            if (d > 0.f || (d == 0.f && (c & 1))) word = (word & ~(0xffu << shift)) | up << shift;
            open[0] &= half ? ~0u : ~(0xffu << shift);
            open[1] &= half ? ~(0xffu << shift) : ~0u;
        } while (open[0] | open[1]);
    }
    return make_uint2(w[0], w[1]);
}

// A unit: one block of one (sequence, head), `threads` of the CTA's.
struct QuantGeom {
    int threads;        // of a unit: 32 to 512
    int log2_threads;
    int per_cta;        // units
    uint32_t units;     // of a tensor
    Divisor heads, blocks, row_chunks;
    int row_step, col_step;   // rows and chunks from one of a thread's chunks to the next
};

// PER elements a thread.
template <class T, bool E4M3, int PER>
__global__ void __launch_bounds__(512) kv_quantize_kernel(const QuantArgs a, const QuantGeom g)
{
    __shared__ uint32_t largest[16];   // of each warp
    const QuantPart &p = a.part[blockIdx.y];
    const int tid = threadIdx.x & (g.threads - 1), slot = threadIdx.x >> g.log2_threads;
    const uint32_t unit = blockIdx.x * g.per_cta + slot;
    const bool on = unit < g.units;
    const uint32_t nb = on ? g.heads.quotient(unit) : 0u;
    const int h = on ? (int)(unit - nb * a.H) : 0;
    const int n = (int)g.blocks.quotient(nb), b = (int)nb - n * a.blocks;
    pdl_trigger();   // the next kernel may be set up; it waits for this grid's end
    pdl_wait();
    int len = a.T;
    if (a.k_len) len = max(0, min(len, a.k_len[n]));
    const int row_chunks = a.D / E<T>, t0 = b * a.block;
    const int rows = on ? max(0, min(a.block, len - t0)) : 0;
    const unsigned char *mb = a.key_mask ? a.key_mask + (long long)n * a.T + t0 : nullptr;
    // this thread's chunks: `col` and `row` step by g.threads chunks
    float x[PER / E<T>][E<T>];
    const int dr = g.row_step, dc = g.col_step;
    const int row0 = (int)g.row_chunks.quotient(tid), col0 = tid - row0 * row_chunks;
    const T *xp = static_cast<const T *>(p.x) + n * p.xs.n + (long long)(t0 + row0) * p.xs.t + h * p.xs.h + col0 * E<T>;
    unsigned char *cp = p.codes + n * p.cs.n + (long long)(t0 + row0) * p.cs.t + h * p.cs.h + col0 * E<T>;
    // from a chunk to the next; a turn goes to the next row's start
    const long long xs = dr * p.xs.t + dc * E<T>, xturn = p.xs.t - a.D, cs = dr * p.cs.t + dc * E<T>, cturn = p.cs.t - a.D;
    auto next = [&](int &row, int &col, auto *&at, long long step, long long turn) {
        row += dr;
        at += step;
        if (dc != 0) {   // (heads whose chunks do not divide the threads)
            col += dc;
            if (col >= row_chunks) {
                col -= row_chunks;
                ++row;
                at += turn;
            }
        }
    };
    float top = 0.f;   // a NaN stays
    uint32_t on_bits = 0;
    int row = row0, col = col0;
#pragma unroll
    for (int i = 0; i < PER / E<T>; ++i, next(row, col, xp, xs, xturn))
        if (row < rows && !(mb && mb[row] == 0)) {
            on_bits |= 1u << i;
            load_chunk(xp, x[i]);
        }
#pragma unroll
    for (int i = 0; i < PER / E<T>; ++i)
        if (on_bits >> i & 1u) {
#pragma unroll
            for (int j = 0; j < E<T>; j += 2) top = max_nan(top, x[i][j], x[i][j + 1]);
        }
    // bit 31: a state is valid
    uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(top) | (on_bits ? 0x80000000u : 0u));
    if (g.threads > 32) {
        if ((threadIdx.x & 31) == 0) largest[threadIdx.x >> 5] = m;
        __syncthreads();
        const int warps = g.threads >> 5, lane = threadIdx.x & 31;
        m = __reduce_max_sync(0xffffffffu, lane < warps ? largest[slot * warps + lane] : 0u);
    }
    if (!(m >> 31)) return;
    m &= 0x7fffffffu;
    constexpr float largest_code = E4M3 ? 448.f : 127.f;
    const bool finite = m < 0x7f800000u;
    float amax = __uint_as_float(m);
    if (tid == 0)
        p.scale[((long long)n * a.H + h) * a.blocks + b] = finite ? __fdiv_rn(amax, largest_code) : __uint_as_float(0x7fffffffu);
    const bool zero = m == 0 || !finite;
    // far from 1 in size, top / a or top x may not be finite: all times a power of two
    const float move = amax < 0x1p-100f ? 0x1p100f : (amax > 0x1p100f ? 0x1p-60f : 1.f);
    amax *= move;
    float inv;   // top / a, to 2^-22
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(amax));
    inv = zero ? 0.f : inv * largest_code;
    row = row0, col = col0;
#pragma unroll
    for (int i = 0; i < PER / E<T>; ++i, next(row, col, cp, cs, cturn)) {
        if (!(on_bits >> i & 1u)) continue;
        if (move != 1.f) {
#pragma unroll
            for (int j = 0; j < E<T>; ++j) x[i][j] *= move;
        }
        const uint2 w = zero ? make_uint2(0u, 0u) : codes<E4M3>(x[i], amax, inv);
        if constexpr (E<T> == 8)
            *reinterpret_cast<uint2 *>(cp) = w;
        else
            *reinterpret_cast<uint32_t *>(cp) = w.x;
    }
}

}  // namespace

cudaError_t launch_kv_quantize(const QuantArgs &a, bool bf16, bool e4m3, cudaStream_t st)
{
    QuantGeom g;
    g.threads = 32;
    // 32 elements a thread where 16 would be more than 256 threads to wait for one
    // another
    const int per = a.block * a.D > 4096 ? 32 : 16;
    while (g.threads * per < a.block * a.D) g.threads *= 2;   // at most 512: 128 states of 128
    g.per_cta = g.threads < kQuantThreads ? kQuantThreads / g.threads : 1;
    // (2^31 units are 512 GB of codes)
    const long long units = (long long)a.N * a.blocks * a.H;
    if (units > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    g.units = (uint32_t)units;
    g.log2_threads = 5;
    while (1 << g.log2_threads < g.threads) ++g.log2_threads;
    g.heads = make_divisor(a.H);
    g.blocks = make_divisor(a.blocks);
    const int row_chunks = a.D / (bf16 ? 8 : 4);
    g.row_chunks = make_divisor(row_chunks);
    g.row_step = g.threads / row_chunks;
    g.col_step = g.threads % row_chunks;
    const long long ctas = (units + g.per_cta - 1) / g.per_cta;
    const dim3 grid((unsigned)ctas, a.parts), block(g.threads * g.per_cta);
    auto go = [&](auto small, auto large) { return launch_behind(per == 16 ? small : large, grid, block, st, 1, a, g); };
    if (bf16 && e4m3) return go(kv_quantize_kernel<__nv_bfloat16, true, 16>, kv_quantize_kernel<__nv_bfloat16, true, 32>);
    if (bf16) return go(kv_quantize_kernel<__nv_bfloat16, false, 16>, kv_quantize_kernel<__nv_bfloat16, false, 32>);
    if (e4m3) return go(kv_quantize_kernel<float, true, 16>, kv_quantize_kernel<float, true, 32>);
    return go(kv_quantize_kernel<float, false, 16>, kv_quantize_kernel<float, false, 32>);
}

}  // namespace sc
