// States as 8-bit codes with one scale for each block of states and head:
//
//   a = max |x| over the block's valid states,  scale = a / top,  code = nearest(top x / a)
//
// Bound by memory: 2 or 4 bytes read and one written an element.  A block is
// read once into registers, four 8-element chunks a thread, its largest value
// found as the largest of the magnitudes' bits (so that an infinity or NaN is
// above every number), and the codes written from the registers.
// The quotient is x times top / a in fp32, off by less than 2^-22 of itself; where
// that leaves the code open (a value next to a border between two codes, every
// 2^13th or so), it is taken in 64 bits, which decides every case: two operands of
// 24 bits and a border of 8 cannot be closer than 2^-33 to it without lying on it.
#include <cuda_bf16.h>

#include "common.cuh"
#include "launch.h"
#include "layer.h"

namespace sc {

namespace {

constexpr int kQuantThreads = 256;
constexpr int kChunks = 4;   // of 8 elements, a thread's

__device__ __forceinline__ uint4 ld16(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ void load8(const float *p, float (&v)[8])
{
    const uint4 a = ld16(p), b = ld16(p + 4);
    v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
    v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y), v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8])
{
    const uint4 a = ld16(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// Two floats -> two e4m3 codes (nearest, ties to even), `lo` in the low byte.
__device__ __forceinline__ uint32_t to_e4m3(float lo, float hi)
{
    uint16_t y;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(y) : "f"(hi), "f"(lo));
    return y;
}

// top x / a, rounded to 24 bits so that a second rounding to fewer bits is the
// rounding of the quotient itself: to zero, the last bit set where it is inexact.
__device__ __noinline__ float exact_quotient(float x, float a, float top)
{
    const double q = (double)x * (double)top / (double)a;
    float f = __double2float_rz(q);
    if ((double)f != q) f = __uint_as_float(__float_as_uint(f) | 1u);
    return f;
}

template <bool E4M3>
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float a, float inv, bool tiny)
{
    constexpr float top = E4M3 ? 448.f : 127.f;
    float t[8];
    uint32_t w[2] = {0u, 0u};
    bool open = tiny;
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = x[j] * inv;
    if constexpr (E4M3) {
        uint32_t other = 0;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            constexpr float lo = 1.f - 0x1p-21f, hi = 1.f + 0x1p-21f;
            const uint32_t c = to_e4m3(t[j] * lo, t[j + 1] * lo);
            other |= c ^ to_e4m3(t[j] * hi, t[j + 1] * hi);
            w[j / 4] |= c << (8 * (j & 2));
        }
        open |= other != 0;
    } else {
        float near = 1.f;   // distance to the nearest border
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float r = rintf(t[j]);
            near = fminf(near, fabsf(fabsf(t[j] - r) - 0.5f));
            w[j / 4] |= ((uint32_t)(int)r & 0xffu) << (8 * (j & 3));
        }
        open |= near < 0x1p-14f;
    }
    if (open) {
        w[0] = w[1] = 0u;
#pragma unroll 1
        for (int j = 0; j < 8; ++j) {
            float xj = x[0];   // (indexed by a constant, so that x stays in registers)
#pragma unroll
            for (int i = 1; i < 8; ++i) xj = j == i ? x[i] : xj;
            const float q = exact_quotient(xj, a, top);
            const uint32_t c = E4M3 ? to_e4m3(q, 0.f) & 0xffu : (uint32_t)(int)rintf(q) & 0xffu;
            if (j < 4)
                w[0] |= c << (8 * j);
            else
                w[1] |= c << (8 * j - 32);
        }
    }
    return make_uint2(w[0], w[1]);
}

// A unit: one block of one (sequence, head), `threads` of the CTA's.
struct QuantGeom {
    int threads;        // of a unit: 32 to 512
    int per_cta;        // units
    long long units;    // of a tensor
};

template <class T, bool E4M3>
__global__ void __launch_bounds__(512) kv_quantize_kernel(const QuantArgs a, const QuantGeom g)
{
    __shared__ uint32_t largest[16];   // of each warp
    const QuantPart &p = a.part[blockIdx.y];
    const int tid = threadIdx.x % g.threads, slot = threadIdx.x / g.threads;
    const long long unit = (long long)blockIdx.x * g.per_cta + slot;
    const bool on = unit < g.units;
    const int h = on ? (int)(unit % a.H) : 0;
    const long long nb = on ? unit / a.H : 0;
    const int n = (int)(nb / a.blocks), b = (int)(nb - (long long)n * a.blocks);
    int len = a.T;
    if (a.k_len) len = max(0, min(len, a.k_len[n]));
    const int row_chunks = a.D / 8, t0 = b * a.block;
    const int rows = on ? max(0, min(a.block, len - t0)) : 0;
    const unsigned char *mb = a.key_mask ? a.key_mask + (long long)n * a.T + t0 : nullptr;
    float x[kChunks][8];
    int row[kChunks], col[kChunks];
    uint32_t top_bits = 0;
    bool any = false;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int c = tid + i * g.threads;
        row[i] = c / row_chunks;
        col[i] = (c - row[i] * row_chunks) * 8;
        if (row[i] >= rows || (mb && mb[row[i]] == 0)) {
            row[i] = -1;
            continue;
        }
        any = true;
        load8(static_cast<const T *>(p.x) + n * p.xs.n + (long long)(t0 + row[i]) * p.xs.t + h * p.xs.h + col[i], x[i]);
    }
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
        if (row[i] >= 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) top_bits = max(top_bits, __float_as_uint(x[i][j]) & 0x7fffffffu);
        }
    // bit 31: a state is valid
    top_bits |= any ? 0x80000000u : 0u;
    uint32_t m = __reduce_max_sync(0xffffffffu, top_bits);
    if (g.threads > 32) {
        if ((threadIdx.x & 31) == 0) largest[threadIdx.x >> 5] = m;
        __syncthreads();
        const int w0 = slot * (g.threads >> 5);
        m = 0;
        for (int w = 0; w < g.threads >> 5; ++w) m = max(m, largest[w0 + w]);
    }
    if (!(m >> 31)) return;
    m &= 0x7fffffffu;
    constexpr float top = E4M3 ? 448.f : 127.f;
    const bool finite = m < 0x7f800000u;
    const float amax = __uint_as_float(m);
    if (tid == 0)
        p.scale[((long long)n * a.H + h) * a.blocks + b] = finite ? __fdiv_rn(amax, top) : __uint_as_float(0x7fffffffu);
    const bool zero = m == 0 || !finite;
    const float inv = zero ? 0.f : __fdiv_rn(top, amax);
    const bool tiny = !zero && amax < 0x1p-100f;   // top / a may not be finite
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        if (row[i] < 0) continue;
        const uint2 w = zero ? make_uint2(0u, 0u) : codes8<E4M3>(x[i], amax, inv, tiny);
        *reinterpret_cast<uint2 *>(p.codes + n * p.cs.n + (long long)(t0 + row[i]) * p.cs.t + h * p.cs.h + col[i]) = w;
    }
}

}  // namespace

cudaError_t launch_kv_quantize(const QuantArgs &a, bool bf16, bool e4m3, cudaStream_t st)
{
    QuantGeom g;
    const int chunks = a.block * a.D / 8;
    g.threads = 32;
    while (g.threads * kChunks < chunks) g.threads *= 2;   // at most 512: 128 states of 128
    g.per_cta = g.threads < kQuantThreads ? kQuantThreads / g.threads : 1;
    g.units = (long long)a.N * a.blocks * a.H;
    const long long ctas = (g.units + g.per_cta - 1) / g.per_cta;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)ctas, a.parts), block(g.threads * g.per_cta);
    if (bf16) {
        if (e4m3)
            kv_quantize_kernel<__nv_bfloat16, true><<<grid, block, 0, st>>>(a, g);
        else
            kv_quantize_kernel<__nv_bfloat16, false><<<grid, block, 0, st>>>(a, g);
    } else {
        if (e4m3)
            kv_quantize_kernel<float, true><<<grid, block, 0, st>>>(a, g);
        else
            kv_quantize_kernel<float, false><<<grid, block, 0, st>>>(a, g);
    }
    return cudaGetLastError();
}

}  // namespace sc
