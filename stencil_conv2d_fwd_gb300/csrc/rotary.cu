// RMS norm of every head and the rotation of its positions, in one pass; the
// rotation alone; and the table of the rotation's cosines and sines.
//
//   y = x * (mean(x^2) + eps)^(-1/2) * weight          (norm)
//   (a, b) -> (a cos - b sin, b cos + a sin)           pair i of the first `rot` elements,
//   half: (i, i + rot / 2); interleaved: (2 i, 2 i + 1)
//
// Bound by memory: each element is read and written once.  A thread holds
// both members of its V pairs (two 16-byte chunks, rot / 2 elements apart in
// the half layout, adjacent in the interleaved one), so the rotation needs no
// exchange; elements beyond `rot` are handled as chunk pairs that are only
// copied.  A row's D / (2 V) threads sum their squares by shuffles.  A thread
// does kHeads heads of one token, with the token's cosines, sines and the
// norm's weights in registers and all its loads issued first, and keeps what
// it loaded as stored until each head's turn: with floats for all four heads
// (116 registers, 16 warps an SM) 131072 tokens of 8 x 128 bf16 took 149.6 us,
// now (32 warps an SM) 92.8 (6.5 TB/s); 65536 + 14400 tokens of 16 x 128 fp32
// with the norm 210 and 192 us (6.8 TB/s); 2464 + 100352 of 8 x 64 bf16 with the
// norm 67.6 and 41.1 us (5.1 TB/s; half-heads of 64 bytes).  Two heads a thread
// read the table twice as often: 100, 200 and 45 us.
#include <cuda_bf16.h>

#include <cmath>

#include "attn.h"
#include "launch.h"

namespace sc {

namespace {

constexpr int kRotThreads = 128;
constexpr int kHeads = 4;     // heads of a token per thread
// CTAs an SM: at most 64 registers a thread, 96 where eight weights and angles
// of each chunk are held (64 spill them: 91 us, not 41, for the keys of 32 maps
// of 56 x 56, 8 x 64 bf16, and their prompts' queries).  The rotation alone
// spills 20 to 32 bytes of its eight angles at 64, and runs at the memory's rate.
template <int V, bool NORM>
constexpr int rot_ctas() { return V == 8 && NORM ? 5 : 8; }

// V elements (16 bytes, or 8 for four bf16) as stored, and as floats.
template <class T, int V>
struct Packed {
    static constexpr int W = V * (int)sizeof(T) / 4;
    uint32_t w[W];
    __device__ __forceinline__ void load(const T *p)
    {
        if constexpr (W == 4) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p);
            w[0] = u.x;
            w[1] = u.y;
            w[2] = u.z;
            w[3] = u.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            w[0] = u.x;
            w[1] = u.y;
        }
    }
    __device__ __forceinline__ void store(T *p) const
    {
        if constexpr (W == 4)
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
    __device__ __forceinline__ void unpack(float *f) const
    {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if constexpr (sizeof(T) == 4) {
                f[i] = __uint_as_float(w[i]);
            } else {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
    __device__ __forceinline__ void pack(const float *f)
    {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if constexpr (sizeof(T) == 4) {
                w[i] = __float_as_uint(f[i]);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
    }
};

// V floats at p, 16-byte aligned, of a table that every CTA reads.
template <int V>
__device__ __forceinline__ void load_floats(const float *p, float *f)
{
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const float4 u = __ldg(reinterpret_cast<const float4 *>(p + i));
        f[i] = u.x;
        f[i + 1] = u.y;
        f[i + 2] = u.z;
        f[i + 3] = u.w;
    }
}

struct RotGeom {
    int lanes;           // threads per row: a power of two >= D / (2 V)
    int slots;           // D / (2 V)
    float inv_d;         // 1 / D
    long long blocks0;   // CTAs of part[0]; the others do part[1]
};

template <class T, int V, bool INTERLEAVED, bool NORM>
__global__ void __launch_bounds__(kRotThreads, rot_ctas<V, NORM>()) rotary_kernel(const RotaryArgs a, const RotGeom g, int *status)
{
    const bool second = blockIdx.x >= g.blocks0;
    const NormHeads &P = a.part[second ? 1 : 0];
    const long long blk = (long long)blockIdx.x - (second ? g.blocks0 : 0);
    const int hblocks = (P.heads + kHeads - 1) / kHeads;
    const int per_cta = kRotThreads / g.lanes;
    const long long unit = blk * per_cta + threadIdx.x / g.lanes;
    const long long units = (long long)P.tokens * hblocks;
    const int slot = threadIdx.x & (g.lanes - 1);
    const bool act = unit < units && slot < g.slots;   // the others take part in the shuffles only
    const int tok = act ? (units <= 0xffffffffLL ? (int)((uint32_t)unit / (uint32_t)hblocks) : (int)(unit / hblocks)) : 0;
    const int h0 = act ? (int)(unit - (long long)tok * hblocks) * kHeads : 0;
    const int nh = act ? min(kHeads, P.heads - h0) : 0;

    // the thread's two chunks of a row
    const int rslots = a.rot / (2 * V);
    const bool turn = slot < rslots;
    int ca, cb;
    if (INTERLEAVED || !turn) {
        ca = slot * 2 * V;
        cb = ca + V;
    } else {
        ca = slot * V;
        cb = ca + a.rot / 2;
    }

    // the position first: the table's row waits for it
    int pos = 0, axis = 0, p0 = 0;
    const int pairs = a.rot / (2 * a.axes);
    if (act && turn) {
        // V pairs lie on one axis: rot is a multiple of 2 V axes
        axis = slot * V / pairs;
        p0 = slot * V - axis * pairs;
        pos = __ldg(P.pos + (long long)axis * P.tokens + tok);
    }
    const T *x = static_cast<const T *>(P.x) + tok * P.x_t + h0 * P.x_h;
    T *y = static_cast<T *>(P.y) + tok * P.y_t + h0 * P.y_h;
    Packed<T, V> ra[kHeads], rb[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        if (i < nh) {
            ra[i].load(x + ca);
            rb[i].load(x + cb);
            x += P.x_h;
        } else {
#pragma unroll
            for (int j = 0; j < Packed<T, V>::W; ++j) ra[i].w[j] = rb[i].w[j] = 0u;
        }
    }
    float cs[V], sn[V];
    if (act && turn) {
        if (pos >= 0 && pos < a.positions) {
            const float4 *row = reinterpret_cast<const float4 *>(a.table + ((long long)pos * pairs + p0) * 2);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                const float4 t = __ldg(row + j);
                cs[2 * j] = t.x;
                sn[2 * j] = t.y;
                cs[2 * j + 1] = t.z;
                sn[2 * j + 1] = t.w;
            }
            if (a.inverse) {
#pragma unroll
                for (int j = 0; j < V; ++j) sn[j] = -sn[j];
            }
        } else {
            // a position outside the table: nothing is read, the rotated
            // elements become NaN and the device status says so
            atomicExch(status, kErrRange);
#pragma unroll
            for (int j = 0; j < V; ++j) cs[j] = sn[j] = __int_as_float(0x7fc00000);
        }
    }
    // Pair p of the thread is (fa[p], fb[p]), or with adjacent pairs (2p, 2p + 1)
    // of fa and fb in turn.  With the norm, the weights go into the factors:
    //   x -> rs (x wx cos - y wy sin),  y -> rs (y wy cos + x wx sin)
    auto px = [](int p) { return INTERLEAVED ? 2 * p : p; };
    auto py = [](int p) { return INTERLEAVED ? 2 * p + 1 : V + p; };
    // and where nothing is turned kx and ky are the weights.
    float kx[V], ky[V];   // wx cos, wy cos (wx sin and wy sin are cs and sn afterwards)
    if constexpr (NORM) {
        float w[2 * V];
#pragma unroll
        for (int j = 0; j < 2 * V; ++j) w[j] = 1.f;
        if (act && P.weight) {
            load_floats<V>(P.weight + ca, w);
            load_floats<V>(P.weight + cb, w + V);
        }
#pragma unroll
        for (int p = 0; p < V; ++p) {
            kx[p] = w[px(p)];
            ky[p] = w[py(p)];
            if (turn) {
                const float c = cs[p], s = sn[p];
                cs[p] = kx[p] * s;
                sn[p] = ky[p] * s;
                kx[p] *= c;
                ky[p] *= c;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        float f[2 * V];   // the thread's elements: chunk a, then chunk b
        ra[i].unpack(f);
        rb[i].unpack(f + V);
        float rs = 1.f;
        if constexpr (NORM) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 2 * V; ++j) ss = fmaf(f[j], f[j], ss);
            if (g.lanes > 16) ss += __shfl_xor_sync(0xffffffffu, ss, 16);
            if (g.lanes > 8) ss += __shfl_xor_sync(0xffffffffu, ss, 8);
            if (g.lanes > 4) ss += __shfl_xor_sync(0xffffffffu, ss, 4);
            if (g.lanes > 2) ss += __shfl_xor_sync(0xffffffffu, ss, 2);
            if (g.lanes > 1) ss += __shfl_xor_sync(0xffffffffu, ss, 1);
            rs = rsqrtf(fmaf(ss, g.inv_d, a.eps));
        }
        if (i >= nh) continue;
        if (turn) {
#pragma unroll
            for (int p = 0; p < V; ++p) {
                float &x = f[px(p)], &y = f[py(p)];
                const float u = x, v = y;
                if constexpr (NORM) {
                    x = rs * (u * kx[p] - v * sn[p]);
                    y = rs * (v * ky[p] + u * cs[p]);
                } else {
                    x = u * cs[p] - v * sn[p];
                    y = v * cs[p] + u * sn[p];
                }
            }
        } else if constexpr (NORM) {
#pragma unroll
            for (int p = 0; p < V; ++p) {
                f[px(p)] *= rs * kx[p];
                f[py(p)] *= rs * ky[p];
            }
        }
        ra[i].pack(f);
        rb[i].pack(f + V);
        ra[i].store(y + ca);
        rb[i].store(y + cb);
        y += P.y_h;
    }
}

template <class T, int V, bool INTERLEAVED, bool NORM>
cudaError_t launch_rot(const RotaryArgs &a, cudaStream_t st)
{
    RotGeom g;
    g.slots = a.D / (2 * V);
    g.inv_d = 1.f / (float)a.D;
    g.lanes = 1;
    while (g.lanes < g.slots) g.lanes *= 2;
    const int per_cta = kRotThreads / g.lanes;
    long long blocks[2];
    for (int i = 0; i < 2; ++i) {
        const long long units = (long long)a.part[i].tokens * ((a.part[i].heads + kHeads - 1) / kHeads);
        blocks[i] = (units + per_cta - 1) / per_cta;
    }
    g.blocks0 = blocks[0];
    if (blocks[0] + blocks[1] > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    int *status = device_status_ptr();
    if (!status) return cudaErrorInvalidDevice;
    rotary_kernel<T, V, INTERLEAVED, NORM><<<(unsigned)(blocks[0] + blocks[1]), kRotThreads, 0, st>>>(a, g, status);
    return cudaGetLastError();
}

template <class T, int V>
cudaError_t launch_rot_v(const RotaryArgs &a, cudaStream_t st)
{
    if (a.interleaved) return a.norm ? launch_rot<T, V, true, true>(a, st) : launch_rot<T, V, true, false>(a, st);
    return a.norm ? launch_rot<T, V, false, true>(a, st) : launch_rot<T, V, false, false>(a, st);
}

// Pair i of a position p is turned by p f_i, f_i = base^(-i / pairs) changed by
// the scaling rule.  All in 64 bits, rounded once: at positions of 10^5 and
// more a 32-bit product p f_i would be off by 10^-3 radians.  The angle is
// counted in turns, whose whole part is dropped before the sine; a thread has
// one pair and kTablePos positions, so that a power is taken once for them.
constexpr int kTablePos = 16;

__global__ void __launch_bounds__(256) rotary_table_kernel(const RotaryTableArgs a)
{
    const long long e = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const long long p0 = e / a.pairs * kTablePos;
    const int i = (int)(e % a.pairs);
    if (p0 >= a.positions) return;
    const double two_pi = 6.283185307179586476925;
    double f = pow(a.base, -(double)i / (double)a.pairs) / two_pi, magnitude = 1.0;
    if (a.rule == 1) {
        f /= a.factor;
    } else if (a.rule == 3) {
        const double keep = fmin(fmax((a.original * f - 1.0) / 31.0, 0.0), 1.0);
        f = f * keep + f / a.factor * (1.0 - keep);
        magnitude = 0.1 * log(a.factor) + 1.0;
    }
    const int n = (int)min((long long)kTablePos, a.positions - p0);
    for (int k = 0; k < n; ++k) {
        const double turns = (double)(p0 + k) * f;
        double s, c;
        sincospi(2.0 * (turns - rint(turns)), &s, &c);
        reinterpret_cast<float2 *>(a.table)[(p0 + k) * a.pairs + i] =
            make_float2((float)(c * magnitude), (float)(s * magnitude));
    }
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs &a, bool bf16, cudaStream_t st)
{
    if (!bf16) return launch_rot_v<float, 4>(a, st);
    // sixteen-byte chunks of eight bf16 where D and the rotated part are made
    // of whole pairs of them, else eight-byte ones
    if (a.D % 16 == 0 && a.rot % (16 * a.axes) == 0) return launch_rot_v<__nv_bfloat16, 8>(a, st);
    return launch_rot_v<__nv_bfloat16, 4>(a, st);
}

cudaError_t launch_rotary_table(const RotaryTableArgs &a, cudaStream_t st)
{
    const long long total = ((long long)a.positions + kTablePos - 1) / kTablePos * a.pairs;
    const long long blocks = (total + 255) / 256;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    rotary_table_kernel<<<(unsigned)blocks, 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace sc
