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
// norm's weights in registers and all its loads issued first.
#include <cuda_bf16.h>

#include <cmath>

#include "attn.h"
#include "launch.h"

namespace sc {

namespace {

constexpr int kRotThreads = 256;
constexpr int kHeads = 4;   // heads of a token per thread

// V elements at p (16 bytes, or 8 for four bf16), to and from floats
template <int V>
__device__ __forceinline__ void load_v(const float *p, float (&f)[V])
{
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const float4 u = *reinterpret_cast<const float4 *>(p + i);
        f[i] = u.x;
        f[i + 1] = u.y;
        f[i + 2] = u.z;
        f[i + 3] = u.w;
    }
}
template <int V>
__device__ __forceinline__ void load_v(const __nv_bfloat16 *p, float (&f)[V])
{
    uint32_t w[V / 2];
    if constexpr (V == 8) {
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
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
template <int V>
__device__ __forceinline__ void store_v(float *p, const float (&f)[V])
{
#pragma unroll
    for (int i = 0; i < V; i += 4) *reinterpret_cast<float4 *>(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <int V>
__device__ __forceinline__ void store_v(__nv_bfloat16 *p, const float (&f)[V])
{
    if constexpr (V == 8)
        *reinterpret_cast<uint4 *>(p) = make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]),
                                                   bf16_pair(f[6], f[7]));
    else
        *reinterpret_cast<uint2 *>(p) = make_uint2(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]));
}

struct RotGeom {
    int lanes;           // threads per row: a power of two >= D / (2 V)
    int slots;           // D / (2 V)
    long long blocks0;   // CTAs of part[0]; the others do part[1]
};

template <class T, int V, bool INTERLEAVED, bool NORM>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotaryArgs a, const RotGeom g, int *status)
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

    const T *x = static_cast<const T *>(P.x) + tok * P.x_t + h0 * P.x_h;
    T *y = static_cast<T *>(P.y) + tok * P.y_t + h0 * P.y_h;
    float fa[kHeads][V], fb[kHeads][V];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        if (i < nh) {
            load_v<V>(x + i * P.x_h + ca, fa[i]);
            load_v<V>(x + i * P.x_h + cb, fb[i]);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) fa[i][j] = fb[i][j] = 0.f;
        }
    }
    float cs[V], sn[V];
    if (act && turn) {
        // V pairs lie on one axis: rot is a multiple of 2 V axes
        const int pairs = a.rot / (2 * a.axes);
        const int axis = slot * V / pairs, p0 = slot * V - axis * pairs;
        const int pos = P.pos[(long long)axis * P.tokens + tok];
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
    float wa[V], wb[V];
    if constexpr (NORM) {
#pragma unroll
        for (int j = 0; j < V; ++j) wa[j] = wb[j] = 1.f;
        if (act && P.weight) {
            load_v<V>(P.weight + ca, wa);
            load_v<V>(P.weight + cb, wb);
        }
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        if constexpr (NORM) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) ss = fmaf(fa[i][j], fa[i][j], fmaf(fb[i][j], fb[i][j], ss));
            for (int off = g.lanes / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            const float rs = rsqrtf(ss / (float)a.D + a.eps);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                fa[i][j] *= rs * wa[j];
                fb[i][j] *= rs * wb[j];
            }
        }
        if (i >= nh) continue;
        if (turn) {
            if (INTERLEAVED) {
                // pairs (0, 1), (2, 3), ... of the 2 V adjacent elements
#pragma unroll
                for (int j = 0; j < V; j += 2) {
                    const float p = fa[i][j], q = fa[i][j + 1];
                    fa[i][j] = p * cs[j / 2] - q * sn[j / 2];
                    fa[i][j + 1] = q * cs[j / 2] + p * sn[j / 2];
                    const float r = fb[i][j], s = fb[i][j + 1];
                    fb[i][j] = r * cs[V / 2 + j / 2] - s * sn[V / 2 + j / 2];
                    fb[i][j + 1] = s * cs[V / 2 + j / 2] + r * sn[V / 2 + j / 2];
                }
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float p = fa[i][j], q = fb[i][j];
                    fa[i][j] = p * cs[j] - q * sn[j];
                    fb[i][j] = q * cs[j] + p * sn[j];
                }
            }
        }
        store_v<V>(y + i * P.y_h + ca, fa[i]);
        store_v<V>(y + i * P.y_h + cb, fb[i]);
    }
}

template <class T, int V, bool INTERLEAVED, bool NORM>
cudaError_t launch_rot(const RotaryArgs &a, cudaStream_t st)
{
    RotGeom g;
    g.slots = a.D / (2 * V);
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
