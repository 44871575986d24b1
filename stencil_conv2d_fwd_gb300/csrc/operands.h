// Argument checks that the C ABI of the attention and layer operators shares:
// where a strided tensor lies in memory, overlaps, alignment.
#pragma once

#include <cstdint>

#include "../../include/stencilconv.h"
#include "attn.h"
#include "launch.h"

namespace sc {

constexpr long long kMaxOffset = 1LL << 46;   // elements; keeps every byte offset far from 2^63

// A [n][t][h][D] tensor in memory: base address, sizes, strides in bytes.
struct Region {
    uintptr_t base;
    long long n, t, h, row;      // sizes; bytes of a row of D elements
    long long sn, st, sh;
};

inline long long region_bytes(const Region &r) { return (r.n - 1) * r.sn + (r.t - 1) * r.st + (r.h - 1) * r.sh + r.row; }

// Whether two tensors share a byte, or false only if they surely do not:
// disjoint ranges, or rows of one common token pitch whose heads lie in
// disjoint parts of the pitch (the queries and keys of one fused projection).
inline bool may_overlap(const Region &a, const Region &b)
{
    const uintptr_t a1 = a.base + (uintptr_t)region_bytes(a), b1 = b.base + (uintptr_t)region_bytes(b);
    if (a1 <= b.base || b1 <= a.base) return false;
    const long long s = a.st;
    const bool pitched = s > 0 && s == b.st && (a.n == 1 || a.sn % s == 0) && (b.n == 1 || b.sn % s == 0);
    const long long ea = (a.h - 1) * a.sh + a.row, eb = (b.h - 1) * b.sh + b.row;
    if (!pitched || ea > s || eb > s) return true;
    const long long d = (long long)((b.base >= a.base ? b.base - a.base : s - (a.base - b.base) % s) % (uintptr_t)s);
    return d < ea || d + eb > s;
}

inline bool flat_overlap(const Region &a, const void *p, long long bytes)
{
    if (!p || bytes <= 0) return false;
    const Region b{reinterpret_cast<uintptr_t>(p), 1, 1, 1, bytes, 0, bytes, 0};
    return may_overlap(a, b);
}

// Whether the rows of a tensor that is written are distinct: sorted by
// stride, each axis steps over all of the smaller ones.
inline bool rows_distinct(const Region &r)
{
    long long size[3] = {r.n, r.t, r.h}, stride[3] = {r.sn, r.st, r.sh};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (stride[j] < stride[i]) {
                const long long a = stride[i], b = size[i];
                stride[i] = stride[j];
                stride[j] = a;
                size[i] = size[j];
                size[j] = b;
            }
    long long extent = r.row;
    for (int i = 0; i < 3; ++i) {
        if (size[i] == 1) continue;
        if (stride[i] < extent) return false;
        extent += (size[i] - 1) * stride[i];
    }
    return true;
}

inline bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Product of sizes >= 1, or -1 if it passes the largest offset.
inline long long product(long long a, long long b, long long c = 1, long long d = 1)
{
    const long long v[4] = {a, b, c, d};
    long long n = 1;
    for (long long x : v) {
        if (x < 1 || n > kMaxOffset / x) return -1;
        n *= x;
    }
    return n;
}

// Strides of a tensor: the caller's, or those of packed [n][t][h][D].
// SC_ERR_SHAPE for a negative stride or one whose tensor is too large.
inline int take_strides(const sc_head_strides *s, int N, int T, int H, int D, HeadStrides &out)
{
    out.h = D;
    out.t = (long long)H * D;
    out.n = out.t * T;
    if (s) {
        out.n = s->batch;
        out.t = s->token;
        out.h = s->head;
    }
    const long long v[3] = {out.n, out.t, out.h}, size[3] = {N, T, H};
    for (int i = 0; i < 3; ++i)
        if (v[i] < 0 || (v[i] > 0 && size[i] - 1 > kMaxOffset / v[i])) return SC_ERR_SHAPE;
    return SC_OK;
}

inline bool strides_aligned(const HeadStrides &s, int N, int T, int H, int esize)
{
    const int v = 16 / esize;
    return (N == 1 || s.n % v == 0) && (T == 1 || s.t % v == 0) && (H == 1 || s.h % v == 0);
}

inline Region region(const void *p, int N, int T, int H, int D, const HeadStrides &s, int esize)
{
    return Region{reinterpret_cast<uintptr_t>(p), N, T, H, (long long)D * esize, s.n * esize, s.t * esize, s.h * esize};
}

inline int from_cuda(cudaError_t e)
{
    if (e == cudaSuccess) return SC_OK;
    if (e == cudaErrorInvalidConfiguration) return SC_ERR_SHAPE;   // more CTAs than a grid holds
    return record_cuda_error(e);
}

// The argument checks of cross_attention_fwd and cross_attention_q8_fwd (attn_api.cu).
int take_attention(const void *q, const void *k, const void *v, void *out, float *lse, const int *k_len,
                   const unsigned char *key_mask, int N, int Tq, int Tk, int Hq, int Hkv, int D, float scale, int dtype,
                   int state_bytes, const sc_attn_strides *strides, AttnArgs &a);

}  // namespace sc
