// C ABI of the attention operators: argument checks and dispatch.
// Declarations and contracts: include/stencilconv.h.
#include <cmath>
#include <cstdint>

#include "../../include/stencilconv.h"
#include "attn.h"
#include "launch.h"

namespace {

constexpr long long kMaxOffset = 1LL << 46;   // elements; keeps every byte offset far from 2^63

// A [n][t][h][D] tensor in memory: base address, sizes, strides in bytes.
struct Region {
    uintptr_t base;
    long long n, t, h, row;      // sizes; bytes of a row of D elements
    long long sn, st, sh;
};

long long region_bytes(const Region &r) { return (r.n - 1) * r.sn + (r.t - 1) * r.st + (r.h - 1) * r.sh + r.row; }

// Whether two tensors share a byte, or false only if they surely do not:
// disjoint ranges, or rows of one common token pitch whose heads lie in
// disjoint parts of the pitch (the queries and keys of one fused projection).
bool may_overlap(const Region &a, const Region &b)
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

bool flat_overlap(const Region &a, const void *p, long long bytes)
{
    if (!p || bytes <= 0) return false;
    const Region b{reinterpret_cast<uintptr_t>(p), 1, 1, 1, bytes, 0, bytes, 0};
    return may_overlap(a, b);
}

// Whether the rows of a tensor that is written are distinct: sorted by
// stride, each axis steps over all of the smaller ones.
bool rows_distinct(const Region &r)
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

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Product of sizes >= 1, or -1 if it passes the largest offset.
long long product(long long a, long long b, long long c = 1, long long d = 1)
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
int take_strides(const sc_head_strides *s, int N, int T, int H, int D, sc::HeadStrides &out)
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

bool strides_aligned(const sc::HeadStrides &s, int N, int T, int H, int esize)
{
    const int v = 16 / esize;
    return (N == 1 || s.n % v == 0) && (T == 1 || s.t % v == 0) && (H == 1 || s.h % v == 0);
}

Region region(const void *p, int N, int T, int H, int D, const sc::HeadStrides &s, int esize)
{
    return Region{reinterpret_cast<uintptr_t>(p), N, T, H, (long long)D * esize, s.n * esize, s.t * esize, s.h * esize};
}

int from_cuda(cudaError_t e)
{
    if (e == cudaSuccess) return SC_OK;
    if (e == cudaErrorInvalidConfiguration) return SC_ERR_SHAPE;   // more CTAs than a grid holds
    return sc::record_cuda_error(e);
}

// One tensor of a norm or rotation, and whether x and y are packed, whatever
// their strides say (two strides of 0 may be a row that all tokens and heads share).
struct Heads {
    sc_norm_heads t;
    bool packed_x, packed_y;
};

// The arguments of one tensor of a norm or rotation.
int take_heads(const Heads &heads, int D, int rot, int axes, int esize, sc::NormHeads &out, Region &rx, Region &ry)
{
    const sc_norm_heads &t = heads.t;
    if (!t.x || !t.y || (rot > 0 && !t.pos)) return SC_ERR_NULL;
    if (product(t.tokens, t.heads, D) < 0) return SC_ERR_SHAPE;
    const sc_head_strides sx{0, t.x_token_stride, t.x_head_stride}, sy{0, t.y_token_stride, t.y_head_stride};
    sc::HeadStrides hx, hy;
    if (take_strides(heads.packed_x ? nullptr : &sx, 1, t.tokens, t.heads, D, hx) != SC_OK) return SC_ERR_SHAPE;
    if (take_strides(heads.packed_y ? nullptr : &sy, 1, t.tokens, t.heads, D, hy) != SC_OK) return SC_ERR_SHAPE;
    if (!aligned(t.x, 16) || !aligned(t.y, 16) || !aligned(t.weight, 16) || !aligned(t.pos, 4)) return SC_ERR_ALIGN;
    if (!strides_aligned(hx, 1, t.tokens, t.heads, esize) || !strides_aligned(hy, 1, t.tokens, t.heads, esize))
        return SC_ERR_ALIGN;
    rx = region(t.x, 1, t.tokens, t.heads, D, hx, esize);
    ry = region(t.y, 1, t.tokens, t.heads, D, hy, esize);
    const bool in_place = t.x == t.y && (t.tokens == 1 || hx.t == hy.t) && (t.heads == 1 || hx.h == hy.h);
    if (!rows_distinct(ry) || (!in_place && may_overlap(rx, ry))) return SC_ERR_ALIAS;
    if (flat_overlap(ry, t.weight, 4LL * D) || flat_overlap(ry, t.pos, rot > 0 ? 4LL * axes * t.tokens : 0))
        return SC_ERR_ALIAS;
    out = sc::NormHeads{t.x, t.y, t.weight, t.pos, t.tokens, t.heads, hx.t, hx.h, hy.t, hy.h};
    return SC_OK;
}

// What rotary_fwd and qk_norm_rotary_fwd have in common.
int rotate_heads(const Heads *t0, const Heads *t1, const float *table, int D, int rot_dim, int positions,
                 bool norm, float eps, int mode, int axes, int inverse, int dtype, sc_stream_t stream)
{
    if (!t0 && !t1) return SC_ERR_NULL;
    if (rot_dim > 0 && !table) return SC_ERR_NULL;
    if (D < 1 || rot_dim < 0 || (rot_dim > 0 && positions < 1)) return SC_ERR_SHAPE;
    if (dtype != SC_F32 && dtype != SC_BF16) return SC_ERR_UNSUPPORTED;
    if (mode != SC_ROT_HALF && mode != SC_ROT_INTERLEAVED) return SC_ERR_UNSUPPORTED;
    if (axes != 1 && axes != 2) return SC_ERR_UNSUPPORTED;
    if (D % 8 != 0 || D > 256 || rot_dim > D || rot_dim % (8 * axes) != 0) return SC_ERR_UNSUPPORTED;
    if (norm && !(eps >= 0.f && std::isfinite(eps))) return SC_ERR_UNSUPPORTED;
    if (rot_dim > 0 && !aligned(table, 16)) return SC_ERR_ALIGN;
    sc::RotaryArgs a = {};
    a.table = table;
    a.D = D;
    a.rot = rot_dim;
    a.positions = positions;
    a.axes = axes;
    a.interleaved = mode == SC_ROT_INTERLEAVED;
    a.inverse = inverse != 0;
    a.norm = norm;
    a.eps = eps;
    const Heads *t[2] = {t0 ? t0 : t1, t0 ? t1 : nullptr};
    Region rx[2], ry[2];
    const long long table_bytes = rot_dim > 0 ? (long long)positions * (rot_dim / axes) * 4 : 0;
    for (int i = 0; i < 2 && t[i]; ++i) {
        const int rc = take_heads(*t[i], D, rot_dim, axes, dtype == SC_BF16 ? 2 : 4, a.part[i], rx[i], ry[i]);
        if (rc != SC_OK) return rc;
        if (flat_overlap(ry[i], table, table_bytes)) return SC_ERR_ALIAS;
    }
    if (t[1]) {
        if (may_overlap(ry[0], rx[1]) || may_overlap(ry[1], rx[0]) || may_overlap(ry[0], ry[1])) return SC_ERR_ALIAS;
        for (int i = 0; i < 2; ++i)
            if (flat_overlap(ry[i], t[1 - i]->t.weight, 4LL * D) ||
                flat_overlap(ry[i], t[1 - i]->t.pos, rot_dim > 0 ? 4LL * axes * t[1 - i]->t.tokens : 0))
                return SC_ERR_ALIAS;
    }
    return from_cuda(sc::launch_rotary(a, dtype == SC_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

// cross_attention_fwd's argument checks; SC_OK with `a` filled in when the
// call may launch.
int take_attention(const void *q, const void *k, const void *v, void *out, float *lse, const int *k_len,
                   const unsigned char *key_mask, int N, int Tq, int Tk, int Hq, int Hkv, int D, float scale, int dtype,
                   const sc_attn_strides *strides, sc::AttnArgs &a)
{
    if (!q || !k || !v || !out) return SC_ERR_NULL;
    if (product(N, Tq, Hq, D) < 0 || product(N, Tk, Hkv, D) < 0) return SC_ERR_SHAPE;
    if (Tq > (1 << 30) || Tk > (1 << 30)) return SC_ERR_SHAPE;
    if (product(N, Tq, Hq) > (1 << 30)) return SC_ERR_SHAPE;   // one index of 32 bits for a row
    if (dtype != SC_F32 && dtype != SC_BF16) return SC_ERR_UNSUPPORTED;
    if (Hq % Hkv != 0 || D % 8 != 0 || D > sc::kAttnMaxD) return SC_ERR_UNSUPPORTED;
    if (!(scale > 0.f) || !std::isfinite(scale)) return SC_ERR_UNSUPPORTED;
    const int es = dtype == SC_BF16 ? 2 : 4;
    a = sc::AttnArgs{};
    if (take_strides(strides ? &strides->q : nullptr, N, Tq, Hq, D, a.qs) != SC_OK ||
        take_strides(strides ? &strides->k : nullptr, N, Tk, Hkv, D, a.ks) != SC_OK ||
        take_strides(strides ? &strides->v : nullptr, N, Tk, Hkv, D, a.vs) != SC_OK ||
        take_strides(strides ? &strides->out : nullptr, N, Tq, Hq, D, a.os) != SC_OK)
        return SC_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
        !aligned(k_len, 4))
        return SC_ERR_ALIGN;
    if (!strides_aligned(a.qs, N, Tq, Hq, es) || !strides_aligned(a.ks, N, Tk, Hkv, es) ||
        !strides_aligned(a.vs, N, Tk, Hkv, es) || !strides_aligned(a.os, N, Tq, Hq, es))
        return SC_ERR_ALIGN;
    const Region rq = region(q, N, Tq, Hq, D, a.qs, es), rk = region(k, N, Tk, Hkv, D, a.ks, es);
    const Region rv = region(v, N, Tk, Hkv, D, a.vs, es), ro = region(out, N, Tq, Hq, D, a.os, es);
    const long long lse_bytes = lse ? 4LL * N * Hq * Tq : 0;
    if (!rows_distinct(ro) || may_overlap(ro, rq) || may_overlap(ro, rk) || may_overlap(ro, rv) ||
        flat_overlap(ro, k_len, 4LL * N) || flat_overlap(ro, key_mask, (long long)N * Tk) ||
        flat_overlap(ro, lse, lse_bytes) || flat_overlap(rq, lse, lse_bytes) || flat_overlap(rk, lse, lse_bytes) ||
        flat_overlap(rv, lse, lse_bytes))
        return SC_ERR_ALIAS;
    if (lse) {
        const Region rl{reinterpret_cast<uintptr_t>(lse), 1, 1, 1, lse_bytes, 0, lse_bytes, 0};
        if (flat_overlap(rl, k_len, 4LL * N) || flat_overlap(rl, key_mask, (long long)N * Tk)) return SC_ERR_ALIAS;
    }
    a.q = q;
    a.k = k;
    a.v = v;
    a.out = out;
    a.lse = lse;
    a.k_len = k_len;
    a.key_mask = key_mask;
    a.N = N;
    a.Tq = Tq;
    a.Tk = Tk;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = D;
    a.G = Hq / Hkv;
    a.scale = scale;
    return SC_OK;
}

}  // namespace

extern "C" {

int rotary_table_fwd(float *table, int positions, int pairs, double base, int rule, double factor, double original,
                     sc_stream_t stream)
{
    if (!table) return SC_ERR_NULL;
    if (product(positions, pairs) < 0) return SC_ERR_SHAPE;
    if (rule < SC_ROT_SCALE_NONE || rule > SC_ROT_SCALE_BANDS) return SC_ERR_UNSUPPORTED;
    if (!(base > 1.0) || !std::isfinite(base)) return SC_ERR_UNSUPPORTED;
    if (rule != SC_ROT_SCALE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return SC_ERR_UNSUPPORTED;
    if (rule == SC_ROT_SCALE_NTK && pairs < 2) return SC_ERR_UNSUPPORTED;
    if (rule == SC_ROT_SCALE_BANDS && (!(original > 0.0) || !std::isfinite(original))) return SC_ERR_UNSUPPORTED;
    if (!aligned(table, 16)) return SC_ERR_ALIGN;
    sc::RotaryTableArgs a{table, positions, pairs, rule, base, factor, original};
    if (rule == SC_ROT_SCALE_NTK) a.base = base * std::pow(factor, pairs / (pairs - 1.0));
    return from_cuda(sc::launch_rotary_table(a, reinterpret_cast<cudaStream_t>(stream)));
}

int rotary_fwd(const void *x, void *y, const float *table, const int *pos, int tokens, int heads, int D, int rot_dim,
               int positions, int mode, int axes, int inverse, int dtype, const sc_head_strides *x_strides,
               const sc_head_strides *y_strides, sc_stream_t stream)
{
    Heads xy = {};
    xy.packed_x = !x_strides;
    xy.packed_y = !y_strides;
    sc_norm_heads &t = xy.t;
    t.x = x;
    t.y = y;
    t.pos = pos;
    t.tokens = tokens;
    t.heads = heads;
    if (x_strides) {
        t.x_token_stride = x_strides->token;
        t.x_head_stride = x_strides->head;
    }
    if (y_strides) {
        t.y_token_stride = y_strides->token;
        t.y_head_stride = y_strides->head;
    }
    return rotate_heads(&xy, nullptr, table, D, rot_dim, positions, false, 0.f, mode, axes, inverse, dtype, stream);
}

int qk_norm_rotary_fwd(const sc_norm_heads *q, const sc_norm_heads *k, const float *table, int D, int rot_dim,
                       int positions, float eps, int mode, int axes, int dtype, sc_stream_t stream)
{
    const sc_norm_heads *t[2] = {q, k};
    Heads heads[2];
    for (int i = 0; i < 2; ++i)
        if (t[i])
            heads[i] = Heads{*t[i], t[i]->x_token_stride == 0 && t[i]->x_head_stride == 0,
                             t[i]->y_token_stride == 0 && t[i]->y_head_stride == 0};
    return rotate_heads(q ? &heads[0] : nullptr, k ? &heads[1] : nullptr, table, D, rot_dim, positions, true, eps, mode,
                        axes, 0, dtype, stream);
}

int cross_attention_fwd(const void *q, const void *k, const void *v, void *out, float *lse, const int *k_len,
                        const unsigned char *key_mask, int N, int Tq, int Tk, int Hq, int Hkv, int D, float scale,
                        int dtype, const sc_attn_strides *strides, sc_stream_t stream)
{
    sc::AttnArgs a;
    const int rc = take_attention(q, k, v, out, lse, k_len, key_mask, N, Tq, Tk, Hq, Hkv, D, scale, dtype, strides, a);
    if (rc != SC_OK) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool bf16 = dtype == SC_BF16;
    const long long rows = (long long)Tq * a.G;
    // More than 16 rows go to the tensor cores, except small fp32 calls: their
    // planes are a launch of their own there, and the warp-wide MMAs take row
    // blocks of 8 (4 heads of 64, 20 rows over 300 states 10.2 against 15.9 us; 8
    // heads, 77 rows over 1000 24.6 and 26.6; 4 x 8 heads, 40 rows over 1000, 82 M
    // products, 33.3 and 31.6).
    const double products = (double)N * Hq * Tq * (double)Tk * D;
    if (rows > 16 && (bf16 || products > 48e6)) return from_cuda(sc::launch_attn_tc(a, bf16, st));
    return from_cuda(!bf16 && rows <= 3 ? sc::launch_attn_rows(a, st) : sc::launch_attn_mma(a, bf16, st));
}

int sc_test_attn_wait_expiry(const void *q, const void *k, const void *v, void *out, int N, int Tq, int Tk, int Hq,
                             int Hkv, int D, int drop_copy, int timeout_us, sc_stream_t stream)
{
    sc::AttnArgs a;
    const int rc = take_attention(q, k, v, out, nullptr, nullptr, nullptr, N, Tq, Tk, Hq, Hkv, D, 1.f, SC_BF16, nullptr, a);
    if (rc != SC_OK) return rc;
    if (drop_copy < 0 || timeout_us < 1) return SC_ERR_SHAPE;
    sc::TcTest test;
    test.drop_copy = drop_copy;
    test.timeout_ns = 1000ull * (unsigned long long)timeout_us;
    return from_cuda(sc::launch_attn_tc(a, true, reinterpret_cast<cudaStream_t>(stream), test));
}

int sc_test_attn_slow_clear(const void *q, const void *k, const void *v, void *out, const int *k_len,
                            const unsigned char *key_mask, int N, int Tq, int Tk, int Hq, int Hkv, int D, int dtype,
                            int delay_us, sc_stream_t stream)
{
    sc::AttnArgs a;
    const int rc = take_attention(q, k, v, out, nullptr, k_len, key_mask, N, Tq, Tk, Hq, Hkv, D, 1.f, dtype, nullptr, a);
    if (rc != SC_OK) return rc;
    if (!k_len && !key_mask) return SC_ERR_NULL;
    if (delay_us < 0 || delay_us > 1000) return SC_ERR_SHAPE;
    sc::TcTest test;
    test.clear_delay_ns = 1000u * (unsigned)delay_us;
    return from_cuda(sc::launch_attn_tc(a, dtype == SC_BF16, reinterpret_cast<cudaStream_t>(stream), test));
}

}  // extern "C"
