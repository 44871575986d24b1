// C ABI of the attention operators: argument checks and dispatch.
// Declarations and contracts: include/stencilconv.h.
#include <cmath>
#include <cstdint>

#include "../../include/stencilconv.h"
#include "attn.h"
#include "launch.h"
#include "operands.h"

namespace {

using sc::aligned;
using sc::flat_overlap;
using sc::from_cuda;
using sc::may_overlap;
using sc::product;
using sc::region;
using sc::Region;
using sc::rows_distinct;
using sc::strides_aligned;
using sc::take_strides;

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

}  // namespace

namespace sc {

// The argument checks of cross_attention_fwd and cross_attention_q8_fwd; SC_OK
// with `a` filled in when the call may launch.  Queries and output are of
// `dtype`, an element of a key or value has state_bytes bytes.
int take_attention(const void *q, const void *k, const void *v, void *out, float *lse, const int *k_len,
                   const unsigned char *key_mask, int N, int Tq, int Tk, int Hq, int Hkv, int D, float scale, int dtype,
                   int state_bytes, const sc_attn_strides *strides, AttnArgs &a)
{
    if (!q || !k || !v || !out) return SC_ERR_NULL;
    if (product(N, Tq, Hq, D) < 0 || product(N, Tk, Hkv, D) < 0) return SC_ERR_SHAPE;
    if (Tq > (1 << 30) || Tk > (1 << 30)) return SC_ERR_SHAPE;
    if (product(N, Tq, Hq) > (1 << 30)) return SC_ERR_SHAPE;   // one index of 32 bits for a row
    if (dtype != SC_F32 && dtype != SC_BF16) return SC_ERR_UNSUPPORTED;
    if (Hq % Hkv != 0 || D % 8 != 0 || D > kAttnMaxD) return SC_ERR_UNSUPPORTED;
    if (!(scale > 0.f) || !std::isfinite(scale)) return SC_ERR_UNSUPPORTED;
    const int es = dtype == SC_BF16 ? 2 : 4, ss = state_bytes;
    a = AttnArgs{};
    if (take_strides(strides ? &strides->q : nullptr, N, Tq, Hq, D, a.qs) != SC_OK ||
        take_strides(strides ? &strides->k : nullptr, N, Tk, Hkv, D, a.ks) != SC_OK ||
        take_strides(strides ? &strides->v : nullptr, N, Tk, Hkv, D, a.vs) != SC_OK ||
        take_strides(strides ? &strides->out : nullptr, N, Tq, Hq, D, a.os) != SC_OK)
        return SC_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
        !aligned(k_len, 4))
        return SC_ERR_ALIGN;
    if (!strides_aligned(a.qs, N, Tq, Hq, es) || !strides_aligned(a.ks, N, Tk, Hkv, ss) ||
        !strides_aligned(a.vs, N, Tk, Hkv, ss) || !strides_aligned(a.os, N, Tq, Hq, es))
        return SC_ERR_ALIGN;
    const Region rq = region(q, N, Tq, Hq, D, a.qs, es), rk = region(k, N, Tk, Hkv, D, a.ks, ss);
    const Region rv = region(v, N, Tk, Hkv, D, a.vs, ss), ro = region(out, N, Tq, Hq, D, a.os, es);
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

}  // namespace sc

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
    const int rc = sc::take_attention(q, k, v, out, lse, k_len, key_mask, N, Tq, Tk, Hq, Hkv, D, scale, dtype, dtype == SC_BF16 ? 2 : 4,
                                  strides, a);
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
    const int rc = sc::take_attention(q, k, v, out, nullptr, nullptr, nullptr, N, Tq, Tk, Hq, Hkv, D, 1.f, SC_BF16, 2, nullptr, a);
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
    const int rc = sc::take_attention(q, k, v, out, nullptr, k_len, key_mask, N, Tq, Tk, Hq, Hkv, D, 1.f, dtype,
                                  dtype == SC_BF16 ? 2 : 4, nullptr, a);
    if (rc != SC_OK) return rc;
    if (!k_len && !key_mask) return SC_ERR_NULL;
    if (delay_us < 0 || delay_us > 1000) return SC_ERR_SHAPE;
    sc::TcTest test;
    test.clear_delay_ns = 1000u * (unsigned)delay_us;
    return from_cuda(sc::launch_attn_tc(a, dtype == SC_BF16, reinterpret_cast<cudaStream_t>(stream), test));
}

}  // extern "C"
