// C ABI of the decoder layer's operators: argument checks and dispatch.
// Declarations and contracts: include/stencilconv.h.
#include <cmath>
#include <cstdint>

#include "layer.h"
#include "operands.h"

namespace {

using sc::Region;

constexpr int kMaxRows = 1 << 30;
// Rows that stream w through registers (linear_rows.cu) rather than go to the tensor
// cores (linear_tc.cu), which in fp32 first split x and w in a launch of their own.
//   bf16, w of 8192 x 2048: 16 rows 10.2 us, 17 there 14.9
//   fp32, w of 8192 x 2048: 32 rows 38.4, there 59.3; 48 rows 68.3, there 59.5
//   fp32, few products: 128 rows, w of 1024 x 1024 11.8, there 14.2; 1001 rows, 256 x 256 8.2 and
//   12.8; 64 rows, 2048 x 2048 19.7 and 19.6; 2000 rows, 256 x 128 10.2 and 9.6
bool few_rows(const sc::LinearArgs &a, bool bf16)
{
    if (bf16) return a.rows <= 16;
    return a.rows <= 32 || (a.rows <= 1024 && (double)a.rows * a.Cin * a.Cout <= 140e6);
}

constexpr long long kMaxMapStride = 1LL << 40;   // bytes

// [rows][cols] with a row stride in elements.
Region rows_region(const void *p, int rows, int cols, long long stride, int esize)
{
    return sc::region(p, 1, rows, 1, cols, sc::HeadStrides{0, stride, 0}, esize);
}

bool stride_ok(long long s, int rows) { return s >= 0 && (s == 0 || rows - 1 <= sc::kMaxOffset / s); }

// Whether output `o` is input `i` itself, row for row.
bool same_rows(const Region &o, const Region &i) { return o.base == i.base && o.row == i.row && (o.t == 1 || o.st == i.st); }

// The states' sizes and validity that kv_quantize_fwd and cross_attention_q8_fwd share.
int check_block(int D, int block, int code)
{
    if (D % 16 != 0 || D > sc::kAttnMaxD) return SC_ERR_UNSUPPORTED;
    if (block != 16 && block != 32 && block != 64 && block != 128) return SC_ERR_UNSUPPORTED;
    if (code != SC_CODE_I8 && code != SC_CODE_E4M3) return SC_ERR_UNSUPPORTED;
    return SC_OK;
}

int take_norm(const sc_norm *n, sc::NormArgs &out)
{
    out = sc::NormArgs{SC_NORM_NONE, 0.f, nullptr, nullptr};
    if (!n || n->kind == SC_NORM_NONE) return SC_OK;
    if (n->kind != SC_NORM_RMS && n->kind != SC_NORM_LAYER) return SC_ERR_UNSUPPORTED;
    if (!(n->eps >= 0.f) || !std::isfinite(n->eps)) return SC_ERR_UNSUPPORTED;
    if (!sc::aligned(n->weight, 16) || !sc::aligned(n->bias, 16)) return SC_ERR_ALIGN;
    out = sc::NormArgs{n->kind, n->eps, n->weight, n->bias};
    return SC_OK;
}

// linear_fwd's argument checks; SC_OK with `a` filled in when the call may launch.
int take_linear(const void *x, const void *w, const float *b, const void *residual, void *y, int rows, int Cin, int Cout, int act,
                int dtype, const sc_linear_strides *strides, sc::LinearArgs &a)
{
    if (!x || !w || !y) return SC_ERR_NULL;
    if (rows < 1 || Cin < 1 || Cout < 1 || rows > kMaxRows || Cin > kMaxRows || Cout > kMaxRows) return SC_ERR_SHAPE;
    if (sc::product(rows, Cin) < 0 || sc::product(rows, Cout) < 0 || sc::product(Cin, Cout) < 0) return SC_ERR_SHAPE;
    if (dtype != SC_F32 && dtype != SC_BF16) return SC_ERR_UNSUPPORTED;
    if (act < SC_ACT_NONE || act > SC_ACT_SILU) return SC_ERR_UNSUPPORTED;
    if (Cin % 8 != 0) return SC_ERR_UNSUPPORTED;
    const int es = dtype == SC_BF16 ? 2 : 4;
    a = sc::LinearArgs{x, w, b, residual, y, rows, Cin, Cout, act, Cin, Cin, Cout, Cout};
    if (strides) {
        a.xs = strides->x;
        a.ws = strides->w;
        a.ys = strides->y;
        a.rs = strides->residual;
    }
    if (!residual) a.rs = 0;
    // a single row's stride is not used
    if (rows == 1) {
        a.xs = Cin;
        a.ys = a.rs = Cout;
    }
    if (Cout == 1) a.ws = Cin;
    if (!stride_ok(a.xs, rows) || !stride_ok(a.ws, Cout) || !stride_ok(a.ys, rows) || !stride_ok(a.rs, rows)) return SC_ERR_SHAPE;
    if (a.xs < Cin || a.ws < Cin) return SC_ERR_UNSUPPORTED;
    if (!sc::aligned(x, 16) || !sc::aligned(w, 16) || !sc::aligned(y, es) || !sc::aligned(residual, es) || !sc::aligned(b, 4))
        return SC_ERR_ALIGN;
    if (a.xs % (16 / es) != 0 || a.ws % (16 / es) != 0) return SC_ERR_ALIGN;
    if (a.xs * es >= kMaxMapStride || a.ws * es >= kMaxMapStride || a.ys * es >= kMaxMapStride || a.rs * es >= kMaxMapStride)
        return SC_ERR_UNSUPPORTED;
    const Region rx = rows_region(x, rows, Cin, a.xs, es), rw = rows_region(w, Cout, Cin, a.ws, es);
    const Region ry = rows_region(y, rows, Cout, a.ys, es);
    if (!sc::rows_distinct(ry) || sc::may_overlap(ry, rx) || sc::may_overlap(ry, rw) || sc::flat_overlap(ry, b, 4LL * Cout))
        return SC_ERR_ALIAS;
    if (residual) {
        const Region rr = rows_region(residual, rows, Cout, a.rs, es);
        if (!same_rows(ry, rr) && sc::may_overlap(ry, rr)) return SC_ERR_ALIAS;
    }
    return SC_OK;
}

// cross_attention_q8_fwd's argument checks, as take_linear.
int take_q8(const void *q, const void *k, const float *k_scale, const void *v, const float *v_scale, void *out, float *lse,
            const int *k_len, const unsigned char *key_mask, int N, int Tq, int Tk, int Hq, int Hkv, int D, float scale, int block,
            int code, int dtype, const sc_attn_strides *strides, sc::AttnQ8Args &a)
{
    if (!k_scale || !v_scale) return SC_ERR_NULL;
    int rc = check_block(D, block, code);
    if (rc != SC_OK) return rc;
    rc = sc::take_attention(q, k, v, out, lse, k_len, key_mask, N, Tq, Tk, Hq, Hkv, D, scale, dtype, 1, strides, a);
    if (rc != SC_OK) return rc;
    if (!sc::aligned(k_scale, 4) || !sc::aligned(v_scale, 4)) return SC_ERR_ALIGN;
    // a tensor map's strides; states of one stride 0 would be one state
    if (Tk > 1 && (a.ks.t == 0 || a.vs.t == 0)) return SC_ERR_UNSUPPORTED;
    if (a.ks.n >= kMaxMapStride || a.ks.t >= kMaxMapStride || a.ks.h >= kMaxMapStride || a.vs.n >= kMaxMapStride ||
        a.vs.t >= kMaxMapStride || a.vs.h >= kMaxMapStride)
        return SC_ERR_UNSUPPORTED;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.block = block;
    a.log2_block = block == 16 ? 4 : (block == 32 ? 5 : (block == 64 ? 6 : 7));
    a.blocks = (Tk + block - 1) / block;
    const Region ro = sc::region(out, N, Tq, Hq, D, a.os, dtype == SC_BF16 ? 2 : 4);
    const long long bytes = 4LL * N * Hkv * a.blocks;
    if (sc::flat_overlap(ro, k_scale, bytes) || sc::flat_overlap(ro, v_scale, bytes)) return SC_ERR_ALIAS;
    if (lse) {
        const long long lse_bytes = 4LL * N * Hq * Tq;
        const Region rl{reinterpret_cast<uintptr_t>(lse), 1, 1, 1, lse_bytes, 0, lse_bytes, 0};
        if (sc::flat_overlap(rl, k_scale, bytes) || sc::flat_overlap(rl, v_scale, bytes)) return SC_ERR_ALIAS;
    }
    return SC_OK;
}

// The hooks of cross_attention_q8_fwd's bounded waits: its kernel of few rows, or of many.
int q8_wait_expiry(bool few, const void *q, const void *k, const float *k_scale, const void *v, const float *v_scale, void *out,
                   int N, int Tq, int Tk, int Hq, int Hkv, int D, int block, int code, int dtype, int drop_copy, int timeout_us,
                   cudaStream_t st)
{
    sc::AttnQ8Args a;
    const int rc = take_q8(q, k, k_scale, v, v_scale, out, nullptr, nullptr, nullptr, N, Tq, Tk, Hq, Hkv, D, 1.f, block, code, dtype,
                           nullptr, a);
    if (rc != SC_OK) return rc;
    if (drop_copy < 0 || timeout_us < 1) return SC_ERR_SHAPE;
    sc::TcTest test;
    test.drop_copy = drop_copy;
    test.timeout_ns = 1000ull * (unsigned long long)timeout_us;
    const bool bf16 = dtype == SC_BF16, e4m3 = code == SC_CODE_E4M3;
    return sc::from_cuda(few ? sc::launch_attn_q8(a, bf16, e4m3, st, test) : sc::launch_attn_tc_q8(a, bf16, e4m3, st, test));
}

}  // namespace

extern "C" {

int linear_fwd(const void *x, const void *w, const float *b, const void *residual, void *y, int rows, int Cin, int Cout,
               int act, int dtype, const sc_linear_strides *strides, sc_stream_t stream)
{
    sc::LinearArgs a;
    const int rc = take_linear(x, w, b, residual, y, rows, Cin, Cout, act, dtype, strides, a);
    if (rc != SC_OK) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool bf16 = dtype == SC_BF16;
    return sc::from_cuda(few_rows(a, bf16) ? sc::launch_linear_rows(a, bf16, st) : sc::launch_linear_tc(a, bf16, st));
}

int sc_test_linear_wait_expiry(const void *x, const void *w, const void *residual, void *y, int rows, int Cin, int Cout,
                               int dtype, int drop_copy, int timeout_us, sc_stream_t stream)
{
    sc::LinearArgs a;
    const int rc = take_linear(x, w, nullptr, residual, y, rows, Cin, Cout, SC_ACT_NONE, dtype, nullptr, a);
    if (rc != SC_OK) return rc;
    if (drop_copy < 0 || timeout_us < 1) return SC_ERR_SHAPE;
    sc::LinearTest test;
    test.drop_copy = drop_copy;
    test.timeout_ns = 1000ull * (unsigned long long)timeout_us;
    return sc::from_cuda(sc::launch_linear_tc(a, dtype == SC_BF16, reinterpret_cast<cudaStream_t>(stream), test));
}

int residual_norm_fwd(const void *x, const void *residual, void *sum, void *y, int rows, int C, const sc_norm *post,
                      const sc_norm *pre, const float *gate, int gate_rows, float scale, int dtype,
                      const sc_residual_strides *strides, sc_stream_t stream)
{
    if (!x || (!sum && !y)) return SC_ERR_NULL;
    if (rows < 1 || C < 1 || rows > kMaxRows || sc::product(rows, C) < 0) return SC_ERR_SHAPE;
    if (gate && gate_rows < 1) return SC_ERR_SHAPE;
    if (dtype != SC_F32 && dtype != SC_BF16) return SC_ERR_UNSUPPORTED;
    if (C % 8 != 0 || C > sc::kNormMaxC || !std::isfinite(scale)) return SC_ERR_UNSUPPORTED;
    sc::ResidualNormArgs a{x, residual, sum, y, gate, rows, C, gate ? gate_rows : rows, scale, {}, {}, C, C, C, C};
    int rc = take_norm(post, a.post);
    if (rc != SC_OK) return rc;
    if ((rc = take_norm(pre, a.pre)) != SC_OK) return rc;
    if (strides) {
        a.xs = strides->x;
        a.rs = strides->residual;
        a.ss = strides->sum;
        a.ys = strides->y;
    }
    if (rows == 1) a.xs = a.rs = a.ss = a.ys = C;
    if (!residual) a.rs = 0;
    if (!sum) a.ss = 0;
    if (!y) a.ys = 0;
    const int es = dtype == SC_BF16 ? 2 : 4, v = 16 / es;
    if (!stride_ok(a.xs, rows) || !stride_ok(a.rs, rows) || !stride_ok(a.ss, rows) || !stride_ok(a.ys, rows)) return SC_ERR_SHAPE;
    if (!sc::aligned(x, 16) || !sc::aligned(residual, 16) || !sc::aligned(sum, 16) || !sc::aligned(y, 16) ||
        !sc::aligned(gate, 16) || a.xs % v != 0 || a.rs % v != 0 || a.ss % v != 0 || a.ys % v != 0)
        return SC_ERR_ALIGN;
    const long long gate_bytes = gate ? ((long long)rows + gate_rows - 1) / gate_rows * C * 4 : 0;
    Region out[2];
    int outs = 0;
    if (sum) out[outs++] = rows_region(sum, rows, C, a.ss, es);
    if (y) out[outs++] = rows_region(y, rows, C, a.ys, es);
    for (int i = 0; i < outs; ++i) {
        const Region &o = out[i], rx = rows_region(x, rows, C, a.xs, es);
        if (!sc::rows_distinct(o) || (!same_rows(o, rx) && sc::may_overlap(o, rx))) return SC_ERR_ALIAS;
        if (residual) {
            const Region rr = rows_region(residual, rows, C, a.rs, es);
            if (!same_rows(o, rr) && sc::may_overlap(o, rr)) return SC_ERR_ALIAS;
        }
        if (sc::flat_overlap(o, gate, gate_bytes) || sc::flat_overlap(o, a.post.weight, 4LL * C) ||
            sc::flat_overlap(o, a.post.bias, 4LL * C) || sc::flat_overlap(o, a.pre.weight, 4LL * C) ||
            sc::flat_overlap(o, a.pre.bias, 4LL * C))
            return SC_ERR_ALIAS;
    }
    if (outs == 2 && sc::may_overlap(out[0], out[1])) return SC_ERR_ALIAS;
    return sc::from_cuda(sc::launch_residual_norm(a, dtype == SC_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

int kv_quantize_fwd(const sc_quant_states *k, const sc_quant_states *v, const int *k_len, const unsigned char *key_mask,
                    int N, int Tk, int Hkv, int D, int block, int code, int dtype, sc_stream_t stream)
{
    const sc_quant_states *t[2] = {k ? k : v, k ? v : nullptr};
    if (!t[0]) return SC_ERR_NULL;
    if (sc::product(N, Tk, Hkv, D) < 0 || Tk > kMaxRows) return SC_ERR_SHAPE;
    if (dtype != SC_F32 && dtype != SC_BF16) return SC_ERR_UNSUPPORTED;
    const int rc = check_block(D, block, code);
    if (rc != SC_OK) return rc;
    const int es = dtype == SC_BF16 ? 2 : 4;
    sc::QuantArgs a{};
    a.k_len = k_len;
    a.key_mask = key_mask;
    a.N = N;
    a.T = Tk;
    a.H = Hkv;
    a.D = D;
    a.block = block;
    a.blocks = (Tk + block - 1) / block;
    if (!sc::aligned(k_len, 4)) return SC_ERR_ALIGN;
    Region in[2], codes[2], scale[2];
    for (; a.parts < 2 && t[a.parts]; ++a.parts) {
        const sc_quant_states &s = *t[a.parts];
        sc::QuantPart &p = a.part[a.parts];
        if (!s.x || !s.codes || !s.scale) return SC_ERR_NULL;
        p.x = s.x;
        p.codes = static_cast<unsigned char *>(s.codes);
        p.scale = s.scale;
        if (sc::take_strides(s.packed_x ? nullptr : &s.x_strides, N, Tk, Hkv, D, p.xs) != SC_OK ||
            sc::take_strides(s.packed_codes ? nullptr : &s.code_strides, N, Tk, Hkv, D, p.cs) != SC_OK)
            return SC_ERR_SHAPE;
        if (!sc::aligned(s.x, 16) || !sc::aligned(s.codes, 16) || !sc::aligned(s.scale, 4) ||
            !sc::strides_aligned(p.xs, N, Tk, Hkv, es) || !sc::strides_aligned(p.cs, N, Tk, Hkv, 1))
            return SC_ERR_ALIGN;
        in[a.parts] = sc::region(s.x, N, Tk, Hkv, D, p.xs, es);
        codes[a.parts] = sc::region(s.codes, N, Tk, Hkv, D, p.cs, 1);
        const long long bytes = 4LL * N * Hkv * a.blocks;
        scale[a.parts] = Region{reinterpret_cast<uintptr_t>(s.scale), 1, 1, 1, bytes, 0, bytes, 0};
        if (!sc::rows_distinct(codes[a.parts])) return SC_ERR_ALIAS;
    }
    for (int i = 0; i < a.parts; ++i) {
        for (int j = 0; j < a.parts; ++j) {
            if (sc::may_overlap(codes[i], in[j]) || sc::may_overlap(scale[i], in[j]) || sc::may_overlap(scale[i], codes[j]) ||
                (i != j && (sc::may_overlap(codes[i], codes[j]) || sc::may_overlap(scale[i], scale[j]))))
                return SC_ERR_ALIAS;
        }
        if (sc::flat_overlap(codes[i], k_len, 4LL * N) || sc::flat_overlap(codes[i], key_mask, (long long)N * Tk) ||
            sc::flat_overlap(scale[i], k_len, 4LL * N) || sc::flat_overlap(scale[i], key_mask, (long long)N * Tk))
            return SC_ERR_ALIAS;
    }
    return sc::from_cuda(sc::launch_kv_quantize(a, dtype == SC_BF16, code == SC_CODE_E4M3, reinterpret_cast<cudaStream_t>(stream)));
}

int cross_attention_q8_fwd(const void *q, const void *k, const float *k_scale, const void *v, const float *v_scale,
                           void *out, float *lse, const int *k_len, const unsigned char *key_mask, int N, int Tq, int Tk,
                           int Hq, int Hkv, int D, float scale, int block, int code, int dtype,
                           const sc_attn_strides *strides, sc_stream_t stream)
{
    sc::AttnQ8Args a;
    const int rc = take_q8(q, k, k_scale, v, v_scale, out, lse, k_len, key_mask, N, Tq, Tk, Hq, Hkv, D, scale, block, code, dtype,
                           strides, a);
    if (rc != SC_OK) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool bf16 = dtype == SC_BF16, e4m3 = code == SC_CODE_E4M3;
    const long long rows = (long long)Tq * a.G;
    return sc::from_cuda(rows > 16 ? sc::launch_attn_tc_q8(a, bf16, e4m3, st) : sc::launch_attn_q8(a, bf16, e4m3, st));
}

int sc_test_attn_q8_wait_expiry(const void *q, const void *k, const float *k_scale, const void *v, const float *v_scale,
                                void *out, int N, int Tq, int Tk, int Hq, int Hkv, int D, int block, int code, int dtype,
                                int drop_copy, int timeout_us, sc_stream_t stream)
{
    return q8_wait_expiry(false, q, k, k_scale, v, v_scale, out, N, Tq, Tk, Hq, Hkv, D, block, code, dtype, drop_copy, timeout_us,
                          reinterpret_cast<cudaStream_t>(stream));
}

int sc_test_attn_q8_rows_wait_expiry(const void *q, const void *k, const float *k_scale, const void *v, const float *v_scale,
                                     void *out, int N, int Tq, int Tk, int Hq, int Hkv, int D, int block, int code, int dtype,
                                     int drop_copy, int timeout_us, sc_stream_t stream)
{
    return q8_wait_expiry(true, q, k, k_scale, v, v_scale, out, N, Tq, Tk, Hq, Hkv, D, block, code, dtype, drop_copy, timeout_us,
                          reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
