/*
 * stencilconv: direct 2-D convolution forward pass and a fused
 * blur/unsharp stencil pipeline on NVIDIA GB300 (sm_103a).
 *
 * C ABI of libstencilconv.so.  Plain pointers and sizes only.
 *
 * Common conventions
 *  - Every tensor pointer is a DEVICE pointer owned by the caller; the
 *    library never frees or keeps it past the call's stream work.
 *  - Calls are asynchronous on `stream` (NULL = the legacy default stream)
 *    and return once the work is enqueued.  A nonzero return means nothing
 *    was enqueued (argument errors) or a launch failed (SC_ERR_CUDA).
 *  - Arguments are validated on the host before any launch; there is no CPU
 *    fallback.
 *  - All data is fp32 unless an entry point takes a dtype.  Sizes are ints; element offsets are computed in
 *    64-bit, so tensors may exceed 2^31 elements as long as each size fits.
 */
#ifndef STENCILCONV_H
#define STENCILCONV_H

#ifdef __cplusplus
extern "C" {
#endif

/* The library is built with hidden symbol visibility: only the functions
 * declared here are exported, so two copies of the library (or another
 * library with the same internal names) can be loaded in one process. */
#if defined(__GNUC__)
#pragma GCC visibility push(default)
#endif

struct CUstream_st;                     /* = cudaStream_t's target type */
typedef struct CUstream_st *sc_stream_t;

typedef enum {
    SC_OK = 0,
    SC_ERR_NULL = -1,            /* a required pointer is NULL */
    SC_ERR_SHAPE = -2,           /* a size is < 1, or the sizes overflow */
    SC_ERR_UNSUPPORTED = -3,     /* valid parameters the library does not run */
    SC_ERR_ALIGN = -4,           /* a pointer or stride is not 16-byte aligned */
    SC_ERR_ALIAS = -5,           /* output overlaps an input */
    SC_ERR_CUDA = -6,            /* a CUDA call failed; see sc_last_cuda_error */
    SC_ERR_DEVICE_TIMEOUT = -7,  /* a device-side bounded wait gave up */
    SC_ERR_RANGE = -8            /* a device-side index was outside its table */
} sc_status;

typedef enum { SC_NCHW = 0, SC_NHWC = 1 } sc_layout;
typedef enum {
    SC_ACT_NONE = 0,
    SC_ACT_RELU = 1,
    SC_ACT_GELU = 2,   /* v (1 + erf(v / sqrt 2)) / 2; linear_fwd only, as SC_ACT_SILU is */
    SC_ACT_SILU = 3    /* v / (1 + exp(-v)) */
} sc_act;
typedef enum { SC_F32 = 0, SC_BF16 = 1 } sc_dtype;   /* element type of an activation tensor */

/*
 * conv2d_fwd: y = act(conv(x, w) + b), stride 1, zero "same" padding.
 *
 * Operation ("Optimizing convolution kernels - CNNs in Vulkan Part 2/3",
 * section "Where we left off"; "Optimizing Memory Efficiency for
 * Convolution Kernels on Kepler GPUs", Section 3):
 *   y[n][h][w][co] = act( b[co] + sum_{ci<Cin} sum_{r<R} sum_{s<S}
 *                          X(n, h + r - R/2, w + s - S/2, ci) * w[co][ci][r][s] )
 * where X is x inside the image and 0 outside.  This is cross-correlation
 * (weights are not flipped).  act = ReLU is max(v, 0).
 *
 * x : N*H*W*Cin floats, layout `layout` (SC_NHWC: [N][H][W][Cin];
 *     SC_NCHW: [N][Cin][H][W]).
 * w : Cout*Cin*R*S floats, always [Cout][Cin][R][S] (OIHW), row-major.
 * b : Cout floats, or NULL for no bias.
 * y : N*H*W*Cout floats, same layout as x.  Must not overlap x, w or b.
 * R, S : odd, 1..7.
 * Supported: Cin == 1 with Cout == 1 or Cout % 4 == 0; Cin % 4 == 0 with
 *   Cout % 4 == 0.  x and y 16-byte aligned for Cin > 1 (NHWC vectors of 4
 *   channels).  Anything else returns SC_ERR_UNSUPPORTED / SC_ERR_ALIGN.
 * SC_NCHW with more than one channel on either side goes through the
 *   repack kernels and a stream-ordered temporary buffer (allocated on
 *   `stream` from the library's memory pool, freed on `stream` after use;
 *   see sc_release_workspace).
 * Returns SC_OK or a negative sc_status.
 */
int conv2d_fwd(const float *x, const float *w, const float *b, float *y,
               int N, int H, int W, int Cin, int Cout, int R, int S,
               int layout, int act, sc_stream_t stream);

/*
 * One layer of a convolution chain (conv2d_chain_fwd_host): filters w
 * (device memory, [Cout][Cin][R][S] fp32 with Cin the previous layer's
 * output channels), bias b (device memory, Cout floats, or NULL), the
 * filter size R x S and the activation (SC_ACT_NONE or SC_ACT_RELU).
 */
typedef struct {
    const float *w;
    const float *b;
    int Cout, R, S, act;
} sc_conv_layer;

#define SC_CHAIN_MAX_LAYERS 64

/*
 * conv2d_chain_fwd_host: a chain of convolution layers run on an input in
 * host memory, the result returned to host memory, as a network like the
 * upscaling network of "Optimizing convolution kernels - CNNs in Vulkan
 * Part 2/3" (opening paragraphs and "Where we left off": one image through
 * its layers in turn, each layer's output the next one's input):
 *   a_0 = x,  a_l = act_l(conv(a_{l-1}, w_l) + b_l) for l = 1..n_layers,
 *   y = a_{n_layers},
 * each conv exactly conv2d_fwd's (stride 1, zero "same" padding, NHWC).
 * On `stream`, in order: x_host is copied to the device, the layers run
 * with their activations in stream-ordered device buffers from the
 * library's memory pool (freed on `stream` after use; see
 * sc_release_workspace), and the last layer's output is copied to y_host.
 * The call returns once this is enqueued: x_host must stay unchanged and
 * y_host unread until the stream has completed it.  With page-locked
 * (pinned) host buffers both copies are asynchronous DMA transfers; with
 * pageable ones the CUDA runtime stages them and the call may wait for
 * the copies.
 * x_host : N*H*W*Cin floats, NHWC.  y_host : N*H*W*Cout floats of the last
 *   layer, NHWC.  layers : n_layers entries, 1 <= n_layers <=
 *   SC_CHAIN_MAX_LAYERS.
 * Every layer's shape is checked (conv2d_fwd's rules, with its Cin the
 * previous layer's Cout) before anything is enqueued: SC_ERR_NULL for a
 * NULL x_host, y_host, layers or w, SC_ERR_SHAPE / SC_ERR_UNSUPPORTED as
 * conv2d_fwd, SC_ERR_SHAPE for n_layers out of range.  A failed CUDA call
 * returns SC_ERR_CUDA (code in sc_last_cuda_error).
 */
int conv2d_chain_fwd_host(const float *x_host, float *y_host, int N, int H, int W, int Cin,
                          int n_layers, const sc_conv_layer *layers, sc_stream_t stream);

/*
 * conv2d_fwd_tc: the same operation as conv2d_fwd on the tensor cores
 * (tcgen05 MMA, accumulators in tensor memory) as an implicit GEMM
 * (pixels x output channels x (taps, input channels); "Optimizing Memory
 * Efficiency for Convolution Kernels on Kepler GPUs", Section 3.3, sets
 * this GEMM formulation against direct convolution).  x and w enter the
 * MMA as TF32 (10 explicit mantissa bits; the MMA drops the 13 low bits of
 * an fp32 operand, a relative error below 2^-10 per operand), products
 * accumulate in fp32, so results differ from conv2d_fwd by up to about
 * 5e-3 * sum|x * w| per element: a separate variant with its own
 * tolerance, not a replacement.
 * x, y : NHWC, 16-byte aligned.  w : OIHW, 16-byte aligned.  b : Cout
 *   floats or NULL.
 * Supported: Cin % 4 == 0, Cout % 4 == 0, Cout <= 128, R and S odd and <= 3,
 *   and filters small enough to stay resident in shared memory: each CTA
 *   holds the filters of a group of up to 32 output channels (and, while it
 *   starts, a second copy in OIHW order), so the group shrinks to 16, 8 or
 *   4 channels as Cin grows; beyond Cin of about 500, SC_ERR_UNSUPPORTED.
 * Returns SC_OK or a negative sc_status (SC_ERR_UNSUPPORTED outside that,
 *   SC_ERR_ALIGN for unaligned pointers).
 */
int conv2d_fwd_tc(const float *x, const float *w, const float *b, float *y,
                  int N, int H, int W, int Cin, int Cout, int R, int S,
                  int act, sc_stream_t stream);

/*
 * conv2d_fwd_tc_x3: conv2d_fwd_tc with fp32-level accuracy: every operand v
 * is split into a TF32 head hi(v) (v with its 13 low mantissa bits cleared)
 * and a remainder lo(v) = v - hi(v), and each product x * w is computed on
 * the tensor cores as hi(x) hi(w) + hi(x) lo(w) + lo(x) hi(w), the last two
 * in a separate accumulator added once at the end (split or "3xTF32"
 * arithmetic: Ootomo and Yokota, "Recovering single precision accuracy from
 * Tensor Cores while surpassing the FP32 theoretical peak performance",
 * 2022).  The dropped lo(x) lo(w) and the remainders' own TF32 truncation
 * keep every product within about 3 * 2^-20 of exact, so the result meets
 * conv2d_fwd's bound |y - y_ref| <= 1e-5 * (sum|x * w| + |b|).  Three TF32
 * products per product (issued as two MMAs, the filters' heads and
 * remainders side by side in N): a separate variant, not conv2d_fwd's FP32
 * FMA path.
 * Arguments, layouts and errors as for conv2d_fwd_tc.  Both the filters'
 * heads and remainders stay resident in shared memory, so the supported
 * Cin is about half of conv2d_fwd_tc's (about 250).
 */
int conv2d_fwd_tc_x3(const float *x, const float *w, const float *b, float *y,
                     int N, int H, int W, int Cin, int Cout, int R, int S,
                     int act, sc_stream_t stream);

/*
 * conv2d_fwd_tc_bf16: conv2d_fwd_tc with bf16 activation storage and BF16
 * tensor-core operands (tcgen05 kind::f16), fp32 accumulation.  Storing
 * activations in 16-bit floats halves their bytes ("Optimizing convolution
 * kernels - CNNs in Vulkan Part 2/3", the fp16 storage section: the traffic
 * halves at a small loss of precision).  x is bf16, the filters are fp32 and
 * rounded to bf16 (to nearest even) inside, b is fp32, y is bf16 (rounded to
 * nearest even) or fp32.  With x exact in bf16 (8 significant bits, unit
 * roundoff 2^-8), |y - y_ref| <= 2^-8 * sum|x*w| (weight rounding) + fp32
 * accumulation error, within 5e-3 * (sum |x * w| + |b|); a bf16 y adds its
 * own rounding, at most 2^-8 * |y_ref|.
 * x : N*H*W*Cin bf16 (NHWC), 16-byte aligned.  y : N*H*W*Cout elements of
 *   y_dtype (SC_F32 or SC_BF16), NHWC, 16-byte aligned.  w : OIHW fp32,
 *   16-byte aligned.  b : Cout floats or NULL.
 * Supported: Cin % 8 == 0, Cout % 4 == 0, Cout <= 128 (bf16 y with
 *   Cout > 16: Cout % 8 == 0), R and S odd and <= 3, filters that fit in
 *   shared memory as for conv2d_fwd_tc.
 * Returns SC_OK or a negative sc_status.
 */
int conv2d_fwd_tc_bf16(const void *x, const float *w, const float *b, void *y,
                       int N, int H, int W, int Cin, int Cout, int R, int S,
                       int act, int y_dtype, sc_stream_t stream);

/*
 * conv2d_fwd_tc_fused2: two 3 x 3 convolution layers in one pass on the
 * tensor cores, the intermediate activation kept on chip ("Optimizing
 * convolution kernels - CNNs in Vulkan Part 2/3", "Reducing memory traffic";
 * "Model-Based Warp Overlapped Tiling for Image Processing Programs on GPUs",
 * Abstract: overlapped tiles recompute the producer's halo):
 *   t = act1(conv(x, w1) + b1),  y = act2(conv(t, w2) + b2),
 * both "same"-padded with zeros (t is zero outside the image), TF32 operands,
 * fp32 accumulation.  Tolerance: layer 2 of the exact t within
 * 5e-3 * sum|t * w2|, plus layer 1's error (5e-3 * sum|x * w1| per element of
 * t) carried through |w2|.
 * x : N*H*W*C0 NHWC fp32.  w1 : C1*C0*3*3 OIHW.  b1 : C1 floats or NULL.
 * w2 : C2*C1*3*3 OIHW.  b2 : C2 floats or NULL.  y : N*H*W*C2 NHWC fp32.
 * x, y, w1, w2 16-byte aligned.
 * Supported: C0 % 4 == 0 with C0 <= 32 or so (its filters resident in
 *   shared memory beside two input stages), C1 == 32, C2 in {4, 8}.
 * Returns SC_OK or a negative sc_status.
 */
int conv2d_fwd_tc_fused2(const float *x, const float *w1, const float *b1,
                         const float *w2, const float *b2, float *y,
                         int N, int H, int W, int C0, int C1, int C2,
                         int act1, int act2, sc_stream_t stream);

/*
 * ---------------------------------------------------------------------
 * Attention over a feature map.  An NHWC feature map [N][H][W][C] is, as it
 * lies in memory, a batch of N sequences of H*W states of C = heads * D
 * channels: 1x1 convolutions of it (conv2d_fwd, conv2d_fwd_tc_bf16) are the
 * keys and values of the attention below, a pixel (y, x) being state y*W + x
 * with the two positions y and x.
 * ---------------------------------------------------------------------
 */

/* Strides, in elements, of a [batch][token][head][D] tensor whose D elements
 * are contiguous.  Non-negative multiples of 16 bytes (0 on an axis that all
 * share); an axis of size 1 may have any. */
typedef struct {
    long long batch, token, head;
} sc_head_strides;

typedef struct {
    sc_head_strides q, k, v, out;
} sc_attn_strides;

/*
 * cross_attention_fwd: attention of Tq query tokens to Tk states of another
 * length ("Attention Is All You Need", Sections 3.2.1 and 3.2.3; key heads
 * shared by groups of query heads as in "GQA: Training Generalized
 * Multi-Query Transformer Models from Multi-Head Checkpoints"):
 *   s_j = scale * sum_d q[n][t][h][d] k[n][j][h * Hkv / Hq][d]   for the valid states j of sequence n
 *   out[n][t][h] = sum_j exp(s_j) v[n][j][h * Hkv / Hq] / sum_j exp(s_j)
 *   lse[n][h][t] = log(sum_j exp(s_j))
 * State j of sequence n is valid if j < k_len[n] and key_mask[n][j] != 0.
 * Without a valid state, out is 0 and lse is -infinity.  What the keys and
 * values of states that are not valid hold (NaN included) has no effect.
 * q, out : [N][Tq][Hq][D], k, v : [N][Tk][Hkv][D], all of `dtype` (SC_F32 or
 *   SC_BF16), 16-byte aligned, packed in that order if strides is NULL.  out
 *   overlaps no input.
 * lse : N*Hq*Tq floats, or NULL.
 * k_len : N ints in device memory (a value below 0 counts as 0, one above Tk
 *   as Tk), or NULL for Tk.  key_mask : N*Tk bytes, or NULL.
 * Supported: Hq % Hkv == 0; D % 8 == 0, D <= 128; scale > 0; Tq, Tk and
 *   N*Tq*Hq up to 2^30.
 * Scores, weights exp(s_j - m) and sums are fp32.  bf16 tensors: each weight
 * is rounded to bf16 (a relative error up to 2^-8) where it multiplies a value,
 * the sum that divides is one of unrounded weights, and the output is rounded
 * once (to nearest even).  The sums of weight times value have to stay within
 * fp32's range, m being the row's largest score so far, or for bf16 tensors up
 * to 8 log 2 below it.
 * Infinities and NaN in queries and valid states follow the formula, but that
 * a row whose scores are all -infinity counts as one without a valid state.
 * fp32 tensors with more than 3 rows a key head (Tq * Hq / Hkv) are multiplied
 * in three bf16 planes of 24 bits in all: there an infinity times another, or
 * a key's times a query's element above 256, may be NaN, and an element below
 * 2^-110 keeps 2^-134, not 24 bits.
 * A call may take a stream-ordered temporary buffer (see
 * sc_release_workspace).  Returns SC_OK or a negative sc_status.
 */
int cross_attention_fwd(const void *q, const void *k, const void *v, void *out, float *lse, const int *k_len,
                        const unsigned char *key_mask, int N, int Tq, int Tk, int Hq, int Hkv, int D, float scale,
                        int dtype, const sc_attn_strides *strides, sc_stream_t stream);

/* Which elements of a head are a pair: i and i + rot_dim / 2, or 2 i and 2 i + 1. */
typedef enum { SC_ROT_HALF = 0, SC_ROT_INTERLEAVED = 1 } sc_rot_mode;

/* Scaling of a rotation's frequencies for contexts longer than the original one. */
typedef enum {
    SC_ROT_SCALE_NONE = 0,
    SC_ROT_SCALE_LINEAR = 1,   /* f / factor ("Extending Context Window of Large Language Models via Positional
                                  Interpolation") */
    SC_ROT_SCALE_NTK = 2,      /* base * factor^(pairs / (pairs - 1)) */
    SC_ROT_SCALE_BANDS = 3     /* by the turns of a pair over `original` positions: more than 32 keep f, fewer than
                                  one get f / factor, a linear blend between; cos and sin times
                                  0.1 log(factor) + 1 ("YaRN: Efficient Context Window Extension of Large Language
                                  Models", Section 3) */
} sc_rot_scale;

/*
 * rotary_table_fwd: cosines and sines of a rotation ("RoFormer: Enhanced
 * Transformer with Rotary Position Embedding", Section 3.2.2), made once and
 * kept by the caller: table[p][i] = (cos, sin)(p f_i), 0 <= p < positions,
 * 0 <= i < pairs, f_i = base^(-i / pairs) changed by `rule` (sc_rot_scale).
 * Computed in 64 bits, rounded once.
 * table : positions * pairs * 2 floats, 16-byte aligned.  base > 1.
 * factor >= 1 (not used by SC_ROT_SCALE_NONE).  original > 0: the context
 *   that SC_ROT_SCALE_BANDS counts turns over (not used by the others).
 *   SC_ROT_SCALE_NTK needs pairs >= 2.
 * Returns SC_OK or a negative sc_status.
 */
int rotary_table_fwd(float *table, int positions, int pairs, double base, int rule, double factor, double original,
                     sc_stream_t stream);

/*
 * rotary_fwd: rotates each head's first rot_dim elements by its token's
 * position: pair i of (a, b) becomes (a cos - b sin, b cos + a sin) with
 * (cos, sin) = table[p][i]; the others are copied.  With inverse != 0 by the
 * opposite angle (the transposed map).
 * axes 1: pairs = rot_dim / 2, p = pos[t].  axes 2 (a feature map's row and
 *   column): pairs = rot_dim / 4, the first half of the rot_dim / 2 pairs is
 *   turned by p = pos[t], the second by p = pos[tokens + t], each with the
 *   table's pairs from the first.
 * x, y : [tokens][heads][D] of `dtype`, 16-byte aligned, packed unless
 *   strides are given (their batch stride is not used; 0 on an axis of x that
 *   shares one row, 0 on both included).  y's rows are distinct; y may be x
 *   (with the same strides), else it overlaps no input.
 * table : positions * pairs * 2 floats of rotary_table_fwd.  pos : axes *
 *   tokens ints in device memory; for a position outside [0, positions) the
 *   elements that it turns become NaN (with axes 2, those of its axis's pairs)
 *   and sc_last_device_status returns SC_ERR_RANGE.
 * Supported: D % 8 == 0, D <= 256; rot_dim <= D, rot_dim % (8 * axes) == 0
 *   (with rot_dim 0, table and pos may be NULL).
 * Returns SC_OK or a negative sc_status.
 */
int rotary_fwd(const void *x, void *y, const float *table, const int *pos, int tokens, int heads, int D, int rot_dim,
               int positions, int mode, int axes, int inverse, int dtype, const sc_head_strides *x_strides,
               const sc_head_strides *y_strides, sc_stream_t stream);

/* One tensor of qk_norm_rotary_fwd: x and y as in rotary_fwd (token and head
 * strides in elements; both 0: packed, so that tokens that share one row need
 * a head stride above 0, also with one head), weight D floats (16-byte
 * aligned) or NULL for ones. */
typedef struct {
    const void *x;
    void *y;
    const float *weight;
    const int *pos;
    int tokens, heads;
    long long x_token_stride, x_head_stride, y_token_stride, y_head_stride;
} sc_norm_heads;

/*
 * qk_norm_rotary_fwd: RMS norm of each head of the queries and the keys
 * ("Root Mean Square Layer Normalization"; per head as in "Scaling Vision
 * Transformers to 22 Billion Parameters", Section 2) and their rotation, in
 * one pass and one launch:
 *   y = rotate(x * (mean_d(x^2) + eps)^(-1/2) * weight)
 * The rotation as rotary_fwd's.  q and k may have different numbers of
 * tokens and heads; either may be NULL (a step's queries whose keys are kept).
 * Returns SC_OK or a negative sc_status.
 */
int qk_norm_rotary_fwd(const sc_norm_heads *q, const sc_norm_heads *k, const float *table, int D, int rot_dim,
                       int positions, float eps, int mode, int axes, int dtype, sc_stream_t stream);

/*
 * ---------------------------------------------------------------------
 * A decoder layer around the attention: its products, its norms, and the
 * feature map's states held in 8 bits.
 * ---------------------------------------------------------------------
 */

/* Strides, in elements, from one row of linear_fwd's tensors to the next. */
typedef struct {
    long long x, w, y, residual;
} sc_linear_strides;

/*
 * linear_fwd: y = act(x w^T + b) + residual, a decoder's projections and MLP
 * ("Attention Is All You Need", Sections 3.2.2 and 3.3) and the 1x1 convolution
 * of a feature map whose pixels are the rows:
 *   y[i][o] = act( sum_c x[i][c] w[o][c] + b[o] ) + residual[i][o]
 * act : SC_ACT_NONE, SC_ACT_RELU, SC_ACT_GELU ("Gaussian Error Linear Units",
 *   the form with erf) or SC_ACT_SILU.  A NaN stays one.
 * x : [rows][Cin], w : [Cout][Cin] (the order of conv2d_fwd's 1x1 filters),
 *   y, residual : [rows][Cout], all of `dtype` (SC_F32 or SC_BF16); b : Cout
 *   floats, or NULL for none; residual NULL for none.  Packed if strides is
 *   NULL.
 * Rows of x and w are 16-byte aligned (Cin % 8 == 0, strides multiples of 16
 *   bytes, at least Cin).  Rows of y and residual are aligned to an element
 *   only, any Cout and strides; y's are distinct, a residual stride of 0 is a
 *   row that all share.  y may be residual (with the same stride), else it
 *   overlaps no input.
 * Products and sums are fp32, and so is everything up to y, which is rounded
 * once (to nearest even).  With bf16 tensors GELU's normal distribution is good to
 * 2^-22 of 1 (not of a far negative v's small tail: 0.4% of it at v = -6, 2% at -10),
 * SiLU to 2^-16 of itself (0 for v < -87.3; with fp32 ones for v < -88.7).  fp32 tensors of more than 4 rows are multiplied in
 * three bf16 planes of 24 bits in all: there an infinity times another, or times
 * an element above 256, may be NaN, and an element below 2^-110 keeps 2^-134.
 * Supported: rows, Cin and Cout up to 2^30, strides below 2^40 bytes.  A call may
 * take a stream-ordered temporary buffer (see sc_release_workspace): with fp32
 * tensors on the tensor cores 6 bytes for each element of x and w.  Returns SC_OK or a negative
 * sc_status.
 */
int linear_fwd(const void *x, const void *w, const float *b, const void *residual, void *y, int rows, int Cin, int Cout,
               int act, int dtype, const sc_linear_strides *strides, sc_stream_t stream);

typedef enum { SC_NORM_NONE = 0, SC_NORM_RMS = 1, SC_NORM_LAYER = 2 } sc_norm_kind;

/* One norm of residual_norm_fwd: weight and bias C floats (16-byte aligned), or
 * NULL for ones and zeros. */
typedef struct {
    int kind;
    float eps;
    const float *weight, *bias;
} sc_norm;

/* Strides, in elements, from one row of residual_norm_fwd's tensors to the next. */
typedef struct {
    long long x, residual, sum, y;
} sc_residual_strides;

/*
 * residual_norm_fwd: the norm behind a block, its gate, the residual stream
 * and the norm before the next block, in one pass:
 *   t = post(x),  s = scale * residual + gate * t,  sum = s,  y = pre(s)
 *   SC_NORM_NONE:  v
 *   SC_NORM_RMS:   v * (mean(v^2) + eps)^(-1/2) * weight + bias
 *   SC_NORM_LAYER: (v - mean(v)) * (mean((v - mean(v))^2) + eps)^(-1/2) * weight + bias
 * ("Root Mean Square Layer Normalization"; "Layer Normalization"), over the C
 * elements of a row.  y is of s as it is in fp32, before sum's rounding.
 * x, residual, sum, y : [rows][C] of `dtype`, 16-byte aligned, packed if
 *   strides is NULL (multiples of 16 bytes; 0 on x or residual is a row that
 *   all share).  residual NULL: s = gate * t.  sum or y may be NULL, not both.
 *   Either may be x or residual (with the same stride), else it overlaps no
 *   input; they do not overlap one another.
 * post, pre : NULL for SC_NORM_NONE.  (A pre that is SC_NORM_NONE makes y the
 *   sum.)
 * gate : [(rows + gate_rows - 1) / gate_rows][C] floats, 16-byte aligned: row i
 *   takes gate row i / gate_rows (gate_rows the tokens of a sequence, or rows
 *   for one gate).  NULL for ones.
 * Supported: C % 8 == 0, C <= 16384; finite scale, eps >= 0 and finite.
 * Sums, means and all that leads to an output are fp32; each output is rounded
 * once (to nearest even).
 * Returns SC_OK or a negative sc_status.
 */
int residual_norm_fwd(const void *x, const void *residual, void *sum, void *y, int rows, int C, const sc_norm *post,
                      const sc_norm *pre, const float *gate, int gate_rows, float scale, int dtype,
                      const sc_residual_strides *strides, sc_stream_t stream);

/* What a byte of an 8-bit state stands for: an integer (-128 .. 127), or a
 * float of 4 exponent and 3 mantissa bits without infinities (up to 448;
 * 0x7f and 0xff are NaN). */
typedef enum { SC_CODE_I8 = 0, SC_CODE_E4M3 = 1 } sc_code;

/* One tensor of kv_quantize_fwd: x as in cross_attention_fwd, codes the same
 * with one byte an element, scale [N][Hkv][(Tk + block - 1) / block] floats.
 * packed_x, packed_codes != 0: packed, whatever the strides say. */
typedef struct {
    const void *x;
    void *codes;
    float *scale;
    int packed_x, packed_codes;
    sc_head_strides x_strides, code_strides;
} sc_quant_states;

/*
 * kv_quantize_fwd: keys and values in 8 bits with one scale for each block of
 * `block` states and head.  With a the largest |x| over the block's valid
 * states and the head's D elements, and top = 127 (SC_CODE_I8) or 448
 * (SC_CODE_E4M3):
 *   scale = a / top,   code = the code nearest to top * x / a (a tie to the even one)
 * the quotient as in exact arithmetic.  A block of zeros has scale 0 and codes
 * 0; one with an infinity or NaN in a valid state has scale NaN and codes 0.
 * State j of sequence n is valid if j < k_len[n] and key_mask[n][j] != 0
 * (NULL: all).  Others are not read; their codes, and the scales of blocks
 * without a valid state, are left as they were.
 * x : [N][Tk][Hkv][D] of `dtype`; k or v may be NULL (not both).  x, codes and
 *   scale do not overlap.  To append whole blocks of states to a cache of Tk
 *   places, mask the others out.
 * Supported: D % 16 == 0, D <= 128; block 16, 32, 64 or 128; rows of x and of
 *   codes 16-byte aligned.  Returns SC_OK or a negative sc_status.
 */
int kv_quantize_fwd(const sc_quant_states *k, const sc_quant_states *v, const int *k_len, const unsigned char *key_mask,
                    int N, int Tk, int Hkv, int D, int block, int code, int dtype, sc_stream_t stream);

/*
 * cross_attention_q8_fwd: cross_attention_fwd over states held as
 * kv_quantize_fwd leaves them,
 *   k[n][j][h][d] = k_scale[n][h][j / block] * code(k[n][j][h][d]),  v likewise,
 * which reads half the bytes of bf16 states.  With few rows that is time gained;
 * with bf16 tensors and more rows a call takes longer than over bf16 states (77 tokens
 * of 32 sequences over 3136 states: 81 us, 47), as the codes are converted on their way
 * to the tensor cores.  Calls of several tiles of 128 rows a key head, and of more
 * tiles than the GPU has SMs, expand the codes first (fp32: D <= 64), into a temporary
 * buffer of twice the size of k and v.
 * q, out : [N][Tq][Hq][D] of `dtype`.  k, v : [N][Tk][Hkv][D] bytes; strides'
 *   k and v count bytes.  k_scale, v_scale : [N][Hkv][(Tk + block - 1) / block]
 *   floats, 4-byte aligned.  Everything else as in cross_attention_fwd; what
 *   states that are not valid hold, and the scales of blocks without a valid
 *   state, have no effect.
 * Codes are multiplied as they are; the scales enter in fp32.
 * Up to 16 rows a key head (Tq * Hq / Hkv): fp32 queries and weights are taken to
 * 22 bits, in two planes of fp16 (queries with a power of two for each row, whose
 * largest element times scale is 2^-110 or more; sums of |v| over the states up to
 * 2^112); a query with an infinity or NaN gives NaN.  With bf16 tensors each weight is
 * rounded to fp16 where it multiplies a code (a relative error up to 2^-11).  A
 * weight below 2^-28 of the largest one among its 16 or 32 neighbours keeps 2^-39
 * of that.
 * More rows: as in cross_attention_fwd, but that it is a weight times its state's
 * scale that is taken in three planes, or with bf16 tensors rounded to fp16 (one
 * below 2^-20 of the row's largest keeps 2^-31 of that; v_scale 0, or between 2^-80
 * and 2^80 in size).
 * The output is rounded once (to nearest even).
 * Supported: D % 16 == 0, D <= 128; block 16, 32, 64 or 128; strides of k and v
 * below 2^40 bytes, their token strides above 0; otherwise as
 * cross_attention_fwd.  Returns SC_OK or a negative sc_status.
 */
int cross_attention_q8_fwd(const void *q, const void *k, const float *k_scale, const void *v, const float *v_scale,
                           void *out, float *lse, const int *k_len, const unsigned char *key_mask, int N, int Tq, int Tk,
                           int Hq, int Hkv, int D, float scale, int block, int code, int dtype,
                           const sc_attn_strides *strides, sc_stream_t stream);

/*
 * stencil_pipeline_fwd: three stencil stages fused in one pass over a
 * single-channel image ("Model-Based Warp Overlapped Tiling for Image
 * Processing Programs on GPUs", Abstract: stages fused into overlapped
 * warp-sized tiles):
 *   t1[y][x] = sum_{k=-2..2} c_k in[y][clamp(x+k, 0, W-1)]
 *   t2[y][x] = sum_{k=-2..2} c_k t1[clamp(y+k, 0, H-1)][x]
 *   out      = min(max(in + 1.5 (in - t2), 0), 1),   c = (1,4,6,4,1)/16.
 * in, out : H*W floats, row-major with pitch W; must not overlap.
 * The intermediates t1 and t2 never leave the chip.
 * Returns SC_OK or a negative sc_status.
 */
int stencil_pipeline_fwd(const float *in, float *out, int H, int W, sc_stream_t stream);

/*
 * sc_repack: change activation layout between NCHW and NHWC
 * ("Optimizing convolution kernels - CNNs in Vulkan Part 2/3", section
 * "Vectorization": the channels of one pixel stored next to each other so
 * a thread moves four of them as one 16-byte vector).
 * src, dst : N*C*H*W floats, device, non-overlapping.
 * src_layout, dst_layout : SC_NCHW or SC_NHWC; equal layouts copy.
 * Returns SC_OK or a negative sc_status.
 */
int sc_repack(const float *src, float *dst, int N, int C, int H, int W,
              int src_layout, int dst_layout, sc_stream_t stream);

/*
 * sc_last_device_status: synchronize `stream`, then return and clear the
 * device-side status word of the current device (SC_OK,
 * SC_ERR_DEVICE_TIMEOUT when a kernel's bounded wait expired, or
 * SC_ERR_RANGE when a position lay outside a rotation table).  Returns
 * SC_ERR_CUDA if the synchronization itself failed.
 */
int sc_last_device_status(sc_stream_t stream);

/* sc_status_string: static English text for a status code (never NULL). */
const char *sc_status_string(int status);

/* sc_last_cuda_error: the cudaError_t value behind the last SC_ERR_CUDA
 * returned on this host thread (0 if none). */
int sc_last_cuda_error(void);

/*
 * sc_measure_ffma_peak: measurement helper, not part of the operation.
 * Runs `blocks` CTAs of 256 threads, each thread doing `iters` iterations
 * of 16 independent fp32 FMA chains (32 FLOP per chain step), and writes
 * one float per thread to `sink` (device, blocks*256 floats) so nothing is
 * optimised away.  Time it on `stream` to measure the FP32 FFMA rate.
 * Returns SC_OK or a negative sc_status.
 */
int sc_measure_ffma_peak(float *sink, int blocks, int iters, sc_stream_t stream);

/*
 * sc_empty_kernel: measurement helper, not part of the operation.  Launches
 * a kernel of `blocks` CTAs of `threads` threads that does nothing, on
 * `stream`; a run of such launches (e.g. replayed from a CUDA graph) gives
 * the cost of one launch, the floor under any kernel of the library.
 * Returns SC_OK, SC_ERR_SHAPE for blocks outside [1, 2^24] or threads
 * outside [1, 1024], or SC_ERR_CUDA.
 */
int sc_empty_kernel(int blocks, int threads, sc_stream_t stream);

/* sc_version: library version as 10000*major + 100*minor + patch. */
int sc_version(void);

/*
 * sc_release_workspace: hand the memory of the library's temporary buffers
 * back to the driver.  Those buffers (the NCHW repack of conv2d_fwd,
 * the partial results and split operands of cross_attention_fwd, and of
 * linear_fwd, the expanded codes of cross_attention_q8_fwd) come from a
 * library-private stream-ordered memory pool per device that otherwise keeps freed memory
 * for the next call.  Memory still in use by queued work is not affected.
 * Returns SC_OK.
 */
int sc_release_workspace(void);

/*
 * sc_set_autotune: first-call autotuning of conv2d_fwd's tile configuration
 * ("Optimizing Memory Efficiency for Convolution Kernels on Kepler GPUs",
 * Table 1: the best configuration differs per filter size and is found by
 * measurement).  With enable != 0, the first conv2d_fwd (NHWC or NCHW, or
 * conv2d_fwd_nchw_noalloc) of each shape with 3 x 3 filters and Cin > 1
 * times every candidate configuration of its output-channel class on the
 * caller's stream and data, which synchronises that stream once; the
 * fastest is cached per device and shape (N, H, W, Cin, Cout, R, S, act,
 * bias present) and used by later calls.  While the stream is being captured
 * into a CUDA graph no timing happens (the default configuration runs and
 * nothing is cached).  Off by default.  Returns the previous setting.
 */
int sc_set_autotune(int enable);

/* sc_autotune_lookup: the cached candidate index (0 = the default
 * configuration) for a shape on the current device, or -1 if not tuned. */
int sc_autotune_lookup(int N, int H, int W, int Cin, int Cout, int R, int S, int act, int has_bias);

/* sc_autotune_clear: forget every cached choice. */
void sc_autotune_clear(void);

/* sc_autotune_candidates: number of candidate configurations for a filter
 * shape (0 if not tuned); if names != NULL, their names, one per line, into
 * names[0 .. names_len-1] (NUL-terminated, truncated to fit). */
int sc_autotune_candidates(int Cin, int Cout, int R, int S, char *names, int names_len);

/*
 * sc_test_conv_candidate: test hook, not part of the operation.  Runs
 * conv2d_fwd (NHWC, 3 x 3) with candidate configuration `candidate` of
 * sc_autotune_candidates; SC_ERR_UNSUPPORTED if it does not exist or does
 * not apply to the shape.
 */
int sc_test_conv_candidate(const float *x, const float *w, const float *b, float *y,
                           int N, int H, int W, int Cin, int Cout, int R, int S,
                           int act, int candidate, sc_stream_t stream);

/*
 * sc_test_conv_wait_expiry: test hook for the device-status path, not part
 * of the operation.  Runs conv2d_fwd's TMA-staged kernel (NHWC, 3 x 3, no
 * activation, the default tile configuration for Cout) with copy
 * `drop_copy` (0-based, in each CTA's issue order) never issued, so the
 * time-bounded waits for it expire after `timeout_us` microseconds (a
 * CTA's consumers on the stage, then its producer on the stage's release).
 * The kernel then records SC_ERR_DEVICE_TIMEOUT (read and cleared by
 * sc_last_device_status), lets its other copies land and returns; the
 * context stays usable.  `y` is left partly written.  Cin % 4 == 0,
 * Cout % 4 == 0, 16-byte aligned x and y; SC_ERR_UNSUPPORTED where the
 * TMA kernel does not apply (a filter bank above its shared-memory limit).
 */
int sc_test_conv_wait_expiry(const float *x, const float *w, const float *b, float *y,
                             int N, int H, int W, int Cin, int Cout, int drop_copy, int timeout_us,
                             sc_stream_t stream);

/*
 * sc_test_stencil_wait_expiry: test hook for the device-status path, not
 * part of the operation.  Runs stencil_pipeline_fwd's TMA kernel with the
 * copy of row chunk `drop_copy` (0-based, per warp) never issued, so each
 * warp's time-bounded wait for it expires after `timeout_us` microseconds.
 * The kernel then records SC_ERR_DEVICE_TIMEOUT (read and cleared by
 * sc_last_device_status), waits for its other copies and returns; the
 * context stays usable.  `out` is left partly written.  Needs the TMA path's
 * conditions (W % 4 == 0, W >= 136, H >= 4, 16-byte aligned in and out),
 * else returns SC_ERR_UNSUPPORTED.
 */
int sc_test_stencil_wait_expiry(const float *in, float *out, int H, int W, int drop_copy,
                                int timeout_us, sc_stream_t stream);

/*
 * sc_test_attn_wait_expiry: test hook for the device-status path, not part
 * of the operation.  Runs cross_attention_fwd's tensor-core kernel (bf16,
 * packed, scale 1) with copy `drop_copy` (0-based, in each CTA's issue order)
 * never issued, so the time-bounded waits for it expire after `timeout_us`
 * microseconds.  The kernel then records SC_ERR_DEVICE_TIMEOUT (read and
 * cleared by sc_last_device_status), waits for its other copies and products
 * and returns; the context stays usable.  `out` is left with no defined
 * values.  With a drop_copy that no CTA reaches the waits that happen to take
 * longer than timeout_us expire, if any.
 */
int sc_test_attn_wait_expiry(const void *q, const void *k, const void *v, void *out, int N, int Tq, int Tk, int Hq,
                             int Hkv, int D, int drop_copy, int timeout_us, sc_stream_t stream);

/*
 * sc_test_attn_slow_clear: test hook, not part of the operation.  Runs
 * cross_attention_fwd's tensor-core kernel (packed, scale 1, whatever the
 * number of rows) with the warps that clear the value rows of states that are
 * not valid held up `delay_us` (0 to 1000) microseconds before each entry of
 * the ring.  The result is cross_attention_fwd's.  One of k_len and key_mask
 * is needed.
 */
int sc_test_attn_slow_clear(const void *q, const void *k, const void *v, void *out, const int *k_len,
                            const unsigned char *key_mask, int N, int Tq, int Tk, int Hq, int Hkv, int D, int dtype,
                            int delay_us, sc_stream_t stream);

/*
 * sc_test_attn_q8_wait_expiry: sc_test_attn_wait_expiry for
 * cross_attention_q8_fwd's tensor-core kernel (packed, scale 1, whatever the
 * number of rows).
 */
int sc_test_attn_q8_wait_expiry(const void *q, const void *k, const float *k_scale, const void *v, const float *v_scale,
                                void *out, int N, int Tq, int Tk, int Hq, int Hkv, int D, int block, int code, int dtype,
                                int drop_copy, int timeout_us, sc_stream_t stream);

/*
 * sc_test_attn_q8_rows_wait_expiry: the same for its kernel of few rows, with the
 * copies of step `drop_copy` (0-based, of each warp) never issued.  A warp whose wait
 * expires stops there.  With a drop_copy that no warp reaches the waits that
 * happen to take longer than timeout_us expire, if any.
 */
int sc_test_attn_q8_rows_wait_expiry(const void *q, const void *k, const float *k_scale, const void *v, const float *v_scale,
                                     void *out, int N, int Tq, int Tk, int Hq, int Hkv, int D, int block, int code, int dtype,
                                     int drop_copy, int timeout_us, sc_stream_t stream);

/*
 * sc_test_linear_wait_expiry: test hook for the device-status path, not part
 * of the operation.  Runs linear_fwd's tensor-core kernel (packed, no bias or
 * activation, residual or NULL, whatever the number of rows) with the copies of
 * stage `drop_copy` (0-based, in each CTA's issue order) never issued, so the
 * time-bounded waits for them expire after `timeout_us` microseconds.  The
 * kernel then records SC_ERR_DEVICE_TIMEOUT (read and cleared by
 * sc_last_device_status), waits for its other copies and products and returns;
 * the context stays usable.  `y` is left with no defined values.  With a drop_copy
 * that no CTA reaches the waits that happen to take longer than timeout_us expire,
 * if any.
 */
int sc_test_linear_wait_expiry(const void *x, const void *w, const void *residual, void *y, int rows, int Cin, int Cout,
                               int dtype, int drop_copy, int timeout_us, sc_stream_t stream);

/*
 * sc_test_workspace_allocs: test hook, not part of the operation.  The
 * number of temporary device buffers the library has taken from its memory
 * pool since it was loaded (conv2d_fwd with SC_NCHW takes one per call);
 * lets a test check that an entry point allocates nothing.
 */
long long sc_test_workspace_allocs(void);

/* Floats of device scratch behind conv2d_fwd_nchw_noalloc (32 MiB). */
#define SC_NOALLOC_SCRATCH_FLOATS (8u * 1024u * 1024u)

/*
 * conv2d_fwd_nchw_noalloc: conv2d_fwd with layout SC_NCHW, for callers that
 * must not allocate device memory while they run.  (The pages describe no
 * such entry point; it has no counterpart there.)
 *
 * conv2d_fwd with SC_NCHW and more than one channel repacks through a
 * temporary buffer it allocates on the stream.  Some callers cannot accept
 * that: a service that reserved the GPU's memory for its own pool at
 * start-up and treats any further allocation as a failure, or a per-frame
 * real-time pipeline that cannot risk an allocation's latency or an
 * out-of-memory error in the middle of a frame.  This entry point does the
 * same work (NCHW -> NHWC repack, convolution, NHWC -> NCHW repack) and calls
 * no cudaMalloc, cudaMallocAsync, cudaFree or other allocating routine.
 *
 * Its scratch is one array of SC_NOALLOC_SCRATCH_FLOATS floats in the
 * library's own device memory, present on every device that loads the
 * library until the process exits.  A call needs
 *   (Cin > 1 ? round_up(N*H*W*Cin, 64) : 0) + (Cout > 1 ? N*H*W*Cout : 0)
 * floats of it; a larger problem returns SC_ERR_SHAPE before any work.
 * The first call on a device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current: make that first call
 * before any stream capture starts.  All calls share the one array and
 * nothing is cleared between calls (every scratch element a call reads it
 * has written first), so calls whose GPU work overlaps in time (different
 * streams, or different host threads on one device) race on it and must be
 * ordered by the caller.
 * The device address is cached per device for the life of the process, so
 * a cudaDeviceReset (which unloads the library's device memory) while the
 * library is loaded is not supported.
 * Arguments, layout (x and y NCHW), supported shapes and status codes are
 * those of conv2d_fwd, checked by the same code; a failed CUDA call returns
 * SC_ERR_CUDA and records its error code for sc_last_cuda_error.
 */
int conv2d_fwd_nchw_noalloc(const float *x, const float *w, const float *b, float *y,
                            int N, int H, int W, int Cin, int Cout, int R, int S,
                            int act, sc_stream_t stream);

#if defined(__GNUC__)
#pragma GCC visibility pop
#endif

#ifdef __cplusplus
}
#endif

#endif /* STENCILCONV_H */
