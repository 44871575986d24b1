// Internal interface of the decoder layer's operators: arguments after
// validation (layer_api.cu) and the launchers of the kernel translation units.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "attn.h"

namespace sc {

// y[i][o] = act(sum_c x[i][c] w[o][c] + b[o]) + residual[i][o]
struct LinearArgs {
    const void *x, *w;
    const float *b;         // or nullptr
    const void *residual;   // or nullptr
    void *y;
    int rows, Cin, Cout, act;
    long long xs, ws, ys, rs;   // row strides in elements
};
cudaError_t launch_linear(const LinearArgs &a, bool bf16, cudaStream_t st);

// One norm: kind as sc_norm_kind.
struct NormArgs {
    int kind;
    float eps;
    const float *weight, *bias;   // or nullptr
};
struct ResidualNormArgs {
    const void *x, *residual;   // residual or nullptr
    void *sum, *y;              // one of them may be nullptr
    const float *gate;          // or nullptr
    int rows, C, gate_rows;
    float scale;
    NormArgs post, pre;
    long long xs, rs, ss, ys;   // row strides in elements
};
constexpr int kNormMaxC = 16384;
cudaError_t launch_residual_norm(const ResidualNormArgs &a, bool bf16, cudaStream_t st);

struct QuantPart {
    const void *x;
    unsigned char *codes;
    float *scale;   // [N][H][blocks]
    HeadStrides xs, cs;
};
struct QuantArgs {
    QuantPart part[2];
    int parts;
    const int *k_len;
    const unsigned char *key_mask;
    int N, T, H, D, block, blocks;
};
cudaError_t launch_kv_quantize(const QuantArgs &a, bool bf16, bool e4m3, cudaStream_t st);

// k and v of AttnArgs are codes; ks and vs count bytes.
struct AttnQ8Args : AttnArgs {
    const float *k_scale, *v_scale;   // [N][Hkv][blocks]
    int block, log2_block, blocks;
};
// Rows in blocks of up to 16, each of which streams the codes through warp-wide
// MMAs (attn_q8.cu).
cudaError_t launch_attn_q8(const AttnQ8Args &a, bool bf16, bool e4m3, cudaStream_t st);

}  // namespace sc
