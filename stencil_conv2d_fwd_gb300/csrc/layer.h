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
// Few rows, and in fp32 few products (linear_rows.cu; layer_api.cu has the rule).
cudaError_t launch_linear_rows(const LinearArgs &a, bool bf16, cudaStream_t st);
// Others: tensor cores (linear_tc.cu).  drop_copy >= 0 leaves that stage's copies
// of every CTA un-issued so that the bounded wait for them expires (tests of the
// device-status path); timeout_ns bounds each wait.
struct LinearTest {
    int drop_copy = -1;
    unsigned long long timeout_ns = 1000000000ull;
};
cudaError_t launch_linear_tc(const LinearArgs &a, bool bf16, cudaStream_t st, const LinearTest &test = LinearTest());

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
// MMAs (attn_q8.cu).  test.drop_copy: that step of every warp.
cudaError_t launch_attn_q8(const AttnQ8Args &a, bool bf16, bool e4m3, cudaStream_t st, const TcTest &test = TcTest());

// Many rows per key head: the codes as bf16 in a workspace, and the tensor cores
// (attn_split.cu, attn_tc.cu).
cudaError_t launch_attn_tc_q8(const AttnQ8Args &a, bool bf16, bool e4m3, cudaStream_t st, const TcTest &test = TcTest());
// q ([plane][N][Hkv][Tq][G][D], as attn_split; nullptr: used as it lies), codes
// as bf16, the values of bf16 tensors as fp16 ([N][Hkv][Tk][D]), and the factors of 16 keys each ([N * Hkv][groups]).
cudaError_t launch_attn_expand(const AttnQ8Args &a, bool bf16, bool e4m3, void *q, void *k, void *v, float *k_factor, float *v_factor,
                               int groups, cudaStream_t st);

// Launches a kernel that may be set up while the stream's last one ends: it has to
// call pdl_wait before it touches global memory.
template <class... P, class... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, dim3 block, cudaStream_t st, int cluster, const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace sc
