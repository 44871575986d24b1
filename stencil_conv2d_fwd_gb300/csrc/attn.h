// Internal interface of the attention operators: arguments after validation
// (attn_api.cu) and the launchers of the kernel translation units.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace sc {

constexpr int kAttnMaxD = 128;   // head width

// Element strides of a [N][T][H][D] tensor whose D elements are contiguous.
struct HeadStrides {
    long long n, t, h;
};

struct AttnArgs {
    const void *q, *k, *v;
    void *out;
    float *lse;                     // [N][Hq][Tq] or nullptr
    const int *k_len;               // [N] or nullptr
    const unsigned char *key_mask;  // [N][Tk] or nullptr
    int N, Tq, Tk, Hq, Hkv, D;
    int G;                          // query heads per key head
    float scale;
    HeadStrides qs, ks, vs, os;
};

// A row of the joint (token, head of the group) axis of one (sequence, key
// head): row = t * G + g.  A partial result of a row over part of the keys:
// m (running maximum, in units of log2), l (sum of 2^(s - m)) and o[D]
// (sum of 2^(s - m) v).  Partials of one row are part_stride rows apart.
struct AttnPartials {
    float *o;     // [parts][N * Hkv][rows][D]
    float2 *ml;   // [parts][N * Hkv][rows]
    int parts;
};

// Few rows per key head: keys streamed through warp-wide MMAs
// (attn_mma.cu).
cudaError_t launch_attn_mma(const AttnArgs &a, bool bf16, cudaStream_t st);
// Up to three fp32 rows per key head: keys streamed through registers
// (attn_rows.cu).
cudaError_t launch_attn_rows(const AttnArgs &a, cudaStream_t st);
// Many rows per key head: tensor cores (attn_tc.cu).
// drop_copy >= 0 leaves that ring entry of every CTA un-issued so that its
// bounded wait expires (tests of the device-status path); timeout_ns bounds
// each wait; clear_delay_ns holds the warps that clear value rows up before
// each entry (tests of the ring's order).
struct TcTest {
    int drop_copy = -1;
    unsigned clear_delay_ns = 0;
    unsigned long long timeout_ns = 1000000000ull;
};
cudaError_t launch_attn_tc(const AttnArgs &a, bool bf16, cudaStream_t st, const TcTest &test = TcTest());
// Copies of q ([plane][N][Hkv][Tq][G][D]), k and v ([plane][N][Hkv][Tk][D]) for
// it: fp32 tensors as three bf16 planes, bf16 ones as one (attn_split.cu).
cudaError_t launch_attn_split(const AttnArgs &a, bool bf16, void *const (&planes)[3], cudaStream_t st);
// Joins partial results into out and lse (attn_join.cu).
cudaError_t launch_attn_join(const AttnArgs &a, bool bf16, const AttnPartials &p, cudaStream_t st);

// Norm and rotation of heads (rotary.cu).
struct NormHeads {
    const void *x;
    void *y;
    const float *weight;   // D or nullptr
    const int *pos;        // [axes][tokens]
    int tokens, heads;
    long long x_t, x_h, y_t, y_h;   // element strides: token, head
};
struct RotaryArgs {
    NormHeads part[2];     // part[1].tokens == 0: one tensor
    const float *table;    // [positions][rot / (2 axes)][2]: cos, sin
    int D, rot, positions, axes;
    bool interleaved, inverse, norm;
    float eps;
};
cudaError_t launch_rotary(const RotaryArgs &a, bool bf16, cudaStream_t st);

struct RotaryTableArgs {
    float *table;
    int positions, pairs, rule;
    double base, factor, original;
};
cudaError_t launch_rotary_table(const RotaryTableArgs &a, cudaStream_t st);

constexpr int kErrRange = -8;   // SC_ERR_RANGE of include/stencilconv.h

#if defined(__CUDACC__)
// 2^x of the special function unit (about 2 ulp; 0 for -inf).
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two floats -> two bf16 (to nearest even, at most bf16's largest finite
// value; NaN stays), `lo` at the lower address.
__device__ __forceinline__ uint32_t pack_bf16_finite(float lo, float hi)
{
    uint32_t y;
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Programmatic dependent launch: let the next kernel on the stream start its
// prologue / wait until the previous kernel's writes are visible.
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
#endif

}  // namespace sc
