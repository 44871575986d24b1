// y = act(x w^T + b) + residual, tiles of 64 x 64 in fp32 FMA.
#include <cuda_bf16.h>

#include "layer.h"
#include "linear.cuh"

namespace sc {

namespace {

template <class T>
__global__ void __launch_bounds__(256) linear_kernel(const LinearArgs a)
{
    __shared__ float xs[16][65], ws[16][65];
    const long long row0 = (long long)blockIdx.y * 64, col0 = (long long)blockIdx.x * 64;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < a.Cin; k0 += 16) {
        for (int e = threadIdx.x; e < 64 * 16; e += 256) {
            const int k = e % 16, r = e / 16;
            xs[k][r] = row0 + r < a.rows && k0 + k < a.Cin ? (float)static_cast<const T *>(a.x)[(row0 + r) * a.xs + k0 + k] : 0.f;
            ws[k][r] = col0 + r < a.Cout && k0 + k < a.Cin ? (float)static_cast<const T *>(a.w)[(col0 + r) * a.ws + k0 + k] : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[k][ty + 16 * i], ws[k][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const long long r = row0 + ty + 16 * i, c = col0 + tx + 16 * j;
            if (r >= a.rows || c >= a.Cout) continue;
            float v = activate(acc[i][j] + (a.b ? a.b[c] : 0.f), a.act);
            if (a.residual) v += (float)static_cast<const T *>(a.residual)[r * a.rs + c];
            static_cast<T *>(a.y)[r * a.ys + c] = (T)v;
        }
}

}  // namespace

cudaError_t launch_linear_rows(const LinearArgs &a, bool bf16, cudaStream_t st)
{
    const long long x = ((long long)a.Cout + 63) / 64, y = ((long long)a.rows + 63) / 64;
    if (y > 65535) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)x, (unsigned)y);
    if (bf16)
        linear_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a);
    else
        linear_kernel<float><<<grid, 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace sc
