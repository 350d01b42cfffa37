// linear_internal.h -- parameter block and launchers shared between the linear layer's plan code
// (linear_api.cu) and its kernels.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "conv_internal.h"

namespace convgb {

// out[m][n] = act(sum_k a(m, k) * b(n, k) + bias[n]) + residual[m][n]
struct ProductParams {
    int M, N, K;
    const __nv_bfloat16* a;  // a(m, k) = a[m * a_m + k * a_k]
    const __nv_bfloat16* b;
    long long a_m, a_k, b_n, b_k;
    const float* bias;            // nullptr: 0
    const __nv_bfloat16* r;       // nullptr: 0
    __nv_bfloat16* y;
    __nv_bfloat16* z;             // nullptr: not wanted
    int act;
};
cudaError_t launch_product(const ProductParams& p, cudaStream_t stream);

// u = dy * act'(z) in BF16, and its sums over the rows
struct LinearGradParams {
    int M, N;
    const __nv_bfloat16* dy;
    const __nv_bfloat16* z;
    __nv_bfloat16* u;  // nullptr: not wanted
    float* dbias;      // nullptr: not wanted
    int act;
};
cudaError_t launch_linear_grad(const LinearGradParams& p, cudaStream_t stream);

}  // namespace convgb
