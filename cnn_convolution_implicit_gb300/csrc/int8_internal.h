// int8_internal.h -- parameter block and launchers shared between the 8-bit
// product's plan code (int8_api.cu) and its kernels (int8_product.cu, quantize.cu).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "conv_internal.h"

namespace convgb {

struct Int8Params {
    int M, N, K;
    int out_bf16;  // y BF16 (else FP32)
    int act;       // conv_act
    const int8_t* x;
    const float* x_scale;
    const int8_t* w;
    const float* w_scale;
    const float* bias;  // nullptr: 0
    void* y;
    unsigned* status;
};
// Whether a product runs on the tensor cores (else, with few rows, on the CUDA cores).
bool int8_use_gemm(const Int8Params& p);
// Tensor-core kernel (int8_gemm.cu); whether its row and tile counts stay within 32 bits.
bool int8_gemm_fits(const Int8Params& p);
cudaError_t launch_int8_gemm(const Int8Params& p, int num_sms, cudaStream_t stream);
// Either, from 8-bit rows.
cudaError_t launch_int8_product(const Int8Params& p, int num_sms, cudaStream_t stream);
// Few rows, straight from BF16 or FP32 x.
cudaError_t launch_int8_few_quantize(const Int8Params& p, const void* x, bool bf16, cudaStream_t stream);

// Rows of x (BF16 or FP32) to 8 bits with one scale each.
cudaError_t launch_quantize_rows(const void* x, bool bf16, int M, int K, int8_t* q, float* scale, int num_sms,
                                 cudaStream_t stream);

}  // namespace convgb
