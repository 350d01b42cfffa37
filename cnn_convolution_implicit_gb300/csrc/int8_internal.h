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
    const int8_t* x;  // rows x_pitch bytes apart
    const float* x_scale;
    const int8_t* w;  // rows w_pitch bytes apart
    int x_pitch, w_pitch;
    int splits;    // CTAs that share the K of a tile (tensor-core kernel)
    const float* w_scale;
    const float* bias;  // nullptr: 0
    void* y;
    unsigned* status;
};
// Whether a product runs in the tensor-core kernel of many rows, or in that of 5 to 64 (else on the CUDA
// cores).
bool int8_use_gemm(const Int8Params& p);
bool int8_use_mid(const Int8Params& p);
// The tile of the many-row kernel: rows of x and columns (256 x 256 on a pair of SMs), and CTAs that
// share its K.
struct Int8Tile {
    int rows, columns, splits;
};
Int8Tile int8_pick_tile(const Int8Params& p, int num_sms);
// Tensor-core kernel (int8_gemm.cu); whether its row and tile counts stay within 32 bits.
bool int8_gemm_fits(const Int8Params& p);
// Rows of x and w start on 16 bytes; after_layout: the kernel before it on the stream laid them out.
cudaError_t launch_int8_gemm(const Int8Params& p, int num_sms, bool after_layout, cudaStream_t stream);
// Rows of x and w (either may have none) to rows `pitch` bytes apart.
cudaError_t launch_int8_layout(const int8_t* x, int8_t* xr, long long x_rows, const int8_t* w, int8_t* wr, long long w_rows,
                               int K, int pitch, int num_sms, cudaStream_t stream);
// Few rows (dense), from 8-bit x or straight from BF16 or FP32 x.
cudaError_t launch_int8_few(const Int8Params& p, cudaStream_t stream);
// 5 to 64 rows of x; after_quantise: x and its scales come from launch_quantize_rows just before.
cudaError_t launch_int8_mid(const Int8Params& p, bool after_quantise, cudaStream_t stream);
cudaError_t launch_int8_few_quantize(const Int8Params& p, const void* x, bool bf16, cudaStream_t stream);

// Rows of x (BF16 or FP32) to 8 bits with one scale each; rows of q `pitch` bytes apart.
cudaError_t launch_quantize_rows(const void* x, bool bf16, int M, int K, int pitch, int8_t* q, float* scale, int num_sms,
                                 cudaStream_t stream);

}  // namespace convgb
