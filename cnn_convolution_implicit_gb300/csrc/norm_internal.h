// norm_internal.h -- parameter block and launchers shared between the group
// norm's plan code (norm_api.cu) and its kernels (group_norm.cu).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "conv_internal.h"

namespace convgb {

constexpr int kNormThreads = 256;

// Group norm over [N][P][C] (P = H * W pixels), G groups of cpg = C / G channels.
struct NormParams {
    int N, P, C, G, cpg;
    float eps;
    int act;      // conv_act
    int bf16;     // element type of x, y, dy, dx (else FP32)
    int vec;      // elements per access: 16 bytes where every pixel starts on 16 bytes, else 1
    int splits;   // pixel ranges per image of the streaming sums
    const void* x;
    const void* dy;
    const float* gamma;  // nullptr: 1
    const float* beta;   // nullptr: 0
    void* y;             // y, or dx in the backward pass
    int8_t* q;           // 8-bit output [N*P][C]
    float* scale;        // its row scales [N*P]
    float* mean;         // [N][G] (read by the backward pass)
    float* rstd;         // [N][G]
    float* dgamma;       // [C]
    float* dbeta;        // [C]
    float2* part;        // workspace [N][splits][C]
    float2* ab;          // workspace [N][G] (backward)
};

size_t norm_workspace_bytes(const NormParams& p);
cudaError_t launch_norm_forward(const NormParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_norm_backward(const NormParams& p, int num_sms, cudaStream_t stream);

}  // namespace convgb
