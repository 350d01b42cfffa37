// rows_internal.h -- parameter blocks and launchers shared between the C ABI of the row operators
// (rows_api.cu) and their kernels (rms_norm.cu, dropout.cu).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "conv_internal.h"

namespace convgb {

// Root-mean-square norm over [M][C].
struct RmsParams {
    int M, C;
    float eps;
    int bf16;            // element type (else FP32)
    const void* x;       // forward: x; backward: dy
    const void* r;       // forward: residual; backward: dh (nullptr: 0)
    const void* h_in;    // backward: the forward pass's h
    const float* gamma;  // nullptr: 1
    void* y;             // forward: y; backward: dx
    void* h;             // forward: x + residual, rounded (nullptr: not wanted)
    int8_t* q;           // 8-bit output, instead of y
    float* scale;        // its row scales
    float* rstd;         // forward: written where given; backward: read
    float* dgamma;       // nullptr: not wanted
    float* part;         // workspace: [parts][C] sums of dy * n
    int parts;           // rows of sums that the backward pass leaves there
    int ctas, rows;      // of the streaming forms: CTAs, and rows of a stage (backward)
    int rounds;          // of the backward pass with dgamma: rounds of CTAs
    unsigned* status;
};

// Fills parts, ctas, rows and rounds.
void rms_plan_backward(RmsParams& p, int num_sms);
cudaError_t launch_rms_forward(const RmsParams& p, cudaStream_t stream);
cudaError_t launch_rms_backward(const RmsParams& p, cudaStream_t stream);

// Rows off 16 bytes, up to 8,192 values (rms_elements.cu).
bool rms_by_elements(const RmsParams& p);
void rms_plan_elements(RmsParams& p);  // fills parts and rounds
cudaError_t launch_rms_elements(const RmsParams& p, bool backward, cudaStream_t stream);

// Sums of `parts` rows of C values each, in one order (column_sums.cu).  early: the kernel before it on the stream lets it
// start early.
cudaError_t launch_join_columns(const float* part, int parts, int C, float* out, bool early, cudaStream_t stream);

struct DropoutParams {
    const void* x;
    const void* r;  // nullptr: 0
    void* y;
    unsigned long long n;
    const unsigned long long* state;  // seed, offset
    uint32_t threshold;               // words below it drop
    float scale;                      // 1 / (1 - p)
    int none_left;                    // p = 1
    int bf16;
};

cudaError_t launch_dropout(const DropoutParams& p, int num_sms, cudaStream_t stream);

}  // namespace convgb
