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
    int vec;      // elements per access: the most, up to 16 bytes, that divide the channels
    int splits;   // pixel ranges per image, or the CTAs of a resident cluster
    int two_pass; // two passes over pixel ranges (else, without a chunk, by channel)
    int joined;   // two passes: a kernel between them joins the ranges
    // resident form (0 chunk: another): a cluster of `splits` CTAs holds `chunk` channels of an image
    int chunk;
    int items;       // 16-byte vectors a thread holds of each tensor
    int smem_bytes;
    int smem_optin;  // what the device lets a block have
    int pix_base, pix_more;  // pixels of a CTA of the cluster or of a range, and how many have one more
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
    float2* ab;          // workspace [N][G] or, in two passes, [N][G][splits] (backward)
};

constexpr int kResMaxCluster = 16;

enum NormMode { kNormForward = 0, kNormInt8 = 1, kNormBackward = 2 };

// Threads of a resident CTA: two CTAs an SM leave each thread 128 registers (76 to 127 are used).
constexpr int kResThreads = 256;

size_t norm_workspace_bytes(const NormParams& p);
size_t norm_part_entries(const NormParams& p);
size_t norm_ab_entries(const NormParams& p);
void norm_pick_two_pass(NormParams& p, int mode, int num_sms);
// Fills the resident form's fields for a mode, or leaves chunk 0 where it does not fit.
void norm_pick_resident(NormParams& p, int mode, int num_sms);
// Clusters of that shape that the device runs at a time, 0 where it runs none (called once per plan,
// with its device current).
int norm_resident_at_a_time(const NormParams& p, int mode, int num_sms);
bool norm_resident_pays(const NormParams& p, int mode, int at_a_time, int num_sms);
cudaError_t launch_norm_forward(const NormParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_norm_backward(const NormParams& p, cudaStream_t stream);

}  // namespace convgb
