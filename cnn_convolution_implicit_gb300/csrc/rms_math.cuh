// rms_math.cuh -- what the kernels of the root-mean-square norm share.
#pragma once

#include "pointwise_math.cuh"
#include "ptx.cuh"

namespace convgb {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) v += __shfl_xor_sync(0xffffffffu, v, i);
    return v;
}

__device__ __forceinline__ float reciprocal_root(float sum, int C, float eps) {
    return __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, static_cast<float>(C)), eps));
}

// Streaming forms: kStreamWarps warps take rows from a ring in shared memory, several rows or one row of all of them at a
// time.
constexpr int kStreamWarps = 8, kStreamMaxStages = 8;

struct Stream {
    int stages, stage_bytes;
    int rows;  // of a stage
};

// Rows of a stage: one where all warps share it, else a multiple of those that they work on together (`at_once`), as many
// as 24 KB hold while the CTAs have two turns at least.
inline int stream_rows(int M, int at_once, int tensors, long long row_bytes, int ctas) {
    if (at_once == 1) return 1;
    long long times = 24 * 1024 / (at_once * tensors * row_bytes);
    const long long most = M / (2LL * at_once * ctas);
    if (times > most) times = most;
    return at_once * static_cast<int>(times < 1 ? 1 : (times > 16 ? 16 : times));
}

__device__ __forceinline__ void sync_consumers() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

}  // namespace convgb
