// linear_internal.h -- parameter blocks and launchers shared between the linear layer's plan code
// (linear_api.cu) and its kernels (linear_gemm.cu, linear_few.cu, column_sums.cu).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "conv_internal.h"

namespace convgb {

// y[m][n] = act(sum_k a(m, k) * b(n, k) + bias[n]) + r[m][n].  An operand is a matrix of rows `pitch` elements
// apart: [m][k], or with *_by_k [k][m].
struct GemmParams {
    int M, N, K;
    const __nv_bfloat16* a;
    const __nv_bfloat16* b;
    int a_pitch, b_pitch;
    bool a_by_k, b_by_k;
    int act;              // conv_act
    const float* bias;    // nullptr: 0
    const __nv_bfloat16* r;  // nullptr: 0
    __nv_bfloat16* y;
    __nv_bfloat16* z;     // nullptr: not wanted
    float* part;          // workspace of parts of K: [splits][M][N rounded up to 4]
    unsigned* status;
};

// The tile of the tensor-core kernel: rows and columns (256 x 256 on a pair of SMs), and how many units share
// its K, for each product of a launch.
struct GemmTile {
    int rows, columns, splits[2];
};
struct GemmSize {
    int M, N, K;
};
GemmTile gemm_pick_tile(const GemmSize* products, int count, bool forward, int num_sms);  // count: 1 (forward) or 2
bool gemm_joins_in_cluster(const GemmTile& t);  // of the forward product: its parts take no workspace
size_t gemm_part_bytes(int splits, int M, int N);
bool gemm_fits(int M, int N);  // tile counts within 32 bits

// Sums over the rows that the kernel before a launch left in parts: added on the side (launch_join_columns' order).
struct ColumnJoin {
    const float* part;
    float* out;  // nullptr: none
    int parts, columns;
};
// One or two products of the same N in a launch.  Rows of their operands start on 16 bytes.  after_other: the kernel before it on the
// stream wrote an operand and lets this one start early.
cudaError_t launch_gemm(const GemmParams* p, int count, const GemmTile& t, const ColumnJoin& join, int num_sms, bool after_other,
                        cudaStream_t stream);

// The forward product with few rows: dense operands, rows anywhere.
struct FewParams {
    int M, N, K;
    const __nv_bfloat16* x;
    const __nv_bfloat16* w;
    const float* bias;
    const __nv_bfloat16* r;
    __nv_bfloat16* y;
    __nv_bfloat16* z;
    int act;
};
bool linear_use_few(int M, int N, int K);
cudaError_t launch_linear_few(const FewParams& p, cudaStream_t stream);

// u = dy * act'(z) in BF16, and its sums over the rows
struct LinearGradParams {
    int M, N;
    const __nv_bfloat16* dy;
    const __nv_bfloat16* z;
    __nv_bfloat16* u;  // rows u_pitch elements apart; nullptr: not wanted
    int u_pitch;
    float* dbias;      // nullptr: not wanted
    float* part;       // workspace: [parts][N], where there is more than one
    int act;
};
int linear_grad_parts(int M, int N, int num_sms);
// join: the parts too; else dbias is complete only where linear_grad_parts is 1.
cudaError_t launch_linear_grad(const LinearGradParams& p, int num_sms, bool join, cudaStream_t stream);

}  // namespace convgb
