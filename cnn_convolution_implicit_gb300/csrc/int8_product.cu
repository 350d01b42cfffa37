// int8_product.cu -- product of 8-bit integers with a scale for each row and
// each output channel:
//
//   y[m][n] = act( x_scale[m] * w_scale[n] * sum_k x[m][k] * w[n][k] + bias[n] )
#include "int8_internal.h"
#include "pointwise_math.cuh"

namespace convgb {

namespace {

template <int ACT>
__global__ void int8_plain_kernel(const Int8Params p) {
    const int n = blockIdx.x * 32 + threadIdx.x;
    for (long long m = static_cast<long long>(blockIdx.y) * 8 + threadIdx.y; m < p.M; m += gridDim.y * 8LL) {
        if (n >= p.N) return;
        const int8_t* x = p.x + m * p.K;
        const int8_t* w = p.w + static_cast<long long>(n) * p.K;
        int acc = 0;
        for (int k = 0; k < p.K; ++k) acc += static_cast<int>(x[k]) * static_cast<int>(w[k]);
        float v = static_cast<float>(acc) * p.x_scale[m] * p.w_scale[n];
        if (p.bias) v += p.bias[n];
        v = activate<ACT>(v);
        const long long o = m * p.N + n;
        if (p.out_bf16) static_cast<__nv_bfloat16*>(p.y)[o] = __float2bfloat16_rn(v);
        else static_cast<float*>(p.y)[o] = v;
    }
}

}  // namespace

cudaError_t launch_int8_product(const Int8Params& p, int num_sms, cudaStream_t stream) {
    if (p.M > 8 && int8_gemm_fits(p)) return launch_int8_gemm(p, num_sms, stream);
    const int rows = (p.M + 7) / 8;
    const dim3 grid((p.N + 31) / 32, rows < 65535 ? rows : 65535), block(32, 8);
    if (p.act == CONV_ACT_RELU) int8_plain_kernel<CONV_ACT_RELU><<<grid, block, 0, stream>>>(p);
    else if (p.act == CONV_ACT_SILU) int8_plain_kernel<CONV_ACT_SILU><<<grid, block, 0, stream>>>(p);
    else int8_plain_kernel<CONV_ACT_NONE><<<grid, block, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace convgb
