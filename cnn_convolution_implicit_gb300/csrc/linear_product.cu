// linear_product.cu -- the linear layer's products and the gradient of its activation.
#include "linear_internal.h"
#include "pointwise_math.cuh"

namespace convgb {

namespace {

constexpr int kTile = 64, kDepth = 16;

__device__ __forceinline__ float act_of(int act, float z) {
    if (act == CONV_ACT_RELU) return activate<CONV_ACT_RELU>(z);
    if (act == CONV_ACT_SILU) return activate<CONV_ACT_SILU>(z);
    return z;
}

// 64 x 64 outputs a CTA, 4 x 4 a thread, FP32 on the CUDA cores.
__global__ void __launch_bounds__(256) product_kernel(const ProductParams p) {
    __shared__ float a[kDepth][kTile + 1], b[kDepth][kTile + 1];
    const int m0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float sum[4][4] = {};
    for (int k0 = 0; k0 < p.K; k0 += kDepth) {
        for (int i = threadIdx.x; i < kTile * kDepth; i += 256) {
            const int r = i / kDepth, k = i % kDepth;
            a[k][r] = m0 + r < p.M && k0 + k < p.K ? __bfloat162float(p.a[(m0 + r) * p.a_m + (k0 + k) * p.a_k]) : 0.0f;
            b[k][r] = n0 + r < p.N && k0 + k < p.K ? __bfloat162float(p.b[(n0 + r) * p.b_n + (k0 + k) * p.b_k]) : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < kDepth; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) sum[i][j] = fmaf(a[k][ty + 16 * i], b[k][tx + 16 * j], sum[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m >= p.M || n >= p.N) continue;
            const long long o = static_cast<long long>(m) * p.N + n;
            const float z = sum[i][j] + (p.bias ? p.bias[n] : 0.0f);
            if (p.z) p.z[o] = __float2bfloat16_rn(z);
            // rounded by itself, so that y is the same with and without z
            p.y[o] = __float2bfloat16_rn(__fadd_rn(act_of(p.act, z), p.r ? __bfloat162float(p.r[o]) : 0.0f));
        }
}

__global__ void __launch_bounds__(256) grad_kernel(const LinearGradParams p) {
    __shared__ float sums[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = blockIdx.x * 32 + lane;
    float total = 0.0f;
    for (int m = warp; m < p.M && n < p.N; m += 8) {
        const long long o = static_cast<long long>(m) * p.N + n;
        float u = __bfloat162float(p.dy[o]);
        if (p.act == CONV_ACT_RELU) u = f2_lo(activate_grad2<CONV_ACT_RELU>(f2_dup(__bfloat162float(p.z[o])), f2_dup(u)));
        if (p.act == CONV_ACT_SILU) u = f2_lo(activate_grad2<CONV_ACT_SILU>(f2_dup(__bfloat162float(p.z[o])), f2_dup(u)));
        if (p.u) p.u[o] = __float2bfloat16_rn(u);
        total += u;
    }
    sums[warp][lane] = total;
    __syncthreads();
    if (warp == 0 && n < p.N && p.dbias) {
        float sum = 0.0f;
        for (int i = 0; i < 8; ++i) sum += sums[i][lane];
        p.dbias[n] = sum;
    }
}

}  // namespace

cudaError_t launch_product(const ProductParams& p, cudaStream_t stream) {
    product_kernel<<<dim3((p.N + kTile - 1) / kTile, (p.M + kTile - 1) / kTile), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_linear_grad(const LinearGradParams& p, cudaStream_t stream) {
    grad_kernel<<<(p.N + 31) / 32, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace convgb
