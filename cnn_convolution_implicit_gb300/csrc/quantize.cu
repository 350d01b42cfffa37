// quantize.cu -- rows of FP32 or BF16 values to 8-bit integers with one scale
// per row: scale = amax / 127, q = rint(x * (127 / amax)).
//
// One warp per row, two sweeps (the row's largest magnitude, then the values); the
// second finds a row of ordinary length in L1.  Bound by the bytes of x read and q
// written.
#include "int8_internal.h"
#include "pointwise_math.cuh"

namespace convgb {

namespace {

constexpr int kQuantThreads = 256;

// VEC = 16 bytes of T (rows that all start on 16 bytes) or 1.
template <typename T, int VEC>
__global__ void __launch_bounds__(kQuantThreads) quantize_rows_kernel(const T* x, int M, int K, int pitch,
                                                                      int8_t* q, float* scale) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the product that may follow
    const int lane = threadIdx.x & 31;
    const int vecs = K / VEC;
    using Io = VecIo<T, VEC>;
    for (long long row = static_cast<long long>(blockIdx.x) * (kQuantThreads / 32) + (threadIdx.x >> 5); row < M;
         row += static_cast<long long>(gridDim.x) * (kQuantThreads / 32)) {
        const auto* src = reinterpret_cast<const typename Io::Raw*>(x) + row * vecs;
        constexpr int H = (VEC + 1) / 2;
        float top = 0.0f;
#pragma unroll 4
        for (int v = lane; v < vecs; v += 32) {
            f2 f[H];
            Io::unpack(src[v], f);
#pragma unroll
            for (int i = 0; i < H; ++i) top = magnitude(top, f[i]);
        }
        const RowScale rs = row_scale(warp_max(magnitude_bits(top)));
        if (lane == 0) scale[row] = rs.scale;
        int8_t* dst = q + row * pitch;
#pragma unroll 4
        for (int v = lane; v < vecs; v += 32) {
            f2 f[H];
            Io::unpack(src[v], f);
            quantise_store<VEC>(dst + v * VEC, f, rs);
        }
    }
}

}  // namespace

cudaError_t launch_quantize_rows(const void* x, bool bf16, int M, int K, int pitch, int8_t* q, float* scale, int num_sms,
                                 cudaStream_t stream) {
    const long long need = (static_cast<long long>(M) + kQuantThreads / 32 - 1) / (kQuantThreads / 32);
    const unsigned grid = static_cast<unsigned>(need < 8LL * num_sms ? need : 8LL * num_sms);
    if (bf16) {
        const auto* b = static_cast<const __nv_bfloat16*>(x);
        if (K % 8 == 0) quantize_rows_kernel<__nv_bfloat16, 8><<<grid, kQuantThreads, 0, stream>>>(b, M, K, pitch, q, scale);
        else quantize_rows_kernel<__nv_bfloat16, 1><<<grid, kQuantThreads, 0, stream>>>(b, M, K, pitch, q, scale);
    } else {
        const auto* f = static_cast<const float*>(x);
        if (K % 4 == 0) quantize_rows_kernel<float, 4><<<grid, kQuantThreads, 0, stream>>>(f, M, K, pitch, q, scale);
        else quantize_rows_kernel<float, 1><<<grid, kQuantThreads, 0, stream>>>(f, M, K, pitch, q, scale);
    }
    return cudaGetLastError();
}

}  // namespace convgb
