// quantize.cu -- rows of FP32 or BF16 values to 8-bit integers with one scale
// per row: scale = amax / 127, q = rint(x * (127 / amax)).
//
// Bound by the bytes of x read and q written.  One warp per row: a row of at most sixteen 16-byte
// vectors a lane (8 KB) stays in registers, and a warp takes several short ones at a time, so
// that a lane has about four loads or more under way (200704 rows of 256 BF16: 40 us one row at
// a time, 27 us four; the divisions of a row's scale are shared out too).  Longer rows take two sweeps, the largest magnitude, then the
// values; the second finds a row of ordinary length in L1.
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
            quantise_store<VEC>(dst + v * VEC, f, row_factor(rs.inv));
        }
    }
}

// Rows of at most 32 P vectors, in registers, R at a time.
template <typename T, int P, int R>
__global__ void __launch_bounds__(kQuantThreads, P >= 16 ? 2 : (P >= 8 ? 3 : 4)) quantize_short_rows_kernel(const T* x, int M, int K, int pitch, int8_t* q,
                                                                               float* scale) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the product that may follow
    constexpr int VEC = 16 / sizeof(T), H = VEC / 2;
    using Io = VecIo<T, VEC>;
    const int lane = threadIdx.x & 31;
    const int vecs = K / VEC;
    for (long long row0 = (static_cast<long long>(blockIdx.x) * (kQuantThreads / 32) + (threadIdx.x >> 5)) * R; row0 < M;
         row0 += static_cast<long long>(gridDim.x) * (kQuantThreads / 32) * R) {
        uint4 raw[R][P];
        const uint4* src = reinterpret_cast<const uint4*>(x) + row0 * vecs + lane;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int h = 0; h < P; ++h) {
                raw[r][h] = make_uint4(0, 0, 0, 0);
                if (row0 + r < M && lane + 32 * h < vecs) raw[r][h] = __ldcs(src + r * vecs + 32 * h);
            }
        uint32_t top[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float m = 0.0f;
#pragma unroll
            for (int h = 0; h < P; ++h) {
                f2 f[H];
                Io::unpack(raw[r][h], f);
#pragma unroll
                for (int i = 0; i < H; ++i) m = magnitude(m, f[i]);
            }
            top[r] = magnitude_bits(m);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) top[r] = warp_max(top[r]);
        RowFactor rf[R];
        const float own = row_factors<R>(top, lane, 32, rf);
        if (lane < R && row0 + lane < M) scale[row0 + lane] = own;
        int8_t* dst = q + row0 * pitch + lane * VEC;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (row0 + r >= M) break;
#pragma unroll
            for (int h = 0; h < P; ++h)
                if (lane + 32 * h < vecs) {
                    f2 f[H];
                    Io::unpack(raw[r][h], f);
                    quantise_store<VEC>(dst + r * pitch + 32 * h * VEC, f, rf[r]);
                }
        }
    }
}

template <typename T>
cudaError_t launch_typed(const T* x, int M, int K, int pitch, int8_t* q, float* scale, int num_sms, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    const bool wide = K % V == 0;
    int parts = 1;  // vectors a lane keeps of a row
    while (parts < 16 && 32 * parts < K / V) parts *= 2;
    const bool in_registers = wide && 32 * parts >= K / V;
    const long long rows = (kQuantThreads / 32) * (in_registers && parts <= 2 ? 4 / parts : 1);
    const long long need = (static_cast<long long>(M) + rows - 1) / rows;
    const unsigned grid = static_cast<unsigned>(need < 8LL * num_sms ? need : 8LL * num_sms);
    if (in_registers && parts == 1) quantize_short_rows_kernel<T, 1, 4><<<grid, kQuantThreads, 0, stream>>>(x, M, K, pitch, q, scale);
    else if (in_registers && parts == 2) quantize_short_rows_kernel<T, 2, 2><<<grid, kQuantThreads, 0, stream>>>(x, M, K, pitch, q, scale);
    else if (in_registers && parts == 4) quantize_short_rows_kernel<T, 4, 1><<<grid, kQuantThreads, 0, stream>>>(x, M, K, pitch, q, scale);
    else if (in_registers && parts == 8) quantize_short_rows_kernel<T, 8, 1><<<grid, kQuantThreads, 0, stream>>>(x, M, K, pitch, q, scale);
    else if (in_registers) quantize_short_rows_kernel<T, 16, 1><<<grid, kQuantThreads, 0, stream>>>(x, M, K, pitch, q, scale);
    else if (wide) quantize_rows_kernel<T, V><<<grid, kQuantThreads, 0, stream>>>(x, M, K, pitch, q, scale);
    else quantize_rows_kernel<T, 1><<<grid, kQuantThreads, 0, stream>>>(x, M, K, pitch, q, scale);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_rows(const void* x, bool bf16, int M, int K, int pitch, int8_t* q, float* scale, int num_sms,
                                 cudaStream_t stream) {
    if (bf16) return launch_typed(static_cast<const __nv_bfloat16*>(x), M, K, pitch, q, scale, num_sms, stream);
    return launch_typed(static_cast<const float*>(x), M, K, pitch, q, scale, num_sms, stream);
}

}  // namespace convgb
