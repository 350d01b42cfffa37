// quantize.cu -- rows of FP32 or BF16 values to 8-bit integers with one scale
// per row: scale = amax / 127, q = rint(x * (127 / amax)).
//
// Bound by the bytes of x read and q written.  One warp per row: a row of at most sixteen 16-byte
// vectors a lane (8 KB) stays in registers, and a warp takes several short ones at a time, so
// that a lane has about four loads or more under way (200704 rows of 256 BF16: 40 us one row at
// a time, 31 us four, 73 % of the memory's rate; 8192 of 4096 25 us, 59 %; the divisions of a row's
// scale are shared out too).
// Longer rows take two sweeps, the largest magnitude, then the values; the second finds a row of
// ordinary length in L1.  Rows that do not start on 16 bytes are read as the aligned granules that hold
// them, shifted (19676 rows of 4090 BF16 in a product to 16 columns: 177 us, 124 so).
#include "int8_internal.h"
#include "int8_rows.cuh"
#include "pointwise_math.cuh"

namespace convgb {

namespace {

constexpr int kQuantThreads = 256;

// Vector v (16 bytes) of a row of K elements, zero past the row; rows may start on any element
// (ALIGNED: every one starts on 16 bytes and holds whole vectors).
template <typename T, bool ALIGNED>
__device__ __forceinline__ uint4 row_vector(const T* x, long long row, int M, int K, int v) {
    constexpr int VEC = 16 / sizeof(T);
    if constexpr (ALIGNED) {
        return __ldcs(reinterpret_cast<const uint4*>(x) + row * (K / VEC) + v);
    } else {
        const int left = K - v * VEC;
        return load_item(reinterpret_cast<const int8_t*>(x), (row * K + static_cast<long long>(v) * VEC) * static_cast<int>(sizeof(T)),
                         (left < VEC ? left : VEC) * static_cast<int>(sizeof(T)), static_cast<long long>(M) * K * static_cast<int>(sizeof(T)));
    }
}

// Its 8-bit values to a row of q; pitch: bytes from row to row.  Rows on whole vectors have room for
// one that runs past K.
template <typename T, bool ALIGNED>
__device__ __forceinline__ void row_store(int8_t* row, int K, int pitch, int v, uint4 raw, const RowFactor& r) {
    constexpr int VEC = 16 / sizeof(T);
    f2 f[VEC / 2];
    VecIo<T, VEC>::unpack(raw, f);
    int8_t* to = row + v * VEC;
    if (ALIGNED || pitch % VEC == 0) {
        quantise_store<VEC>(to, f, r);
        return;
    }
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
        const uint32_t u = quantise4(f[i / 2], f[i / 2 + 1], r);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (v * VEC + i + j < K) to[i + j] = static_cast<int8_t>(u >> (8 * j));
    }
}

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kQuantThreads) quantize_rows_kernel(const T* x, int M, int K, int pitch,
                                                                      int8_t* q, float* scale) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the product that may follow
    constexpr int VEC = 16 / sizeof(T), H = VEC / 2;
    const int lane = threadIdx.x & 31;
    const int vecs = (K + VEC - 1) / VEC;
    for (long long row = static_cast<long long>(blockIdx.x) * (kQuantThreads / 32) + (threadIdx.x >> 5); row < M;
         row += static_cast<long long>(gridDim.x) * (kQuantThreads / 32)) {
        float top = 0.0f;
#pragma unroll 4
        for (int v = lane; v < vecs; v += 32) {
            f2 f[H];
            VecIo<T, VEC>::unpack(row_vector<T, ALIGNED>(x, row, M, K, v), f);
#pragma unroll
            for (int i = 0; i < H; ++i) top = magnitude(top, f[i]);
        }
        const RowScale rs = row_scale(warp_max(magnitude_bits(top)));
        if (lane == 0) scale[row] = rs.scale;
        int8_t* dst = q + row * pitch;
#pragma unroll 4
        for (int v = lane; v < vecs; v += 32)
            row_store<T, ALIGNED>(dst, K, pitch, v, row_vector<T, ALIGNED>(x, row, M, K, v), row_factor(rs.inv));
    }
}

// Rows of at most 32 P vectors, in registers, R at a time.
template <typename T, int P, int R, bool ALIGNED>
__global__ void __launch_bounds__(kQuantThreads, P >= 16 ? 2 : (P >= 8 ? 3 : 4))
    quantize_short_rows_kernel(const T* x, int M, int K, int pitch, int8_t* q, float* scale) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the product that may follow
    constexpr int VEC = 16 / sizeof(T), H = VEC / 2;
    const int lane = threadIdx.x & 31;
    const int vecs = (K + VEC - 1) / VEC;
    for (long long row0 = (static_cast<long long>(blockIdx.x) * (kQuantThreads / 32) + (threadIdx.x >> 5)) * R; row0 < M;
         row0 += static_cast<long long>(gridDim.x) * (kQuantThreads / 32) * R) {
        uint4 raw[R][P];
        if constexpr (ALIGNED) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int h = 0; h < P; ++h) {
                    raw[r][h] = make_uint4(0, 0, 0, 0);
                    if (row0 + r < M && lane + 32 * h < vecs) raw[r][h] = row_vector<T, true>(x, row0 + r, M, K, lane + 32 * h);
                }
        } else {
            constexpr int es = sizeof(T);
            StraddlingRow<P> rows[R];
#pragma unroll
            for (int r = 0; r < R; ++r)  // a row past the last has no bytes
                rows[r].load(reinterpret_cast<const int8_t*>(x), (row0 + r) * K * es, row0 + r < M ? K * es : 0,
                             static_cast<long long>(M) * K * es, lane, raw[r]);
#pragma unroll
            for (int r = 0; r < R; ++r) rows[r].shift(lane, raw[r]);
        }
        uint32_t top[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float m = 0.0f;
#pragma unroll
            for (int h = 0; h < P; ++h) {
                f2 f[H];
                VecIo<T, VEC>::unpack(raw[r][h], f);
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
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (row0 + r >= M) break;
#pragma unroll
            for (int h = 0; h < P; ++h)
                if (lane + 32 * h < vecs) row_store<T, ALIGNED>(q + (row0 + r) * pitch, K, pitch, lane + 32 * h, raw[r][h], rf[r]);
        }
    }
}

template <typename T, bool ALIGNED>
cudaError_t launch_typed(const T* x, int M, int K, int pitch, int8_t* q, float* scale, int num_sms, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    const int vecs = (K + V - 1) / V;
    int parts = 1;  // vectors a lane keeps of a row
    while (parts < 16 && 32 * parts < vecs) parts *= 2;
    const bool in_registers = 32 * parts >= vecs;
    const long long rows = (kQuantThreads / 32) * (in_registers && parts <= 2 ? 4 / parts : 1);
    const long long need = (static_cast<long long>(M) + rows - 1) / rows;
    const unsigned grid = static_cast<unsigned>(need < 8LL * num_sms ? need : 8LL * num_sms);
    const auto run = [&](auto* kernel) { kernel<<<grid, kQuantThreads, 0, stream>>>(x, M, K, pitch, q, scale); };
    if (!in_registers) run(quantize_rows_kernel<T, ALIGNED>);
    else if (parts == 1) run(quantize_short_rows_kernel<T, 1, 4, ALIGNED>);
    else if (parts == 2) run(quantize_short_rows_kernel<T, 2, 2, ALIGNED>);
    else if (parts == 4) run(quantize_short_rows_kernel<T, 4, 1, ALIGNED>);
    else if (parts == 8) run(quantize_short_rows_kernel<T, 8, 1, ALIGNED>);
    else run(quantize_short_rows_kernel<T, 16, 1, ALIGNED>);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_rows(const T* x, int M, int K, int pitch, int8_t* q, float* scale, int num_sms, cudaStream_t stream) {
    if (K % (16 / sizeof(T)) == 0) return launch_typed<T, true>(x, M, K, pitch, q, scale, num_sms, stream);
    return launch_typed<T, false>(x, M, K, pitch, q, scale, num_sms, stream);
}

}  // namespace

cudaError_t launch_quantize_rows(const void* x, bool bf16, int M, int K, int pitch, int8_t* q, float* scale, int num_sms,
                                 cudaStream_t stream) {
    if (bf16) return launch_rows(static_cast<const __nv_bfloat16*>(x), M, K, pitch, q, scale, num_sms, stream);
    return launch_rows(static_cast<const float*>(x), M, K, pitch, q, scale, num_sms, stream);
}

}  // namespace convgb
