// int8_product.cu -- the 8-bit product with few rows (tokens):
//
//   y[m][n] = act( x_scale[m] * w_scale[n] * sum_k x[m][k] * w[n][k] + bias[n] )
//
// Bound by reading w once: N * K bytes.  Every row of x of the call (up to 8) sits in
// shared memory, 8-bit; a warp takes two rows of w, each lane 16 bytes of each at a time
// (both rows' loads for a whole chunk of K under way before the first is used), and adds
// the products four at a time in 32-bit integers (dp4a), so the sum is exact for every K.
// Two rows of w share each read of x from shared memory.
//
// Rows of x that arrive as BF16 or FP32 are brought to 8 bits by every CTA for itself (amax,
// scale, q), between the issue of its first loads of w and their arrival: for a single row that
// costs less than a launch and a trip through memory.
#include "int8_internal.h"
#include "int8_rows.cuh"
#include "pointwise_math.cuh"

namespace convgb {

namespace {

constexpr int kFewThreads = 128;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewRowsW = 2;           // rows of w a warp takes
constexpr int kFewLoads = 8;           // 16-byte loads a lane has under way per row of w
constexpr int kFewChunk = kFewLoads * 32 * 16;  // K of one chunk: 4,096

template <bool ALIGNED>
__device__ __forceinline__ void load_w(const Int8Params& p, int n, int k0, int lane, uint4 (&w)[kFewLoads]) {
    const long long total = static_cast<long long>(p.N) * p.K;
    const long long row = static_cast<long long>(n) * p.K;
#pragma unroll
    for (int i = 0; i < kFewLoads; ++i) {
        const int k = k0 + (i * 32 + lane) * 16;
        w[i] = make_uint4(0, 0, 0, 0);
        if (n < p.N && k < p.K) {
            if constexpr (ALIGNED) w[i] = __ldg(reinterpret_cast<const uint4*>(p.w + row + k));
            else w[i] = load_item(p.w, row + k, p.K - k < 16 ? p.K - k : 16, total);
        }
    }
}

__device__ __forceinline__ float few_load(const float* x, long long i) { return x[i]; }
__device__ __forceinline__ float few_load(const __nv_bfloat16* x, long long i) { return __bfloat162float(x[i]); }
__device__ __forceinline__ float few_load(const int8_t*, long long) { return 0.0f; }

__device__ __forceinline__ void few_load4(const float* x, float (&f)[4]) {
    VecIo<float, 4>::unpack(__ldg(reinterpret_cast<const uint4*>(x)), f);
}
__device__ __forceinline__ void few_load4(const __nv_bfloat16* x, float (&f)[4]) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(x));
    f[0] = __uint_as_float(v.x << 16);
    f[1] = __uint_as_float(v.x & 0xffff0000u);
    f[2] = __uint_as_float(v.y << 16);
    f[3] = __uint_as_float(v.y & 0xffff0000u);
}

// Largest magnitude (bits) of row m of x, over the CTA.
template <typename T>
__device__ __forceinline__ uint32_t few_amax(const T* x, int K, bool vec, uint32_t* scratch) {
    uint32_t a = 0;
    constexpr int V = 16 / sizeof(T);
    if (vec) {
        using Io = VecIo<T, V>;
        for (int i = threadIdx.x; i < K / V; i += kFewThreads) {
            float f[V];
            Io::unpack(__ldg(reinterpret_cast<const uint4*>(x) + i), f);
#pragma unroll
            for (int j = 0; j < V; ++j) a = max(a, magnitude_bits(f[j]));
        }
    } else {
        for (int i = threadIdx.x; i < K; i += kFewThreads) a = max(a, magnitude_bits(few_load(x, i)));
    }
    a = warp_max(a);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = a;
    __syncthreads();
    a = 0;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) a = max(a, scratch[w]);
    __syncthreads();
    return a;
}

// Chunk [k0, k0 + kFewChunk) of M rows of x to shared memory as 8-bit values, zero past K.
template <typename T, int M>
__device__ __forceinline__ void few_stage(const Int8Params& p, const T* x, int rows, int k0, const float (&inv)[M],
                                          uint8_t* sx) {
    const int words = min(kFewChunk, (p.K - k0 + 15) & ~15) / 4;
    for (int m = 0; m < rows; ++m) {
        const long long row = static_cast<long long>(m) * p.K + k0;
        for (int i = threadIdx.x; i < words; i += kFewThreads) {
            uint32_t v = 0;
            const int k = k0 + 4 * i;
            if constexpr (sizeof(T) == 1) {
                if (k + 4 <= p.K && ((row + 4 * i) & 3) == 0) v = *reinterpret_cast<const uint32_t*>(x + row + 4 * i);
                else
                    for (int j = 0; j < 4; ++j)
                        if (k + j < p.K) v |= static_cast<uint32_t>(static_cast<uint8_t>(x[row + 4 * i + j])) << (8 * j);
            } else {
                float f[4];
                if (p.K % 4 == 0 && k < p.K) {  // every row starts on four elements
                    few_load4(x + row + 4 * i, f);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) f[j] = k + j < p.K ? few_load(x, row + 4 * i + j) : 0.0f;
                }
                int q[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) q[j] = quantise(f[j], inv[m]);
                v = pack_int8x4(q[0], q[1], q[2], q[3]);
            }
            reinterpret_cast<uint32_t*>(sx + m * kFewChunk)[i] = v;
        }
    }
}

// T: int8_t (x and its scales as given), __nv_bfloat16 or float (x brought to 8 bits here).
// M: rows of x a CTA holds (p.M <= M).
template <typename T, int M, bool ALIGNED>
__global__ void __launch_bounds__(kFewThreads) int8_few_rows_kernel(const Int8Params p, const T* x) {
    extern __shared__ __align__(16) uint8_t sx[];  // [M][kFewChunk]
    __shared__ uint32_t scratch[kFewWarps];
    const int lane = threadIdx.x & 31;
    const int n0 = (blockIdx.x * kFewWarps + (threadIdx.x >> 5)) * kFewRowsW;
    uint4 w[kFewRowsW][kFewLoads];
#pragma unroll
    for (int r = 0; r < kFewRowsW; ++r) load_w<ALIGNED>(p, n0 + r, 0, lane, w[r]);

    float inv[M], scale[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        inv[m] = scale[m] = 0.0f;
        if (m >= p.M) continue;
        if constexpr (sizeof(T) == 1) {
            scale[m] = __ldg(p.x_scale + m);
        } else {
            const bool vec = p.K % (16 / sizeof(T)) == 0;
            const RowScale rs = row_scale(few_amax(x + static_cast<long long>(m) * p.K, p.K, vec, scratch));
            inv[m] = rs.inv;
            scale[m] = rs.scale;
        }
    }
    int acc[kFewRowsW][M];
#pragma unroll
    for (int r = 0; r < kFewRowsW; ++r)
#pragma unroll
        for (int m = 0; m < M; ++m) acc[r][m] = 0;

    for (int k0 = 0; k0 < p.K; k0 += kFewChunk) {
        if (k0 > 0) {
            __syncthreads();
#pragma unroll
            for (int r = 0; r < kFewRowsW; ++r) load_w<ALIGNED>(p, n0 + r, k0, lane, w[r]);
        }
        few_stage<T, M>(p, x, p.M, k0, inv, sx);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kFewLoads; ++i) {
            const int at = (i * 32 + lane) * 16;
            if (k0 + at >= p.K) break;
#pragma unroll
            for (int m = 0; m < M; ++m) {
                if (m >= p.M) break;
                const uint4 xv = *reinterpret_cast<const uint4*>(sx + m * kFewChunk + at);
#pragma unroll
                for (int r = 0; r < kFewRowsW; ++r) {
                    acc[r][m] = __dp4a(static_cast<int>(xv.x), static_cast<int>(w[r][i].x), acc[r][m]);
                    acc[r][m] = __dp4a(static_cast<int>(xv.y), static_cast<int>(w[r][i].y), acc[r][m]);
                    acc[r][m] = __dp4a(static_cast<int>(xv.z), static_cast<int>(w[r][i].z), acc[r][m]);
                    acc[r][m] = __dp4a(static_cast<int>(xv.w), static_cast<int>(w[r][i].w), acc[r][m]);
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kFewRowsW; ++r)
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int sum = __reduce_add_sync(0xffffffffu, acc[r][m]);
            const int n = n0 + r;
            if (lane == m && m < p.M && n < p.N) {
                float v = fmaf(static_cast<float>(sum) * scale[m], __ldg(p.w_scale + n), p.bias ? __ldg(p.bias + n) : 0.0f);
                if (p.act == CONV_ACT_RELU) v = activate<CONV_ACT_RELU>(v);
                else if (p.act == CONV_ACT_SILU) v = activate<CONV_ACT_SILU>(v);
                const long long o = static_cast<long long>(m) * p.N + n;
                if (p.out_bf16) static_cast<__nv_bfloat16*>(p.y)[o] = __float2bfloat16_rn(v);
                else static_cast<float*>(p.y)[o] = v;
            }
        }
}

template <typename T, int M>
cudaError_t launch_few(const Int8Params& p, const T* x, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>((static_cast<long long>(p.N) + kFewWarps * kFewRowsW - 1) / (kFewWarps * kFewRowsW));
    const int smem = M * kFewChunk;  // 32 KB at most
    if (p.K % 16 == 0) int8_few_rows_kernel<T, M, true><<<grid, kFewThreads, smem, stream>>>(p, x);
    else int8_few_rows_kernel<T, M, false><<<grid, kFewThreads, smem, stream>>>(p, x);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_few(const Int8Params& p, const T* x, cudaStream_t stream) {
    if (p.M == 1) return launch_few<T, 1>(p, x, stream);
    if (p.M == 2) return launch_few<T, 2>(p, x, stream);
    if (p.M <= 4) return launch_few<T, 4>(p, x, stream);
    return launch_few<T, 8>(p, x, stream);
}

}  // namespace

bool int8_use_gemm(const Int8Params& p) { return p.M > 8; }

cudaError_t launch_int8_product(const Int8Params& p, int num_sms, cudaStream_t stream) {
    if (int8_use_gemm(p)) return launch_int8_gemm(p, num_sms, stream);
    return launch_few<int8_t>(p, p.x, stream);
}

cudaError_t launch_int8_few_quantize(const Int8Params& p, const void* x, bool bf16, cudaStream_t stream) {
    if (bf16) return launch_few<__nv_bfloat16>(p, static_cast<const __nv_bfloat16*>(x), stream);
    return launch_few<float>(p, static_cast<const float*>(x), stream);
}

}  // namespace convgb
