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
// One token, 4096 -> 4096: 10 us with cold caches and the launch (3.9 us a call in a graph, the
// weights then in L2), floor 2.5; eight tokens 17: each row of x adds 16 bytes of shared memory
// read for every 32 of w.
//
// Rows of x that arrive as BF16 or FP32 are brought to 8 bits by every CTA for itself (amax,
// scale, q), between the issue of its first loads of w and their arrival: for a single row that
// costs less than a launch and a trip through memory.
#include "int8_internal.h"
#include "int8_rows.cuh"
#include "pointwise_math.cuh"

namespace convgb {

namespace {

constexpr int kFewThreads = 256;
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

// Largest magnitudes (bits) of the rows of x, over the CTA: every row at once, kFewWarps / M warps
// (one at least) to a row.  One barrier.
template <typename T, int M>
__device__ __forceinline__ void few_amax(const Int8Params& p, const T* x, uint32_t* top) {
    constexpr int V = 16 / sizeof(T);
    constexpr int kSegs = kFewWarps / M;  // M is 1, 2, 4 or 8
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int m = warp / kSegs, seg = warp - m * kSegs;
    float a = 0.0f;
    if (m < p.M) {
        const T* row = x + static_cast<long long>(m) * p.K;
        if (p.K % V == 0) {  // every row starts on 16 bytes
            using Io = VecIo<T, V>;
#pragma unroll 8
            for (int i = seg * 32 + lane; i < p.K / V; i += 32 * kSegs) {
                f2 f[V / 2];
                Io::unpack(__ldg(reinterpret_cast<const uint4*>(row) + i), f);
#pragma unroll
                for (int j = 0; j < V / 2; ++j) a = magnitude(a, f[j]);
            }
        } else {
            for (int i = seg * 32 + lane; i < p.K; i += 32 * kSegs) a = max_magnitude(a, few_load(row, i));
        }
    }
    const uint32_t bits = warp_max(magnitude_bits(a));
    if (lane == 0) top[warp] = bits;
    __syncthreads();
}

// Chunk [k0, k0 + kFewChunk) of the rows of x to shared memory as 8-bit values, zero from K up to
// the next multiple of 16.
template <typename T, int M>
__device__ __forceinline__ void few_stage(const Int8Params& p, const T* x, int k0, const RowScale (&rs)[M], uint8_t* sx) {
    const int len = min(kFewChunk, p.K - k0);
#pragma unroll
    for (int m = 0; m < M; ++m) {
        if (m >= p.M) break;
        const T* row = x + static_cast<long long>(m) * p.K + k0;
        uint8_t* dst = sx + m * kFewChunk;
        if constexpr (sizeof(T) == 1) {
            if (p.K % 16 == 0) {
#pragma unroll
                for (int i = threadIdx.x; i < kFewChunk / 16; i += kFewThreads)
                    if (i < len / 16) reinterpret_cast<uint4*>(dst)[i] = __ldg(reinterpret_cast<const uint4*>(row) + i);
            } else {
                for (int i = threadIdx.x; i < ((len + 15) & ~15); i += kFewThreads)
                    dst[i] = i < len ? static_cast<uint8_t>(row[i]) : 0;
            }
        } else {
            constexpr int V = 16 / sizeof(T);
            if (p.K % V == 0) {
                using Io = VecIo<T, V>;
#pragma unroll
                for (int i = threadIdx.x; i < kFewChunk / V; i += kFewThreads) {
                    if (i >= len / V) break;
                    f2 f[V / 2];
                    Io::unpack(__ldg(reinterpret_cast<const uint4*>(row) + i), f);
                    quantise_store<V>(reinterpret_cast<int8_t*>(dst) + i * V, f, row_factor(rs[m].inv));
                }
                if (threadIdx.x < 16 && (len & 15) > 0 && threadIdx.x >= (len & 15)) dst[(len & ~15) + threadIdx.x] = 0;
            } else {
                for (int i = threadIdx.x; i < ((len + 15) & ~15); i += kFewThreads)
                    dst[i] = i < len ? static_cast<uint8_t>(quantise1(few_load(row, i), row_factor(rs[m].inv))) : 0;
            }
        }
    }
}

// T: int8_t (x and its scales as given), __nv_bfloat16 or float (x brought to 8 bits here).
// M: rows of x a CTA holds (p.M <= M).
template <typename T, int M, bool ALIGNED>
__global__ void __launch_bounds__(kFewThreads) int8_few_rows_kernel(const Int8Params p, const T* x) {
    extern __shared__ __align__(16) uint8_t sx[];  // [M][kFewChunk]
    __shared__ uint32_t top[kFewWarps];
    const int lane = threadIdx.x & 31;
    const int n0 = (blockIdx.x * kFewWarps + (threadIdx.x >> 5)) * kFewRowsW;
    uint4 w[kFewRowsW][kFewLoads];
#pragma unroll
    for (int r = 0; r < kFewRowsW; ++r) load_w<ALIGNED>(p, n0 + r, 0, lane, w[r]);

    RowScale rs[M];
    if constexpr (sizeof(T) > 1) few_amax<T, M>(p, x, top);
#pragma unroll
    for (int m = 0; m < M; ++m) {
        if constexpr (sizeof(T) == 1) {
            rs[m] = {m < p.M ? __ldg(p.x_scale + m) : 0.0f, 0.0f};
        } else {
            uint32_t a = 0;
#pragma unroll
            for (int i = 0; i < kFewWarps / M; ++i) a = max(a, top[m * (kFewWarps / M) + i]);
            rs[m] = row_scale(a);
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
        few_stage<T, M>(p, x, k0, rs, sx);
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
                float v = fmaf(static_cast<float>(sum) * rs[m].scale, __ldg(p.w_scale + n), p.bias ? __ldg(p.bias + n) : 0.0f);
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

cudaError_t launch_int8_few(const Int8Params& p, cudaStream_t stream) { return launch_few<int8_t>(p, p.x, stream); }

cudaError_t launch_int8_few_quantize(const Int8Params& p, const void* x, bool bf16, cudaStream_t stream) {
    if (bf16) return launch_few<__nv_bfloat16>(p, static_cast<const __nv_bfloat16*>(x), stream);
    return launch_few<float>(p, static_cast<const float*>(x), stream);
}

}  // namespace convgb
