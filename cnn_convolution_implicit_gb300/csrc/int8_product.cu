// int8_product.cu -- the 8-bit product with few rows (tokens), up to 4 and up to 64:
//
//   y[m][n] = act( x_scale[m] * w_scale[n] * sum_k x[m][k] * w[n][k] + bias[n] )
//
// Bound by reading w once: N * K bytes.  Every row of x of the call (up to 4) sits in
// shared memory, 8-bit; a warp takes two rows of w, each lane 16 bytes of each at a time
// (both rows' loads for a whole chunk of K under way before the first is used), and adds
// the products four at a time in 32-bit integers (dp4a), so the sum is exact for every K.
// Two rows of w share each read of x from shared memory.
//
// One token, 4096 -> 4096: 11 us with cold caches and the launch (3.4 us a call in a graph, the
// weights then in L2), floor 2.5; four tokens 13 (5.7): each row of x adds 16 bytes of shared memory
// read for every 32 of w.  Past one chunk of K the next one's loads wait for the last use of this:
// 16384 -> 4096 21 us (8.0), floor 9.9.
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
    constexpr int kSegs = kFewWarps / M;  // M is 1, 2 or 4
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
    const int smem = M * kFewChunk;  // 16 KB at most
    if (p.K % 16 == 0) int8_few_rows_kernel<T, M, true><<<grid, kFewThreads, smem, stream>>>(p, x);
    else int8_few_rows_kernel<T, M, false><<<grid, kFewThreads, smem, stream>>>(p, x);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_few(const Int8Params& p, const T* x, cudaStream_t stream) {
    if (p.M == 1) return launch_few<T, 1>(p, x, stream);
    if (p.M == 2) return launch_few<T, 2>(p, x, stream);
    return launch_few<T, 4>(p, x, stream);
}

// ---------------------------------------------------------------- 5 to 64 rows
// Still bound by reading w once, but too many products for the CUDA cores: FP16 MMAs of 16 x 8 x 16
// on operands that go from memory to registers and from there to FP16, exact as in the
// tensor-core kernel of many rows, whose 128-row tiles, shared-memory stages and launch cost more
// than the bytes here: 16 x 4096 -> 4096 5.4 to 5.8 us a call in a graph against 14.9, 13 and 21 with cold caches
// and the launch (floor 2.5).
//
// A CTA takes 16 rows of w; its eight warps share K, 64 at a time.  Lane 4 g + q holds k = 16 q ..
// 16 q + 15 of rows g of w and g, g + 8 of x: the MMA sums over k in any order, so its slots
// (2 q, 2 q + 1, 2 q + 8, 2 q + 9) take the lane's four values of word j, for both operands alike.
// The warps' sums meet in shared memory in one order.
constexpr int kMidColumns = 16;

template <bool ALIGNED, bool LATE>
__device__ __forceinline__ uint4 mid_item(const int8_t* base, int row, int rows, int pitch, int k, int K) {
    if (row >= rows || k >= K) return make_uint4(0, 0, 0, 0);
    const long long at = static_cast<long long>(row) * pitch + k;
    if constexpr (ALIGNED) return load16<LATE>(reinterpret_cast<const uint4*>(base + at));
    else return load_item<LATE>(base, at, K - k < 16 ? K - k : 16, static_cast<long long>(rows) * pitch);
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int j) { return j == 0 ? v.x : (j == 1 ? v.y : (j == 2 ? v.z : v.w)); }

__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint2 a_lo, uint2 a_hi, uint2 b) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a_lo.x), "r"(a_hi.x), "r"(a_lo.y), "r"(a_hi.y), "r"(b.x), "r"(b.y));
}

// MT: 16-row tiles of x.
template <int MT, bool ALIGNED>
__global__ void __launch_bounds__(kFewThreads, 2) int8_mid_rows_kernel(const Int8Params p) {
    constexpr int B = 4, BX = MT == 1 ? 4 : (MT == 2 ? 2 : 1);  // steps of K whose loads of w and of x are under way
    constexpr int kStep = 64 * kFewWarps;
    __shared__ float2 parts[kFewWarps][MT * 16][kMidColumns / 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int n0 = blockIdx.x * kMidColumns;
    float acc[MT][2][4] = {};
    uint4 w[B][2];
    const auto load_weights = [&](int k0) {
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
            for (int t = 0; t < 2; ++t) w[b][t] = mid_item<ALIGNED, false>(p.w, n0 + 8 * t + g, p.N, p.w_pitch, k0 + b * kStep + 16 * q, p.K);
    };
    load_weights(64 * warp);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // x and its scales may come from the kernel before
    for (int k0 = 64 * warp; k0 < p.K; k0 += B * kStep) {
#pragma unroll
        for (int b0 = 0; b0 < B; b0 += BX) {
            if (b0 > 0 && k0 + b0 * kStep >= p.K) break;
            uint4 x[BX][MT][2];
#pragma unroll
            for (int b = 0; b < BX; ++b)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        x[b][m][h] = mid_item<ALIGNED, true>(p.x, 16 * m + 8 * h + g, p.M, p.x_pitch, k0 + (b0 + b) * kStep + 16 * q, p.K);
#pragma unroll
            for (int b = 0; b < BX; ++b)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint2 w0 = to_half4(word_of(w[b0 + b][0], j)), w1 = to_half4(word_of(w[b0 + b][1], j));
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const uint2 lo = to_half4(word_of(x[b][m][0], j)), hi = to_half4(word_of(x[b][m][1], j));
                        mma_16x8x16(acc[m][0], lo, hi, w0);
                        mma_16x8x16(acc[m][1], lo, hi, w1);
                    }
                }
        }
        if (k0 + B * kStep < p.K) load_weights(k0 + B * kStep);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            parts[warp][16 * m + g][4 * t + q] = make_float2(acc[m][t][0], acc[m][t][1]);
            parts[warp][16 * m + 8 + g][4 * t + q] = make_float2(acc[m][t][2], acc[m][t][3]);
        }
    __syncthreads();
#pragma unroll
    for (int i = threadIdx.x; i < MT * 16 * kMidColumns; i += kFewThreads) {
        const int m = i / kMidColumns, n = n0 + i % kMidColumns;
        if (m >= p.M || n >= p.N) continue;
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < kFewWarps; ++k) sum += reinterpret_cast<const float*>(parts[k][m])[i % kMidColumns];
        float v = fmaf(sum * load1_late(p.x_scale + m), __ldg(p.w_scale + n), p.bias ? __ldg(p.bias + n) : 0.0f);
        if (p.act == CONV_ACT_RELU) v = activate<CONV_ACT_RELU>(v);
        else if (p.act == CONV_ACT_SILU) v = activate<CONV_ACT_SILU>(v);
        const long long o = static_cast<long long>(m) * p.N + n;
        if (p.out_bf16) static_cast<__nv_bfloat16*>(p.y)[o] = __float2bfloat16_rn(v);
        else static_cast<float*>(p.y)[o] = v;
    }
}

}  // namespace

// This kernel and the tiles of many rows, 8-bit input, microseconds in a graph (cold caches and the launch):
//    5 x 4096 -> 4096 5.2 (13) and 15.2 (21)      16 x 512 -> 512 2.6 (7) and 7.2 (13)     32 x 8192 -> 8192 24.0 (40) and 34.7 (46)
//   48 x 4096 -> 4096 10.1 (17) and 15.5 (23)     48 x 4096 -> 8192 18.2 (28) and 22.1 (29)   48 x 4096 -> 16384 31.6 (47) and 32.4 (42)
//   64 x 1024 -> 1024 4.6 (11) and 8.6 (13)       64 x 4096 -> 4096 12.8 (21) and 15.6 (23)   64 x 4096 -> 16384 42.7 (62) and 32.6 (43)
// x is read again by every 16 columns, so with more rows and weights the tiles win, with cold caches first (56 x 8192 ->
// 2048 35 and 27 cold); the bounds lie on their side of where the two meet.
// This kernel and the CUDA cores': 1 x 4096 -> 4096 5.1 (13) and 3.4 (11), 2 rows 5.2 (13) and 4.1 (11), 4 rows
// 5.1 (13) and 5.7 (13), 4 x 16384 -> 4096 14.5 (25) and 14.3 (31); a BF16 row takes a launch more here.
bool int8_use_mid(const Int8Params& p) {
    const long long weights = static_cast<long long>(p.N) * p.K;
    return p.M > 4 && (p.M <= 32 || (p.M <= 48 && weights <= 1LL << 24) || (p.M <= 64 && weights <= 1LL << 21));
}
bool int8_use_gemm(const Int8Params& p) { return p.M > 4 && !int8_use_mid(p); }

cudaError_t launch_int8_mid(const Int8Params& p, bool after_quantise, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((static_cast<long long>(p.N) + kMidColumns - 1) / kMidColumns));
    cfg.blockDim = dim3(kFewThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // the first loads of w overlap the kernel before
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = after_quantise ? 1 : 0;
    const bool aligned = p.K % 16 == 0;  // of both operands, then
    const auto run = [&](auto* whole, auto* any) { return cudaLaunchKernelEx(&cfg, aligned ? whole : any, p); };
    if (p.M <= 16) return run(int8_mid_rows_kernel<1, true>, int8_mid_rows_kernel<1, false>);
    if (p.M <= 32) return run(int8_mid_rows_kernel<2, true>, int8_mid_rows_kernel<2, false>);
    if (p.M <= 48) return run(int8_mid_rows_kernel<3, true>, int8_mid_rows_kernel<3, false>);
    return run(int8_mid_rows_kernel<4, true>, int8_mid_rows_kernel<4, false>);
}

cudaError_t launch_int8_few(const Int8Params& p, cudaStream_t stream) { return launch_few<int8_t>(p, p.x, stream); }

cudaError_t launch_int8_few_quantize(const Int8Params& p, const void* x, bool bf16, cudaStream_t stream) {
    if (bf16) return launch_few<__nv_bfloat16>(p, static_cast<const __nv_bfloat16*>(x), stream);
    return launch_few<float>(p, static_cast<const float*>(x), stream);
}

}  // namespace convgb
