// linear_few.cu -- the linear layer with few rows (tokens), up to 32:
//
//   z[m][n] = sum_k x[m][k] * w[n][k] + bias[n],   y = act(z) + residual
//
// Bound by reading w once: 2 N K bytes (1 x 4096 -> 16384 23 us, 5.8 TB/s; 1 x 4096 -> 4096 7.8, 4.3, the launch among them).  Both operands go from memory to registers and from there into BF16 MMAs of
// 16 x 8 x 16 (16 rows of w, 8 of x), whose rate does not matter here; the 128-row tiles of the kernel for many rows
// and their set-up would.  A CTA takes 16 rows of w; its eight warps share K, 64 at a time.  Lane 4 g + q holds
// k = 8 q .. 8 q + 7 of each 32 of rows g and g + 8 of w and of row g of x: the MMA sums over k in any order, so its
// slots (2 q, 2 q + 1, 2 q + 8, 2 q + 9) take the lane's words 2 j and 2 j + 1, for both operands alike.  The warps'
// sums meet in shared memory in one order.
#include "int8_rows.cuh"
#include "linear_internal.h"
#include "pointwise_math.cuh"

namespace convgb {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kColumns = 16;            // rows of w of a CTA
constexpr int kStep = 64 * kWarps;      // K of a step of all warps

template <bool ALIGNED>
__device__ __forceinline__ uint4 item(const __nv_bfloat16* base, int row, int rows, int k, int K) {
    if (row >= rows || k >= K) return make_uint4(0, 0, 0, 0);
    const long long at = static_cast<long long>(row) * K + k;
    if constexpr (ALIGNED) return __ldg(reinterpret_cast<const uint4*>(base + at));
    else return load_item(reinterpret_cast<const int8_t*>(base), 2 * at, K - k < 8 ? 2 * (K - k) : 16, 2LL * rows * K);
}

// words 2 j, 2 j + 1 of an item
__device__ __forceinline__ uint2 words(const uint4& v, int j) { return j == 0 ? make_uint2(v.x, v.y) : make_uint2(v.z, v.w); }

__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint2 lo, uint2 hi, uint2 b) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(lo.x), "r"(hi.x), "r"(lo.y), "r"(hi.y), "r"(b.x), "r"(b.y));
}

// T: 8-row tiles of x.
template <int T, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 2) linear_few_kernel(const FewParams p) {
    constexpr int B = 4;                    // steps whose loads of w are under way
    constexpr int BX = T == 1 ? 4 : (T == 2 ? 2 : 1);  // and of x
    __shared__ float parts[kWarps][T * 8][kColumns + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int n0 = blockIdx.x * kColumns;
    float acc[T][4] = {};
    uint4 w[B][2][2];  // step, half of 64, rows g and g + 8
    const auto load_weights = [&](int k0) {
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int t = 0; t < 2; ++t) w[b][h][t] = item<ALIGNED>(p.w, n0 + 8 * t + g, p.N, k0 + b * kStep + 32 * h + 8 * q, p.K);
    };
    load_weights(64 * warp);
    for (int k0 = 64 * warp; k0 < p.K; k0 += B * kStep) {
#pragma unroll
        for (int b0 = 0; b0 < B; b0 += BX) {
            if (b0 > 0 && k0 + b0 * kStep >= p.K) break;
            uint4 x[BX][2][T];
#pragma unroll
            for (int b = 0; b < BX; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int t = 0; t < T; ++t)
                        x[b][h][t] = item<ALIGNED>(p.x, 8 * t + g, p.M, k0 + (b0 + b) * kStep + 32 * h + 8 * q, p.K);
#pragma unroll
            for (int b = 0; b < BX; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int t = 0; t < T; ++t)
                            mma_16x8x16(acc[t], words(w[b0 + b][h][0], j), words(w[b0 + b][h][1], j), words(x[b][h][t], j));
        }
        if (k0 + B * kStep < p.K) load_weights(k0 + B * kStep);
    }
    // lane: rows g and g + 8 of w, rows 2 q and 2 q + 1 of x
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) parts[warp][8 * t + 2 * q + (i & 1)][g + 8 * (i >> 1)] = acc[t][i];
    __syncthreads();
#pragma unroll
    for (int i = threadIdx.x; i < T * 8 * kColumns; i += kThreads) {
        const int m = i / kColumns, c = i % kColumns, n = n0 + c;
        if (m >= p.M || n >= p.N) continue;
        float z = 0.0f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) z += parts[k][m][c];
        if (p.bias != nullptr) z = __fadd_rn(z, __ldg(p.bias + n));
        const long long o = static_cast<long long>(m) * p.N + n;
        if (p.z != nullptr) p.z[o] = __float2bfloat16_rn(z);
        float y = p.act == CONV_ACT_RELU ? activate<CONV_ACT_RELU>(z) : (p.act == CONV_ACT_SILU ? activate<CONV_ACT_SILU>(z) : z);
        if (p.r != nullptr) y = __fadd_rn(y, __bfloat162float(p.r[o]));  // an ordinary load: y may be the residual
        p.y[o] = __float2bfloat16_rn(y);
    }
}

template <int T>
cudaError_t launch(const FewParams& p, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>((static_cast<long long>(p.N) + kColumns - 1) / kColumns);
    if (p.K % 8 == 0) linear_few_kernel<T, true><<<grid, kThreads, 0, stream>>>(p);
    else linear_few_kernel<T, false><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

// This kernel and the tiles of many rows, microseconds in a graph with cold weights:
//   8 x 4096 -> 4096 8.6 and 14.5    16 x 4096 -> 4096 10.1 and 12.8   24 x 4096 -> 4096 14.0 and 13.4   32 x 1024 -> 1024 4.9 and 7.1
//   8 x 16384 -> 4096 24.4 and 29.7  16 x 8192 -> 4096 17.5 and 18.5   16 x 4096 -> 16384 33.7 and 26.8  32 x 2048 -> 2048 8.4 and 8.6
//   8 x 4096 -> 16384 25.5 and 40.4  16 x 16384 -> 1024 18.7 and 12.1  32 x 4096 -> 1024 12.8 and 9.3
// x is read again by every 16 columns, so with more rows and weights the tiles win, and where K is long, which they share.
// Rows of K off 16 bytes take two loads and a shift for each item, and a time that goes by K and M; the tiles take a launch
// more, that lays rows out (4 of a call where the host bounds it):
//   8 x 2045 -> 2048 13.8 and 12.8   8 x 2500 -> 512 16.6 and 9.4      16 x 1003 -> 1000 8.2 and 8.2     16 x 2045 -> 2048 18.1 and 12.8
//   8 x 1027 -> 4096 9.0 and 12.9    32 x 501 -> 300 7.0 and 8.2       32 x 1003 -> 1000 11.1 and 8.0
bool linear_use_few(int M, int N, int K) {
    if (K % 8 != 0 && K > (M <= 8 ? 2300 : (M <= 16 ? 1500 : 1200))) return false;
    const long long weights = static_cast<long long>(N) * K;
    return M <= 8 || (M <= 16 && weights <= 1LL << 25 && K <= 8192) || (M <= 32 && weights <= 1LL << 22 && K <= 3000);
}

cudaError_t launch_linear_few(const FewParams& p, cudaStream_t stream) {
    if (p.M <= 8) return launch<1>(p, stream);
    if (p.M <= 16) return launch<2>(p, stream);
    if (p.M <= 24) return launch<3>(p, stream);
    return launch<4>(p, stream);
}

}  // namespace convgb
