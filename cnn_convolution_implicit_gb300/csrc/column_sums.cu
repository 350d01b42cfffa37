// column_sums.cu -- gradients of what is broadcast over the rows: the linear layer's u = dy * act'(z) with its sums
// over the rows (dbias), and the join of such sums' parts.
//
// Bound by reading dy and z and writing u: 8192 x 4096 with SiLU 30 us with cold caches, 6.7 TB/s (the last of u is still in L2 when it
// ends).  A CTA takes a strip of columns of a range of rows; a thread keeps its columns' sums over its rows in FP32, the threads' meet
// in shared memory and the ranges' in the workspace, always in one order.
#include <type_traits>

#include "linear_internal.h"
#include "pointwise_math.cuh"
#include "row_sums.cuh"
#include "rows_internal.h"

namespace convgb {

namespace {

constexpr int kThreads = 256;

// A strip: `lanes` threads (a power of two) of VEC columns each to a row, kThreads / lanes rows at a time.
struct Strip {
    int vec, lanes, strips;
};
Strip strip_of(int N) {
    Strip s;
    s.vec = N % 8 == 0 ? 8 : (N % 4 == 0 ? 4 : (N % 2 == 0 ? 2 : 1));
    const int vecs = N / s.vec;
    s.lanes = 1;
    while (s.lanes < 32 && s.lanes < vecs) s.lanes *= 2;
    s.strips = (vecs + s.lanes - 1) / s.lanes;
    return s;
}

// Rows whose loads a thread has under way: more of them where the loads are narrow.
__host__ __device__ constexpr int batch_of(int vec) { return vec == 8 ? 2 : (vec == 4 ? 4 : 8); }

template <int VEC, int ACT>
__global__ void __launch_bounds__(kThreads) linear_grad_kernel(const LinearGradParams p, int lanes, float* sums_out) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the product that may follow
    constexpr int H = (VEC + 1) / 2, kBatch = batch_of(VEC);
    using Io = VecIo<__nv_bfloat16, VEC>;
    using Raw = typename Io::Raw;
    __shared__ float sums[kThreads * VEC];
    const int lane = threadIdx.x % lanes, slot = threadIdx.x / lanes, slots = kThreads / lanes;
    const int n = (blockIdx.x * lanes + lane) * VEC;
    f2 total[H] = {};
    if (n < p.N) {
        const long long step = static_cast<long long>(gridDim.y) * slots;
        for (long long m0 = static_cast<long long>(blockIdx.y) * slots + slot; m0 < p.M; m0 += kBatch * step) {
            Raw dy[kBatch] = {}, z[kBatch] = {};
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const long long m = m0 + i * step;
                if (m >= p.M) break;
                dy[i] = *reinterpret_cast<const Raw*>(p.dy + m * p.N + n);
                if constexpr (ACT != CONV_ACT_NONE) z[i] = *reinterpret_cast<const Raw*>(p.z + m * p.N + n);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const long long m = m0 + i * step;
                if (m >= p.M) break;
                f2 u[H], v[H];
                Io::unpack(dy[i], u);
                if constexpr (ACT != CONV_ACT_NONE) {
                    Io::unpack(z[i], v);
#pragma unroll
                    for (int j = 0; j < H; ++j) u[j] = activate_grad2<ACT>(v[j], u[j]);
                }
#pragma unroll
                for (int j = 0; j < H; ++j) total[j] = f2_add_rounded(total[j], u[j]);  // the same sums with and without u
                if (p.u != nullptr) *reinterpret_cast<Raw*>(p.u + m * p.u_pitch + n) = Io::pack(u);
            }
        }
    }
    if (sums_out == nullptr) return;
#pragma unroll
    for (int j = 0; j < VEC; ++j) sums[slot * lanes * VEC + lane * VEC + j] = j & 1 ? f2_hi(total[j / 2]) : f2_lo(total[j / 2]);
    __syncthreads();
    for (int i = threadIdx.x; i < lanes * VEC; i += kThreads) {
        const int c = blockIdx.x * lanes * VEC + i;
        if (c >= p.N) break;
        float sum = 0.0f;
        for (int k = 0; k < slots; ++k) sum += sums[k * lanes * VEC + i];
        sums_out[static_cast<long long>(blockIdx.y) * p.N + c] = sum;
    }
}

// 32 columns a CTA.
__global__ void __launch_bounds__(1024) join_columns_kernel(const float* part, int parts, int C, float* out) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float sums[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    sums[warp][lane] = c < C ? sum_of_parts(part, warp, parts, C, c) : 0.0f;
    __syncthreads();
    float sum = sums[lane][warp];  // column `warp` of the block
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
    if (lane == 0 && blockIdx.x * 32 + warp < C) out[blockIdx.x * 32 + warp] = sum;
}

}  // namespace

cudaError_t launch_join_columns(const float* part, int parts, int C, float* out, bool early, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((C + 31) / 32);
    cfg.blockDim = dim3(1024);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, join_columns_kernel, part, parts, C, out);
}

// About four CTAs an SM (eight where accesses are narrow), a batch of rows a thread at least.  Where a thread's chain would pass
// kChainRows, parts for a quarter of that, up to a grid's 65,535 (262144 x 4096 with SiLU, dbias alone: 553 us in 38 parts, 577 in
// the 64 of 512 rows, 530 in 256).
int linear_grad_parts(int M, int N, int num_sms) {
    const Strip s = strip_of(N);
    const int slots = kThreads / s.lanes;
    const int rows = slots * batch_of(s.vec);
    const long long need = (static_cast<long long>(M) + rows - 1) / rows, most = ((s.vec >= 4 ? 4LL : 8LL) * num_sms + s.strips - 1) / s.strips;
    const long long chains = (M + static_cast<long long>(slots) * kChainRows - 1) / (static_cast<long long>(slots) * kChainRows);
    const long long parts = need < most ? need : (most >= chains ? most : 4 * chains);
    return static_cast<int>(parts < 65535 ? parts : 65535);
}

cudaError_t launch_linear_grad(const LinearGradParams& p, int num_sms, bool join, cudaStream_t stream) {
    const Strip s = strip_of(p.N);
    const int parts = linear_grad_parts(p.M, p.N, num_sms);
    float* sums = p.dbias == nullptr ? nullptr : (parts > 1 ? p.part : p.dbias);
    const dim3 grid(s.strips, parts);
    const auto run = [&](auto vec) {
        constexpr int V = decltype(vec)::value;
        if (p.act == CONV_ACT_RELU) linear_grad_kernel<V, CONV_ACT_RELU><<<grid, kThreads, 0, stream>>>(p, s.lanes, sums);
        else if (p.act == CONV_ACT_SILU) linear_grad_kernel<V, CONV_ACT_SILU><<<grid, kThreads, 0, stream>>>(p, s.lanes, sums);
        else linear_grad_kernel<V, CONV_ACT_NONE><<<grid, kThreads, 0, stream>>>(p, s.lanes, sums);
    };
    if (s.vec == 8) run(std::integral_constant<int, 8>());
    else if (s.vec == 4) run(std::integral_constant<int, 4>());
    else if (s.vec == 2) run(std::integral_constant<int, 2>());
    else run(std::integral_constant<int, 1>());
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.dbias == nullptr || parts == 1 || !join) return e;
    return launch_join_columns(p.part, parts, p.N, p.dbias, true, stream);
}

}  // namespace convgb
