// group_norm.cu -- group norm with an activation over NHWC tensors, forward,
// backward, and with an 8-bit output.
//
//   group S = (image n, group g): P * cpg values, P = H * W, cpg = C / G
//   mean = sum x / |S|, rstd = 1 / sqrt(sum (x - mean)^2 / |S| + eps)
//   z = ((x - mean) * rstd) * gamma[c] + beta[c],  y = act(z)
//
// backward, with u = dy * act'(z) and h = (x - mean) * rstd:
//   dbeta[c] = sum_{n,p} u,  dgamma[c] = sum_{n,p} u * h
//   a = sum_S u * gamma / |S|,  b = sum_S u * gamma * h / |S|
//   dx = rstd * (u * gamma - a - h * b)
//
// Both directions compute h and z in the same order of rounded operations, so
// the backward pass takes ReLU's kink where the forward pass had it.
//
// Sums are FP32.  The variance never comes from a difference of large sums: each
// thread sums the distances to its own first value, and partial (count, mean,
// sum of squares) triples join as
//   mean = sum n_i mean_i / n,  M2 = sum M2_i + n_i (mean_i - mean)^2.
//
// Streaming form (any shape): one pass that leaves per-channel partials of pixel
// ranges in the workspace, a small kernel that joins them per group, and a
// second pass that applies them.
#include "norm_internal.h"
#include "pointwise_math.cuh"

namespace convgb {

namespace {

// A CTA's threads over [pixels][vectors of channels]: cv vectors side by side, as many pixels as fit.
struct Lanes {
    int cv, rows;  // vectors side by side, pixel rows
    int v, r;      // this thread's vector of the pixel, and its row
    bool on;
};

__device__ __forceinline__ Lanes lanes_of(int vecs, int block) {
    const int cv = min(vecs, kNormThreads);
    Lanes l;
    l.cv = cv;
    l.rows = kNormThreads / cv;
    l.r = threadIdx.x / cv;
    l.v = block * cv + (threadIdx.x - l.r * cv);
    l.on = l.r < l.rows && l.v < vecs;
    return l;
}

__device__ __forceinline__ void split_range(int P, int splits, int s, int& p0, int& p1) {
    p0 = static_cast<int>(static_cast<long long>(P) * s / splits);
    p1 = static_cast<int>(static_cast<long long>(P) * (s + 1) / splits);
}

// Sum over the CTA's pixel rows of one value per (row, channel of the block), the same
// order every time.  Every thread gets the sums of its own channels back.
template <int VEC>
__device__ __forceinline__ void column_sums(float (&val)[VEC], const Lanes& l, float* scratch) {
    const int col = threadIdx.x - l.r * l.cv;
    const int width = l.cv * VEC;
    __syncthreads();
    if (l.r < l.rows)
#pragma unroll
        for (int i = 0; i < VEC; ++i) scratch[l.r * width + col * VEC + i] = l.on ? val[i] : 0.0f;
    __syncthreads();
    for (int c = threadIdx.x; c < width; c += kNormThreads) {
        float s = 0.0f;
        for (int r = 0; r < l.rows; ++r) s += scratch[r * width + c];
        scratch[c] = s;  // row 0 of this column: read above by this thread only
    }
    __syncthreads();
    if (l.r < l.rows)
#pragma unroll
        for (int i = 0; i < VEC; ++i) val[i] = scratch[col * VEC + i];
}

// Per-channel (mean, M2) of one pixel range.
template <typename T, int VEC>
__global__ void __launch_bounds__(kNormThreads) norm_moments_kernel(const NormParams p) {
    __shared__ float scratch[kNormThreads * VEC];
    const int n = blockIdx.x / p.splits, s = blockIdx.x - n * p.splits;
    const int vecs = p.C / VEC;
    const Lanes l = lanes_of(vecs, blockIdx.y);
    int p0, p1;
    split_range(p.P, p.splits, s, p0, p1);
    using Io = VecIo<T, VEC>;
    const auto* x = reinterpret_cast<const typename Io::Raw*>(p.x) + static_cast<long long>(n) * p.P * vecs + l.v;
    float pivot[VEC], sum[VEC], sq[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) pivot[i] = sum[i] = sq[i] = 0.0f;
    int cnt = 0;
    if (l.on) {
        for (int px = p0 + l.r; px < p1; px += l.rows, ++cnt) {
            float v[VEC];
            Io::unpack(x[static_cast<long long>(px) * vecs], v);
            if (cnt == 0)
#pragma unroll
                for (int i = 0; i < VEC; ++i) pivot[i] = v[i];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float d = v[i] - pivot[i];
                sum[i] += d;
                sq[i] = fmaf(d, d, sq[i]);
            }
        }
    }
    const float total = static_cast<float>(p1 - p0), n_t = static_cast<float>(cnt);
    float mean[VEC], m2[VEC], joint[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const float d = cnt ? sum[i] / n_t : 0.0f;
        mean[i] = pivot[i] + d;
        m2[i] = fmaxf(sq[i] - d * sum[i], sq[i] * 0.0f);  // not below 0; NaN stays
        joint[i] = n_t * mean[i];
    }
    column_sums<VEC>(joint, l, scratch);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        joint[i] /= total;
        const float d = mean[i] - joint[i];
        if (cnt) m2[i] = fmaf(n_t * d, d, m2[i]);
    }
    column_sums<VEC>(m2, l, scratch);
    if (l.on && l.r == 0)
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            p.part[static_cast<long long>(blockIdx.x) * p.C + l.v * VEC + i] = make_float2(joint[i], m2[i]);
}

__device__ __forceinline__ float block_sum(float v, float* scratch) {
    __syncthreads();
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) s += scratch[w];
    return s;
}

// One CTA per (image, group): joins the ranges and channels of the group.
__global__ void __launch_bounds__(128) norm_join_kernel(const NormParams p) {
    __shared__ float scratch[4];
    const int n = blockIdx.x / p.G, g = blockIdx.x - n * p.G;
    const int entries = p.splits * p.cpg;
    const float2* part = p.part + static_cast<long long>(n) * p.splits * p.C + g * p.cpg;
    const float total = static_cast<float>(p.P) * static_cast<float>(p.cpg);
    float s = 0.0f;
    for (int e = threadIdx.x; e < entries; e += blockDim.x) {
        const int sp = e / p.cpg, c = e - sp * p.cpg;
        int p0, p1;
        split_range(p.P, p.splits, sp, p0, p1);
        s = fmaf(static_cast<float>(p1 - p0), part[static_cast<long long>(sp) * p.C + c].x, s);
    }
    const float mean = block_sum(s, scratch) / total;
    float m2 = 0.0f;
    for (int e = threadIdx.x; e < entries; e += blockDim.x) {
        const int sp = e / p.cpg, c = e - sp * p.cpg;
        int p0, p1;
        split_range(p.P, p.splits, sp, p0, p1);
        const float2 v = part[static_cast<long long>(sp) * p.C + c];
        const float d = v.x - mean;
        m2 += v.y + static_cast<float>(p1 - p0) * d * d;
    }
    const float var = block_sum(m2, scratch) / total;
    if (threadIdx.x == 0) {
        p.mean[blockIdx.x] = mean;
        p.rstd[blockIdx.x] = __fdiv_rn(1.0f, __fsqrt_rn(var + p.eps));
    }
}

// What a channel needs to apply the norm.
struct Channel {
    float mean, rstd, gamma, beta;
};

__device__ __forceinline__ Channel channel_of(const NormParams& p, int n, int c) {
    const int s = n * p.G + c / p.cpg;
    return {p.mean[s], p.rstd[s], p.gamma ? p.gamma[c] : 1.0f, p.beta ? p.beta[c] : 0.0f};
}

__device__ __forceinline__ float norm_h(float x, float mean, float rstd) { return __fmul_rn(__fsub_rn(x, mean), rstd); }
__device__ __forceinline__ float norm_z(float h, float gamma, float beta) { return __fadd_rn(__fmul_rn(h, gamma), beta); }

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kNormThreads) norm_apply_kernel(const NormParams p) {
    const int n = blockIdx.x / p.splits, s = blockIdx.x - n * p.splits;
    const int vecs = p.C / VEC;
    const Lanes l = lanes_of(vecs, blockIdx.y);
    if (!l.on) return;
    int p0, p1;
    split_range(p.P, p.splits, s, p0, p1);
    using Io = VecIo<T, VEC>;
    const long long base = static_cast<long long>(n) * p.P * vecs + l.v;
    const auto* x = reinterpret_cast<const typename Io::Raw*>(p.x) + base;
    auto* y = reinterpret_cast<typename Io::Raw*>(p.y) + base;
    Channel ch[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) ch[i] = channel_of(p, n, l.v * VEC + i);
    for (int px = p0 + l.r; px < p1; px += l.rows) {
        float v[VEC];
        Io::unpack(x[static_cast<long long>(px) * vecs], v);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            v[i] = activate<ACT>(norm_z(norm_h(v[i], ch[i].mean, ch[i].rstd), ch[i].gamma, ch[i].beta));
        y[static_cast<long long>(px) * vecs] = Io::pack(v);
    }
}

// 8-bit output: one warp per pixel, two sweeps over its channels (the row's largest
// magnitude, then the values; the second sweep finds the row in L1).
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kNormThreads) norm_apply_int8_kernel(const NormParams p) {
    const int lane = threadIdx.x & 31;
    const int vecs = p.C / VEC;
    const long long pixels = static_cast<long long>(p.N) * p.P;
    using Io = VecIo<T, VEC>;
    for (long long row = static_cast<long long>(blockIdx.x) * (kNormThreads / 32) + (threadIdx.x >> 5); row < pixels;
         row += static_cast<long long>(gridDim.x) * (kNormThreads / 32)) {
        const int n = static_cast<int>(row / p.P);
        const auto* x = reinterpret_cast<const typename Io::Raw*>(p.x) + row * vecs;
        uint32_t amax = 0;
        for (int v = lane; v < vecs; v += 32) {
            float f[VEC];
            Io::unpack(x[v], f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const Channel ch = channel_of(p, n, v * VEC + i);
                amax = max(amax, magnitude_bits(activate<ACT>(norm_z(norm_h(f[i], ch.mean, ch.rstd), ch.gamma, ch.beta))));
            }
        }
        const RowScale rs = row_scale(warp_max(amax));
        if (lane == 0) p.scale[row] = rs.scale;
        int8_t* q = p.q + row * p.C;
        for (int v = lane; v < vecs; v += 32) {
            float f[VEC];
            Io::unpack(x[v], f);
            int o[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const Channel ch = channel_of(p, n, v * VEC + i);
                o[i] = quantise(activate<ACT>(norm_z(norm_h(f[i], ch.mean, ch.rstd), ch.gamma, ch.beta)), rs.inv);
            }
            if constexpr (VEC == 8)
                *reinterpret_cast<uint2*>(q + v * 8) =
                    make_uint2(pack_int8x4(o[0], o[1], o[2], o[3]), pack_int8x4(o[4], o[5], o[6], o[7]));
            else if constexpr (VEC == 4)
                *reinterpret_cast<uint32_t*>(q + v * 4) = pack_int8x4(o[0], o[1], o[2], o[3]);
            else
                q[v] = static_cast<int8_t>(o[0]);
        }
    }
}

// ---------------------------------------------------------------- backward
// Per-channel (sum u, sum u * h) of one pixel range.
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kNormThreads) norm_grad_sums_kernel(const NormParams p) {
    __shared__ float scratch[kNormThreads * VEC];
    const int n = blockIdx.x / p.splits, s = blockIdx.x - n * p.splits;
    const int vecs = p.C / VEC;
    const Lanes l = lanes_of(vecs, blockIdx.y);
    int p0, p1;
    split_range(p.P, p.splits, s, p0, p1);
    using Io = VecIo<T, VEC>;
    const long long base = static_cast<long long>(n) * p.P * vecs + l.v;
    const auto* x = reinterpret_cast<const typename Io::Raw*>(p.x) + base;
    const auto* dy = reinterpret_cast<const typename Io::Raw*>(p.dy) + base;
    float su[VEC], suh[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) su[i] = suh[i] = 0.0f;
    if (l.on) {
        Channel ch[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) ch[i] = channel_of(p, n, l.v * VEC + i);
        for (int px = p0 + l.r; px < p1; px += l.rows) {
            float v[VEC], d[VEC];
            Io::unpack(x[static_cast<long long>(px) * vecs], v);
            Io::unpack(dy[static_cast<long long>(px) * vecs], d);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float h = norm_h(v[i], ch[i].mean, ch[i].rstd);
                const float u = activate_grad<ACT>(norm_z(h, ch[i].gamma, ch[i].beta), d[i]);
                su[i] += u;
                suh[i] = fmaf(u, h, suh[i]);
            }
        }
    }
    column_sums<VEC>(su, l, scratch);
    column_sums<VEC>(suh, l, scratch);
    if (l.on && l.r == 0)
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            p.part[static_cast<long long>(blockIdx.x) * p.C + l.v * VEC + i] = make_float2(su[i], suh[i]);
}

// One CTA per (image, group): a and b.
__global__ void __launch_bounds__(128) norm_grad_join_kernel(const NormParams p) {
    __shared__ float scratch[4];
    const int n = blockIdx.x / p.G, g = blockIdx.x - n * p.G;
    const int entries = p.splits * p.cpg;
    const float2* part = p.part + static_cast<long long>(n) * p.splits * p.C + g * p.cpg;
    float a = 0.0f, b = 0.0f;
    for (int e = threadIdx.x; e < entries; e += blockDim.x) {
        const int sp = e / p.cpg, c = e - sp * p.cpg;
        const float2 v = part[static_cast<long long>(sp) * p.C + c];
        const float gm = p.gamma ? p.gamma[g * p.cpg + c] : 1.0f;
        a = fmaf(gm, v.x, a);
        b = fmaf(gm, v.y, b);
    }
    const float total = static_cast<float>(p.P) * static_cast<float>(p.cpg);
    a = block_sum(a, scratch) / total;
    b = block_sum(b, scratch) / total;
    if (threadIdx.x == 0) p.ab[blockIdx.x] = make_float2(a, b);
}

// One CTA per channel: dgamma and dbeta over every image and range.
__global__ void __launch_bounds__(128) norm_grad_channels_kernel(const NormParams p) {
    __shared__ float scratch[4];
    const int c = blockIdx.x;
    const long long entries = static_cast<long long>(p.N) * p.splits;
    float s = 0.0f, h = 0.0f;
    for (long long e = threadIdx.x; e < entries; e += blockDim.x) {
        const float2 v = p.part[e * p.C + c];
        s += v.x;
        h += v.y;
    }
    s = block_sum(s, scratch);
    h = block_sum(h, scratch);
    if (threadIdx.x == 0) {
        p.dbeta[c] = s;
        p.dgamma[c] = h;
    }
}

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kNormThreads) norm_grad_apply_kernel(const NormParams p) {
    const int n = blockIdx.x / p.splits, s = blockIdx.x - n * p.splits;
    const int vecs = p.C / VEC;
    const Lanes l = lanes_of(vecs, blockIdx.y);
    if (!l.on) return;
    int p0, p1;
    split_range(p.P, p.splits, s, p0, p1);
    using Io = VecIo<T, VEC>;
    const long long base = static_cast<long long>(n) * p.P * vecs + l.v;
    const auto* x = reinterpret_cast<const typename Io::Raw*>(p.x) + base;
    const auto* dy = reinterpret_cast<const typename Io::Raw*>(p.dy) + base;
    auto* dx = reinterpret_cast<typename Io::Raw*>(p.y) + base;
    Channel ch[VEC];
    float2 ab[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        ch[i] = channel_of(p, n, l.v * VEC + i);
        ab[i] = p.ab[n * p.G + (l.v * VEC + i) / p.cpg];
    }
    for (int px = p0 + l.r; px < p1; px += l.rows) {
        float v[VEC], d[VEC];
        Io::unpack(x[static_cast<long long>(px) * vecs], v);
        Io::unpack(dy[static_cast<long long>(px) * vecs], d);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float h = norm_h(v[i], ch[i].mean, ch[i].rstd);
            const float u = activate_grad<ACT>(norm_z(h, ch[i].gamma, ch[i].beta), d[i]);
            v[i] = ch[i].rstd * (fmaf(u, ch[i].gamma, -ab[i].x) - h * ab[i].y);
        }
        dx[static_cast<long long>(px) * vecs] = Io::pack(v);
    }
}

// ---------------------------------------------------------------- launch
template <typename F>
void with_types(const NormParams& p, F&& f) {
    if (p.bf16) {
        if (p.vec == 8) f(__nv_bfloat16(), std::integral_constant<int, 8>());
        else f(__nv_bfloat16(), std::integral_constant<int, 1>());
    } else {
        if (p.vec == 4) f(float(), std::integral_constant<int, 4>());
        else f(float(), std::integral_constant<int, 1>());
    }
}

template <typename F>
void with_act(int act, F&& f) {
    if (act == CONV_ACT_RELU) f(std::integral_constant<int, CONV_ACT_RELU>());
    else if (act == CONV_ACT_SILU) f(std::integral_constant<int, CONV_ACT_SILU>());
    else f(std::integral_constant<int, CONV_ACT_NONE>());
}

dim3 stream_grid(const NormParams& p) {
    const int vecs = p.C / p.vec;
    const int cv = vecs < kNormThreads ? vecs : kNormThreads;
    return dim3(static_cast<unsigned>(p.N) * p.splits, (vecs + cv - 1) / cv);
}

}  // namespace

size_t norm_workspace_bytes(const NormParams& p) {
    return (static_cast<size_t>(p.N) * p.splits * p.C + static_cast<size_t>(p.N) * p.G) * sizeof(float2) +
           2 * static_cast<size_t>(p.N) * p.G * sizeof(float);
}

cudaError_t launch_norm_forward(const NormParams& p, int num_sms, cudaStream_t stream) {
    const dim3 grid = stream_grid(p);
    with_types(p, [&](auto t, auto vec) {
        norm_moments_kernel<decltype(t), vec.value><<<grid, kNormThreads, 0, stream>>>(p);
    });
    norm_join_kernel<<<p.N * p.G, 128, 0, stream>>>(p);
    with_types(p, [&](auto t, auto vec) {
        with_act(p.act, [&](auto act) {
            if (p.q != nullptr) {
                const long long rows = (static_cast<long long>(p.N) * p.P + 7) / 8;
                const unsigned g = static_cast<unsigned>(rows < num_sms * 8LL ? rows : num_sms * 8LL);
                norm_apply_int8_kernel<decltype(t), vec.value, act.value><<<g, kNormThreads, 0, stream>>>(p);
            } else {
                norm_apply_kernel<decltype(t), vec.value, act.value><<<grid, kNormThreads, 0, stream>>>(p);
            }
        });
    });
    return cudaGetLastError();
}

cudaError_t launch_norm_backward(const NormParams& p, int num_sms, cudaStream_t stream) {
    (void)num_sms;
    const dim3 grid = stream_grid(p);
    with_types(p, [&](auto t, auto vec) {
        with_act(p.act, [&](auto act) {
            norm_grad_sums_kernel<decltype(t), vec.value, act.value><<<grid, kNormThreads, 0, stream>>>(p);
            norm_grad_join_kernel<<<p.N * p.G, 128, 0, stream>>>(p);
            if (p.dgamma != nullptr) norm_grad_channels_kernel<<<p.C, 128, 0, stream>>>(p);
            norm_grad_apply_kernel<decltype(t), vec.value, act.value><<<grid, kNormThreads, 0, stream>>>(p);
        });
    });
    return cudaGetLastError();
}

}  // namespace convgb
