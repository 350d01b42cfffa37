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
// The forward pass takes z as a difference and one fused multiply-add, (x - mean) * (rstd *
// gamma) + beta (a flat group gives beta itself); the backward pass, which needs h, rounds
// each operation as written, so that ReLU's kink lies where the formula in FP32 puts it.
//
// Sums are FP32.  The variance never comes from a difference of large sums: each
// thread sums the distances to its own first value, and partial (count, mean,
// sum of squares) triples join as
//   mean = sum n_i mean_i / n,  M2 = sum M2_i + n_i (mean_i - mean)^2.
//
// Bound by memory: x read and y written once (backward: x and dy read, dx written).  Three forms,
// chosen per plan (norm_resident_pays); times with cold caches, launch included, against the
// bytes at the card's measured copy rate:
//
//   Resident: each CTA copies its pixels of `chunk` channels into shared memory once
//   (cp.async, each thread reads back only what it copied), pushes its groups' sums into the
//   shared memory of its cluster, and after one cluster barrier writes the values from
//   there: every byte crosses the memory bus once, in one launch.  Two CTAs an SM, so one loads
//   while the other stores; with 200 KB an SM in flight the rate is those bytes over a CTA's
//   life (~11 us: 5.5 loading, 3 from the last load to the first store, 2.5 storing), and clusters
//   of eight fill 288 of 304 places, of sixteen 224.
//     1 x 8 x 8 x 256 BF16: 9 us; 64 x 56 x 56 x 256: 57 us (floor 30); 32 x 112 x 112 x 256, ReLU: 95 (61).
//   Two passes (maps that no cluster of 16 holds, and where clusters fill the SMs badly): one
//   kernel leaves each pixel range's group sums, streaming it through shared memory; the next joins
//   them in its prologue and writes the values, walking its range backwards and storing past
//   the caches, so that part of x is still in L2.  The second is launched early and waits for
//   the first.  It reads x twice; where a CTA's life would be long or clusters large it wins.
//     1 x 512 x 512 x 128 BF16: 44 us (floor 20); 64 x 56 x 56 x 256 to 8 bits: 70 (23), resident 93;
//     backward, SiLU, 32 x 112 x 112 x 128: 109 (45), resident 138 (ReLU 97); 16 x 64 x 64 x 256 44 (15), resident 50.
//   By channel (pixels that do not start on 16 bytes, over 256 vectors a pixel): as two passes, the
//   sums kept per channel and joined by a kernel of their own; 4- or 8-byte accesses where the
//   channels allow.  32 x 112 x 112 x 250 BF16: 192 us (floor 59), to 8 bits 564 (45), backward 437 (89).
#include "norm_internal.h"
#include "pointwise_math.cuh"

namespace convgb {

namespace {

// Sum over segments of `width` lanes (a power of two), every lane of the warp calling it.
__device__ __forceinline__ float segment_sum(float v, int width) {
    for (int o = width >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The smallest power of two that is at least n, at most a warp.
__device__ __forceinline__ int segment_width(int n) { return n >= 32 ? 32 : (n <= 1 ? 1 : 1 << (32 - __clz(n - 1))); }

// A CTA's threads over [pixels][vectors of channels]: cv vectors side by side, as many pixels as fit.
struct Lanes {
    int cv, rows;  // vectors side by side, pixel rows
    int v, r;      // this thread's vector of the pixel, and its row
    bool on;
};

__device__ __forceinline__ Lanes lanes_of(int vecs, unsigned block) {
    const int cv = min(vecs, kNormThreads);
    Lanes l;
    l.cv = cv;
    l.rows = kNormThreads / cv;
    l.r = threadIdx.x / cv;
    const unsigned v = block * cv + (threadIdx.x - l.r * cv);  // past 31 bits in a block past the last
    l.v = static_cast<int>(v);
    l.on = l.r < l.rows && v < static_cast<unsigned>(vecs);
    return l;
}

// Pixels of range (or cluster CTA) k of an image: pix_base, one more in the first pix_more.
__device__ __forceinline__ void pixel_range(const NormParams& p, int k, int& p0, int& p1) {
    p0 = k * p.pix_base + min(k, p.pix_more);
    p1 = p0 + p.pix_base + (k < p.pix_more);
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

// Sums of distances to the thread's first value, then its mean and sum of squares about it.
template <int VEC>
struct Moments {
    static constexpr int H = (VEC + 1) / 2;
    f2 minus_pivot[H], sum[H], sq[H];
    __device__ __forceinline__ Moments() {
#pragma unroll
        for (int i = 0; i < H; ++i) minus_pivot[i] = sum[i] = sq[i] = 0;
    }
    __device__ __forceinline__ void start(const f2 (&v)[H]) {
#pragma unroll
        for (int i = 0; i < H; ++i) minus_pivot[i] = f2_make(-f2_lo(v[i]), -f2_hi(v[i]));
    }
    __device__ __forceinline__ void add(const f2 (&v)[H]) {
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const f2 d = f2_add(v[i], minus_pivot[i]);
            sum[i] = f2_add(sum[i], d);
            sq[i] = f2_fma(d, d, sq[i]);
        }
    }
    __device__ __forceinline__ void finish(int cnt, float (&mean)[VEC], float (&m2)[VEC]) const {
        const float over_n = cnt ? __frcp_rn(static_cast<float>(cnt)) : 0.0f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float pv = i & 1 ? f2_hi(minus_pivot[i / 2]) : f2_lo(minus_pivot[i / 2]);
            const float s = i & 1 ? f2_hi(sum[i / 2]) : f2_lo(sum[i / 2]);
            const float q = i & 1 ? f2_hi(sq[i / 2]) : f2_lo(sq[i / 2]);
            const float d = s * over_n;
            mean[i] = d - pv;
            m2[i] = fmaxf(q - d * s, q * 0.0f);  // not below 0; NaN stays
        }
    }
};

// Per-channel (mean, M2) of one pixel range.
template <typename T, int VEC>
__global__ void __launch_bounds__(kNormThreads) norm_moments_kernel(const NormParams p) {
    __shared__ float scratch[kNormThreads * VEC];
    const int n = blockIdx.x / p.splits, s = blockIdx.x - n * p.splits;
    const int vecs = p.C / VEC;
    const Lanes l = lanes_of(vecs, blockIdx.y + blockIdx.z * gridDim.y);
    int p0, p1;
    pixel_range(p, s, p0, p1);
    using Io = VecIo<T, VEC>;
    const auto* x = reinterpret_cast<const typename Io::Raw*>(p.x) + static_cast<long long>(n) * p.P * vecs + l.v;
    Moments<VEC> mo;
    const int cnt = l.on && p0 + l.r < p1 ? (p1 - p0 - l.r + l.rows - 1) / l.rows : 0;
    if (cnt) {
        x += static_cast<long long>(p0 + l.r) * vecs;
        const long long step = static_cast<long long>(l.rows) * vecs;
        f2 v[Moments<VEC>::H];
        Io::unpack(x[0], v);
        mo.start(v);
#pragma unroll 4
        for (int i = 0; i < cnt; ++i) {
            Io::unpack(x[i * step], v);
            mo.add(v);
        }
    }
    const float total = static_cast<float>(p1 - p0), n_t = static_cast<float>(cnt);
    float mean[VEC], m2[VEC], joint[VEC];
    mo.finish(cnt, mean, m2);
#pragma unroll
    for (int i = 0; i < VEC; ++i) joint[i] = n_t * mean[i];
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

constexpr int kJoinThreads = 512;

// Calls f(range, channel) for the ranges and channels of a group, spread over the CTA: a segment of
// lanes to a range, no division per entry; a wide group's channels over every thread, so that few
// ranges leave no warp a long sum to itself (an FP32 chain of 2^19 squares loses 1.6e-4 of its
// value, of 2^15 2.6e-6).
template <typename F>
__device__ __forceinline__ void for_ranges_and_channels(const NormParams& p, F&& f) {
    if (p.cpg >= kJoinThreads) {
        for (int sp = 0; sp < p.splits; ++sp)
            for (int c = threadIdx.x; c < p.cpg; c += kJoinThreads) f(sp, c);
        return;
    }
    const int wide = segment_width(p.cpg), lane = threadIdx.x & 31;
    for (int sp = (threadIdx.x >> 5) * (32 / wide) + lane / wide; sp < p.splits; sp += kJoinThreads / wide)
        for (int c = lane & (wide - 1); c < p.cpg; c += wide) f(sp, c);
}

// One CTA per (image, group): joins the ranges and channels of the group.
__global__ void __launch_bounds__(kJoinThreads) norm_join_kernel(const NormParams p) {
    __shared__ float scratch[kJoinThreads / 32];
    const int n = blockIdx.x / p.G, g = blockIdx.x - n * p.G;
    const float2* part = p.part + static_cast<long long>(n) * p.splits * p.C + g * p.cpg;
    const float total = static_cast<float>(p.P) * static_cast<float>(p.cpg);
    float s = 0.0f;
    for_ranges_and_channels(p, [&](int sp, int c) {
        s = fmaf(static_cast<float>(p.pix_base + (sp < p.pix_more)), part[static_cast<long long>(sp) * p.C + c].x, s);
    });
    const float mean = block_sum(s, scratch) / total;
    float m2 = 0.0f;
    for_ranges_and_channels(p, [&](int sp, int c) {
        const float2 v = part[static_cast<long long>(sp) * p.C + c];
        const float d = v.x - mean;
        m2 += v.y + static_cast<float>(p.pix_base + (sp < p.pix_more)) * d * d;
    });
    const float var = block_sum(m2, scratch) / total;
    if (threadIdx.x == 0) {
        p.mean[blockIdx.x] = mean;
        p.rstd[blockIdx.x] = __fdiv_rn(1.0f, __fsqrt_rn(var + p.eps));
    }
}

// What the channels of a vector need: the forward pass's z = (x - mean) * a + beta.  load() takes
// gamma and beta, set() the statistics.  VEC = 1: the second lane of the pair, which holds no
// channel, stays 0 through every activation, so that a pixel's largest magnitude does not see it.
template <int VEC>
struct Affine {
    static constexpr int H = (VEC + 1) / 2;
    f2 minus_mean[H], a[H], b[H];
    __device__ __forceinline__ void load(const NormParams& p, int c) {
        float av[2 * H], bv[2 * H];
#pragma unroll
        for (int i = 0; i < 2 * H; ++i) {
            av[i] = i < VEC && p.gamma ? __ldg(p.gamma + c + i) : 1.0f;
            bv[i] = i < VEC && p.beta ? __ldg(p.beta + c + i) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < H; ++i) {
            a[i] = f2_make(av[2 * i], av[2 * i + 1]);
            b[i] = f2_make(bv[2 * i], bv[2 * i + 1]);
        }
    }
    template <typename F>
    __device__ __forceinline__ void set(int c, int cpg, F&& stats) {  // stats(channel): (mean, rstd)
        if (VEC > 1 && cpg % VEC == 0) {  // the vector lies in one group
            const float2 st = stats(c);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                minus_mean[i] = f2_dup(-st.x);
                a[i] = f2_mul(a[i], f2_dup(st.y));
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const float2 lo = stats(c + 2 * i), hi = 2 * i + 1 < VEC ? stats(c + 2 * i + 1) : make_float2(0.0f, 0.0f);
            minus_mean[i] = f2_make(-lo.x, -hi.x);
            a[i] = f2_mul(a[i], f2_make(lo.y, hi.y));
        }
    }
    template <int ACT>
    __device__ __forceinline__ void apply(f2 (&v)[H]) const {
#pragma unroll
        for (int i = 0; i < H; ++i) v[i] = activate2<ACT>(f2_fma(f2_add(v[i], minus_mean[i]), a[i], b[i]));
    }
};

// The backward pass: h and z as written, u, and the sums or dx.
template <int VEC>
struct Grad {
    static constexpr int H = (VEC + 1) / 2;
    f2 minus_mean[H], rstd[H], gamma[H], beta[H];
    template <typename F>
    __device__ __forceinline__ void set(const NormParams& p, int c, F&& stats) {
        float m[2 * H], r[2 * H], g[2 * H], be[2 * H];
        const bool one = p.cpg % VEC == 0;  // the vector lies in one group
        const float2 first = stats(c);
#pragma unroll
        for (int i = 0; i < 2 * H; ++i) {
            m[i] = r[i] = g[i] = be[i] = 0.0f;
            if (i < VEC) {
                const float2 st = one ? first : stats(c + i);
                m[i] = -st.x;
                r[i] = st.y;
                g[i] = p.gamma ? __ldg(p.gamma + c + i) : 1.0f;
                be[i] = p.beta ? __ldg(p.beta + c + i) : 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < H; ++i) {
            minus_mean[i] = f2_make(m[2 * i], m[2 * i + 1]);
            rstd[i] = f2_make(r[2 * i], r[2 * i + 1]);
            gamma[i] = f2_make(g[2 * i], g[2 * i + 1]);
            beta[i] = f2_make(be[2 * i], be[2 * i + 1]);
        }
    }
    // x -> h, dy -> u
    template <int ACT>
    __device__ __forceinline__ void apply(f2 (&x)[H], f2 (&dy)[H]) const {
#pragma unroll
        for (int i = 0; i < H; ++i) {
            x[i] = f2_mul(f2_add(x[i], minus_mean[i]), rstd[i]);
            dy[i] = activate_grad2<ACT>(f2_add_rounded(f2_mul(x[i], gamma[i]), beta[i]), dy[i]);
        }
    }
};

// (a, b) of a vector's groups, for dx = rstd * (u * gamma - a - h * b).
template <int VEC>
struct GroupMeans {
    static constexpr int H = (VEC + 1) / 2;
    f2 minus_a[H], minus_b[H];
    template <typename F>
    __device__ __forceinline__ void set(int c, int cpg, F&& means) {
        float a[2 * H], b[2 * H];
        const bool one = cpg % VEC == 0;
        const float2 first = means(c);
#pragma unroll
        for (int i = 0; i < 2 * H; ++i) {
            a[i] = b[i] = 0.0f;
            if (i < VEC) {
                const float2 m = one ? first : means(c + i);
                a[i] = -m.x;
                b[i] = -m.y;
            }
        }
#pragma unroll
        for (int i = 0; i < H; ++i) {
            minus_a[i] = f2_make(a[2 * i], a[2 * i + 1]);
            minus_b[i] = f2_make(b[2 * i], b[2 * i + 1]);
        }
    }
    __device__ __forceinline__ void dx(f2 (&h)[H], const f2 (&u)[H], const Grad<VEC>& g) const {
#pragma unroll
        for (int i = 0; i < H; ++i) h[i] = f2_mul(g.rstd[i], f2_fma(h[i], minus_b[i], f2_fma(u[i], g.gamma[i], minus_a[i])));
    }
};

__device__ __forceinline__ float2 stats_of(const NormParams& p, int n, int c) {
    const int s = n * p.G + c / p.cpg;
    return make_float2(__ldg(p.mean + s), __ldg(p.rstd + s));
}

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kNormThreads) norm_apply_kernel(const NormParams p) {
    const int n = blockIdx.x / p.splits, s = blockIdx.x - n * p.splits;
    const int vecs = p.C / VEC;
    const Lanes l = lanes_of(vecs, blockIdx.y + blockIdx.z * gridDim.y);
    if (!l.on) return;
    int p0, p1;
    pixel_range(p, s, p0, p1);
    using Io = VecIo<T, VEC>;
    const long long base = static_cast<long long>(n) * p.P * vecs + l.v;
    const auto* x = reinterpret_cast<const typename Io::Raw*>(p.x) + base;
    auto* y = reinterpret_cast<typename Io::Raw*>(p.y) + base;
    Affine<VEC> f;
    f.load(p, l.v * VEC);
    f.set(l.v * VEC, p.cpg, [&](int c) { return stats_of(p, n, c); });
#pragma unroll 4
    for (int px = p0 + l.r; px < p1; px += l.rows) {
        f2 v[Affine<VEC>::H];
        Io::unpack(x[static_cast<long long>(px) * vecs], v);
        f.template apply<ACT>(v);
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
        const auto value = [&](int v, f2 (&f)[Affine<VEC>::H]) {
            Affine<VEC> af;
            af.load(p, v * VEC);
            af.set(v * VEC, p.cpg, [&](int c) { return stats_of(p, n, c); });
            Io::unpack(x[v], f);
            af.template apply<ACT>(f);
        };
        float top = 0.0f;
        for (int v = lane; v < vecs; v += 32) {
            f2 f[Affine<VEC>::H];
            value(v, f);
#pragma unroll
            for (int i = 0; i < Affine<VEC>::H; ++i) top = magnitude(top, f[i]);
        }
        const RowScale rs = row_scale(warp_max(magnitude_bits(top)));
        if (lane == 0) p.scale[row] = rs.scale;
        for (int v = lane; v < vecs; v += 32) {
            f2 f[Affine<VEC>::H];
            value(v, f);
            quantise_store<VEC>(p.q + row * p.C + v * VEC, f, row_factor(rs.inv));
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
    const Lanes l = lanes_of(vecs, blockIdx.y + blockIdx.z * gridDim.y);
    int p0, p1;
    pixel_range(p, s, p0, p1);
    using Io = VecIo<T, VEC>;
    const long long base = static_cast<long long>(n) * p.P * vecs + l.v;
    const auto* x = reinterpret_cast<const typename Io::Raw*>(p.x) + base;
    const auto* dy = reinterpret_cast<const typename Io::Raw*>(p.dy) + base;
    constexpr int H = Grad<VEC>::H;
    f2 s1[H], s2[H];
#pragma unroll
    for (int i = 0; i < H; ++i) s1[i] = s2[i] = 0;
    if (l.on) {
        Grad<VEC> g;
        g.set(p, l.v * VEC, [&](int c) { return stats_of(p, n, c); });
#pragma unroll 2
        for (int px = p0 + l.r; px < p1; px += l.rows) {
            f2 v[H], d[H];
            Io::unpack(x[static_cast<long long>(px) * vecs], v);
            Io::unpack(dy[static_cast<long long>(px) * vecs], d);
            g.template apply<ACT>(v, d);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                s1[i] = f2_add(s1[i], d[i]);
                s2[i] = f2_fma(d[i], v[i], s2[i]);
            }
        }
    }
    float su[VEC], suh[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        su[i] = i & 1 ? f2_hi(s1[i / 2]) : f2_lo(s1[i / 2]);
        suh[i] = i & 1 ? f2_hi(s2[i / 2]) : f2_lo(s2[i / 2]);
    }
    column_sums<VEC>(su, l, scratch);
    column_sums<VEC>(suh, l, scratch);
    if (l.on && l.r == 0)
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            p.part[static_cast<long long>(blockIdx.x) * p.C + l.v * VEC + i] = make_float2(su[i], suh[i]);
}

// One CTA per (image, group): a and b.
__global__ void __launch_bounds__(kJoinThreads) norm_grad_join_kernel(const NormParams p) {
    __shared__ float scratch[kJoinThreads / 32];
    const int n = blockIdx.x / p.G, g = blockIdx.x - n * p.G;
    const float2* part = p.part + static_cast<long long>(n) * p.splits * p.C + g * p.cpg;
    float a = 0.0f, b = 0.0f;
    for_ranges_and_channels(p, [&](int sp, int c) {
        const float2 v = part[static_cast<long long>(sp) * p.C + c];
        const float gm = p.gamma ? __ldg(p.gamma + g * p.cpg + c) : 1.0f;
        a = fmaf(gm, v.x, a);
        b = fmaf(gm, v.y, b);
    });
    const float total = static_cast<float>(p.P) * static_cast<float>(p.cpg);
    a = block_sum(a, scratch) / total;
    b = block_sum(b, scratch) / total;
    if (threadIdx.x == 0) p.ab[blockIdx.x] = make_float2(a, b);
}

// Sums of partials first, first + STEP, ... of a channel, dgamma's and dbeta's.  Every 256 of them join
// a total that carries its rounding along: one FP32 chain of 2^15 equal terms is off by up to
// 1.5e-4, 256 terms by 3e-6.
struct CarriedSum {
    float total = 0.0f, lost = 0.0f;
    __device__ __forceinline__ void add(float v) {
        const float y = v - lost, t = total + y;
        lost = (t - total) - y;
        total = t;
    }
};

template <int STEP>
__device__ __forceinline__ float2 channel_sum(const float2* part, long long first, long long entries, int C) {
    constexpr int kBatch = 8;  // loads under way, of a short chain too
    CarriedSum u, uh;
    const long long step = static_cast<long long>(STEP) * C;
    part += first * C;
    for (long long left = first < entries ? (entries - first + STEP - 1) / STEP : 0; left > 0; left -= 256) {
        const int count = static_cast<int>(left < 256 ? left : 256);
        float2 s = make_float2(0.0f, 0.0f);
        for (int i = 0; i < count; i += kBatch) {
            float2 v[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k, part += step) v[k] = i + k < count ? *part : make_float2(0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                s.x += v[k].x;
                s.y += v[k].y;
            }
        }
        u.add(s.x);
        uh.add(s.y);
    }
    return make_float2(u.total, uh.total);
}

// dgamma and dbeta over every image and range: 32 channels a CTA, 16 rows of partials at a time.
__global__ void __launch_bounds__(512) norm_grad_channels_kernel(const NormParams p) {
    __shared__ float2 scratch[16][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5;
    const long long entries = static_cast<long long>(p.N) * p.splits;
    float2 s = make_float2(0.0f, 0.0f);
    if (c < p.C) s = channel_sum<16>(p.part + c, r, entries, p.C);
    scratch[r][threadIdx.x & 31] = s;
    __syncthreads();
    if (r == 0 && c < p.C) {
        for (int k = 1; k < 16; ++k) {
            const float2 v = scratch[k][threadIdx.x];
            s.x += v.x;
            s.y += v.y;
        }
        p.dbeta[c] = s.x;
        p.dgamma[c] = s.y;
    }
}

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kNormThreads) norm_grad_apply_kernel(const NormParams p) {
    const int n = blockIdx.x / p.splits, s = blockIdx.x - n * p.splits;
    const int vecs = p.C / VEC;
    const Lanes l = lanes_of(vecs, blockIdx.y + blockIdx.z * gridDim.y);
    if (!l.on) return;
    int p0, p1;
    pixel_range(p, s, p0, p1);
    using Io = VecIo<T, VEC>;
    const long long base = static_cast<long long>(n) * p.P * vecs + l.v;
    const auto* x = reinterpret_cast<const typename Io::Raw*>(p.x) + base;
    const auto* dy = reinterpret_cast<const typename Io::Raw*>(p.dy) + base;
    auto* dx = reinterpret_cast<typename Io::Raw*>(p.y) + base;
    Grad<VEC> g;
    GroupMeans<VEC> gm;
    g.set(p, l.v * VEC, [&](int c) { return stats_of(p, n, c); });
    gm.set(l.v * VEC, p.cpg, [&](int c) { return p.ab[n * p.G + c / p.cpg]; });
#pragma unroll 2
    for (int px = p0 + l.r; px < p1; px += l.rows) {
        f2 v[Grad<VEC>::H], d[Grad<VEC>::H];
        Io::unpack(x[static_cast<long long>(px) * vecs], v);
        Io::unpack(dy[static_cast<long long>(px) * vecs], d);
        g.template apply<ACT>(v, d);
        gm.dx(v, d, g);
        dx[static_cast<long long>(px) * vecs] = Io::pack(v);
    }
}

// ---------------------------------------------------------------- resident form
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

__device__ __forceinline__ uint32_t res_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// The aligned forms: a warp's lanes arrive, and wait, together, whatever loops they left before.
__device__ __forceinline__ void res_cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void res_cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Two floats to the same shared-memory place of cluster CTA `rank`.
__device__ __forceinline__ void res_push(float2* p, uint32_t rank, float2 v) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(v.x), "f"(v.y) : "memory");
}

// Lanes of a vector that share a group, always: the largest power of two that divides cpg, at most
// a vector.  A thread's statistics are joined over them before they leave it.
__host__ __device__ inline int res_lump(const NormParams& p) {
    int l = 1;
    while (l < p.vec && p.cpg % (2 * l) == 0) l *= 2;
    return l;
}

// Rows of backward partials a CTA keeps: one a warp where neighbouring lanes hold several rows of
// a channel and add them up first (2, 4, .. 16 vectors to a pixel), else one a pixel row.
__host__ __device__ inline bool res_warp_rows(int vpr) { return vpr < 32 && (vpr & (vpr - 1)) == 0; }

__host__ __device__ inline int res_groups(const NormParams& p) { return p.chunk / p.cpg; }
__host__ __device__ inline int res_pixels(const NormParams& p) { return (p.P + p.splits - 1) / p.splits; }

// Shared memory of a resident CTA.
struct ResSmem {
    uint4* x;        // the items [items][threads]
    uint4* dy;       // backward: those of dy
    float2* part;    // forward: (mean, M2) [rows][vectors * lumps]; backward: (sum u, sum u h) [rows][chunk]
    float2* recv;    // per group and cluster CTA [groups][kResMaxCluster]
    float2* result;  // per group
    uint32_t* top;   // 8-bit output: a magnitude a pixel
};

template <int MODE>
__host__ __device__ inline int res_part_entries(const NormParams& p) {
    const int vpr = p.chunk / p.vec, rows = kResThreads / vpr;
    if (MODE == kNormBackward) return (res_warp_rows(vpr) ? kResThreads / 32 : rows) * p.chunk;
    return rows * vpr * (p.vec / res_lump(p));
}

template <int MODE>
__host__ __device__ inline size_t res_smem_bytes(const NormParams& p) {
    return static_cast<size_t>(MODE == kNormBackward ? 2 : 1) * p.items * kResThreads * 16 +
           static_cast<size_t>(res_part_entries<MODE>(p)) * 8 + static_cast<size_t>(res_groups(p)) * (kResMaxCluster + 1) * 8 +
           (MODE == kNormInt8 ? static_cast<size_t>(res_pixels(p)) * 4 : 0);
}

template <int MODE>
__device__ __forceinline__ ResSmem res_carve(uint8_t* raw, const NormParams& p) {
    ResSmem s;
    s.x = reinterpret_cast<uint4*>(raw);
    s.dy = s.x + static_cast<size_t>(p.items) * kResThreads;
    s.part = reinterpret_cast<float2*>(MODE == kNormBackward ? s.dy + static_cast<size_t>(p.items) * kResThreads : s.dy);
    s.recv = s.part + res_part_entries<MODE>(p);
    s.result = s.recv + res_groups(p) * kResMaxCluster;
    s.top = reinterpret_cast<uint32_t*>(s.result + res_groups(p));
    return s;
}

// A thread's VEC lanes, (mean, M2) of `cnt` values each, joined in lumps of L and stored.
template <int VEC, int L>
__device__ __forceinline__ void res_store_lumps(int cnt, const float (&mean)[VEC], const float (&m2)[VEC], float2* to) {
    if constexpr (L <= VEC) {
        const float n = static_cast<float>(cnt);
#pragma unroll
        for (int k = 0; k < VEC / L; ++k) {
            float m = 0.0f, q = 0.0f;
#pragma unroll
            for (int i = 0; i < L; ++i) m += mean[k * L + i];
            m *= 1.0f / L;
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const float d = mean[k * L + i] - m;
                q += fmaf(n * d, d, m2[k * L + i]);
            }
            to[k] = make_float2(m, cnt ? q : 0.0f);
        }
    }
}

constexpr int kResBatches = 4;  // commit groups: sums start when a quarter has landed

// (mean, M2) of a CTA's groups from its threads' lanes, a segment of lanes to each group;
// emit(group, value, lanes of the segment).  between() runs after the CTA barrier.
template <int VEC, typename B, typename E>
__device__ __forceinline__ void cta_group_moments(const NormParams& p, int pixels, int vpr, int rows, int r, int v, int mine,
                                                  const float (&mean)[VEC], const float (&m2)[VEC], int groups,
                                                  float2* part, B&& between, E&& emit) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int lump = res_lump(p), width = vpr * (VEC / lump);
    if (r < rows) {
        float2* to = part + r * width + v * (VEC / lump);
        if (lump == 8) res_store_lumps<VEC, 8>(mine, mean, m2, to);
        else if (lump == 4) res_store_lumps<VEC, 4>(mine, mean, m2, to);
        else if (lump == 2) res_store_lumps<VEC, 2>(mine, mean, m2, to);
        else res_store_lumps<VEC, 1>(mine, mean, m2, to);
    }
    __syncthreads();
    between();
    const int per_row = p.cpg / lump, entries = rows * per_row;
    const int wide = segment_width(entries), e0 = lane & (wide - 1);
    const int first_r = per_row == 1 ? e0 : e0 / per_row, first_k = e0 - first_r * per_row;
    const int step_r = per_row == 1 ? wide : wide / per_row, step_k = wide - step_r * per_row;
    const int whole = pixels / rows, more = pixels - whole * rows;  // items of a row: whole, one more in the first `more`
    const float cta = static_cast<float>(pixels) * static_cast<float>(p.cpg);
    const float over = cta > 0.0f ? __frcp_rn(cta) : 0.0f;
    const int at_once = 32 / wide;
    for (int gb = warp * at_once; gb < groups; gb += warps * at_once) {
        const int g = gb + lane / wide;
        const float2* from = part + g * per_row;
        const int end = g < groups ? entries : 0;
        float m = 0.0f, q = 0.0f;
        int er = first_r, ek = first_k;  // an entry's row and lump
        const auto next = [&] {
            er += step_r;
            ek += step_k;
            if (ek >= per_row) {
                ek -= per_row;
                ++er;
            }
        };
        for (int e = e0; e < end; e += wide, next())
            m = fmaf(static_cast<float>((whole + (er < more)) * lump), from[er * width + ek].x, m);
        m = segment_sum(m, wide) * over;
        er = first_r;
        ek = first_k;
        for (int e = e0; e < end; e += wide, next()) {
            const float2 o = from[er * width + ek];
            const float d = o.x - m, cnt = static_cast<float>((whole + (er < more)) * lump);
            if (cnt > 0.0f) q += fmaf(cnt * d, d, o.y);
        }
        q = segment_sum(q, wide);
        if (g < groups) emit(g, make_float2(m, q), wide);
    }
}

// The backward pass's: channel sums (written to `out`, dgamma's and dbeta's partials), then their
// groups' (sum u gamma, sum u h gamma).
template <int VEC, typename B, typename E>
__device__ __forceinline__ void cta_group_grads(const NormParams& p, int vpr, int rows, int r, int v, f2 (&s1)[VEC / 2],
                                                f2 (&s2)[VEC / 2], int groups, int channels, const float* gamma, float2* out,
                                                float2* part, B&& between, E&& emit) {
    constexpr int H = VEC / 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const bool by_warp = res_warp_rows(vpr);
    if (by_warp) {  // the warp's rows of a channel
        for (int o = vpr; o < 32; o <<= 1)
#pragma unroll
            for (int j = 0; j < H; ++j) {
                s1[j] = f2_add(s1[j], __shfl_xor_sync(0xffffffffu, s1[j], o));
                s2[j] = f2_add(s2[j], __shfl_xor_sync(0xffffffffu, s2[j], o));
            }
    }
    const int part_rows = by_warp ? warps : rows;
    if (by_warp ? lane < vpr : r < rows) {
        float4* to = reinterpret_cast<float4*>(part + (by_warp ? warp : r) * channels + v * VEC);
#pragma unroll
        for (int j = 0; j < H; ++j) to[j] = make_float4(f2_lo(s1[j]), f2_lo(s2[j]), f2_hi(s1[j]), f2_hi(s2[j]));
    }
    __syncthreads();
    between();
    const int wide = segment_width(p.cpg), at_once = 32 / wide;
    for (int gfirst = warp * at_once; gfirst < groups; gfirst += warps * at_once) {
        const int g = gfirst + lane / wide;
        float ga = 0.0f, gb = 0.0f;
        for (int i = lane & (wide - 1); i < p.cpg && g < groups; i += wide) {
            const int c = g * p.cpg + i;
            float2 t = make_float2(0.0f, 0.0f);
#pragma unroll 8
            for (int k = 0; k < part_rows; ++k) {
                const float2 o = part[k * channels + c];
                t.x += o.x;
                t.y += o.y;
            }
            if (out != nullptr) out[c] = t;
            const float gm = gamma ? __ldg(gamma + c) : 1.0f;
            ga = fmaf(gm, t.x, ga);
            gb = fmaf(gm, t.y, gb);
        }
        ga = segment_sum(ga, wide);
        gb = segment_sum(gb, wide);
        if (g < groups) emit(g, make_float2(ga, gb), wide);
    }
}

template <typename T, int MODE, int ACT>
__global__ void __launch_bounds__(kResThreads, 2) norm_resident_kernel(const NormParams p) {
    constexpr int VEC = 16 / sizeof(T), H = VEC / 2;
    using Io = VecIo<T, VEC>;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    const ResSmem sm = res_carve<MODE>(smem_raw, p);
    const int rank = p.splits > 1 ? static_cast<int>(res_rank()) : 0;
    const int unit = blockIdx.x / p.splits;
    const int chunks = p.C / p.chunk;
    const int n = unit / chunks;
    const int c0 = (unit - n * chunks) * p.chunk;
    const int vpr = p.chunk / VEC;           // vectors of a pixel
    const int rows = kResThreads / vpr;
    const int r = threadIdx.x / vpr, v = threadIdx.x - r * vpr;
    int p0, p1;
    pixel_range(p, rank, p0, p1);
    const int mine = r < rows && p0 + r < p1 ? (p1 - p0 - r + rows - 1) / rows : 0;  // this thread's items
    const int step = rows * (p.C / VEC);     // in vectors; an image has fewer than 2^31 of them
    const long long base = ((static_cast<long long>(n) * p.P + p0 + r) * p.C + c0) / VEC + v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int batch = (p.items + kResBatches - 1) / kResBatches;
    if (p.splits > 1) res_cluster_arrive();  // this CTA runs: its peers may write to it after their wait below
    const uint4* items = sm.x + threadIdx.x;
    const uint4* items_dy = sm.dy + threadIdx.x;

    {
        const uint4* x = static_cast<const uint4*>(p.x) + base;
        const uint4* dy = static_cast<const uint4*>(p.dy) + base;
        const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(items));
        const uint32_t dst2 = static_cast<uint32_t>(__cvta_generic_to_shared(items_dy));
#pragma unroll
        for (int b = 0; b < kResBatches; ++b) {
            const int end = min((b + 1) * batch, mine);
#pragma unroll 2
            for (int i = b * batch; i < end; ++i) {
                copy_async16(dst + i * (kResThreads * 16), x + i * step);
                if constexpr (MODE == kNormBackward) copy_async16(dst2 + i * (kResThreads * 16), dy + i * step);
            }
            copy_commit();
        }
    }

    const int groups = res_groups(p);
    const int my_c = c0 + (r < rows ? v : 0) * VEC;
    Grad<VEC> grad;
    Affine<VEC> af;
    if constexpr (MODE == kNormBackward) grad.set(p, my_c, [&](int c) { return stats_of(p, n, c); });
    else af.load(p, my_c);
    // `sweep` over the items as their copies land
    const auto sweep_all = [&](auto&& sweep) {
        copy_wait<3>();
        sweep(0, min(batch, mine));
        copy_wait<2>();
        sweep(batch, min(2 * batch, mine));
        copy_wait<1>();
        sweep(2 * batch, min(3 * batch, mine));
        copy_wait<0>();
        sweep(3 * batch, mine);
    };
    // This CTA's sums of group g, to every CTA of the cluster: by the `width` lanes that hold them.
    const auto push = [&](int g, float2 val, int width) {
        for (int k = lane & (width - 1); k < p.splits; k += width) {
            float2* slot = sm.recv + g * kResMaxCluster + rank;
            if (p.splits > 1) res_push(slot, k, val);
            else *slot = val;
        }
    };

    const auto running = [&] {
        if (p.splits > 1) res_cluster_wait();  // every CTA of the cluster runs
    };

    if constexpr (MODE != kNormBackward) {
        Moments<VEC> mo;
        sweep_all([&](int from, int to) {
            f2 f[H];
            if (from == 0 && to > 0) {
                Io::unpack(items[0], f);
                mo.start(f);
            }
#pragma unroll 4
            for (int i = from; i < to; ++i) {
                Io::unpack(items[i * kResThreads], f);
                mo.add(f);
            }
        });
        float mean[VEC], m2[VEC];
        mo.finish(mine, mean, m2);
        cta_group_moments<VEC>(p, p1 - p0, vpr, rows, r, v, mine, mean, m2, groups, sm.part, running, push);
    } else {
        f2 s1[H], s2[H];
#pragma unroll
        for (int i = 0; i < H; ++i) s1[i] = s2[i] = 0;
        sweep_all([&](int from, int to) {
#pragma unroll 2
            for (int i = from; i < to; ++i) {
                f2 f[H], d[H];
                Io::unpack(items[i * kResThreads], f);
                Io::unpack(items_dy[i * kResThreads], d);
                grad.template apply<ACT>(f, d);
#pragma unroll
                for (int j = 0; j < H; ++j) {
                    s1[j] = f2_add(s1[j], d[j]);
                    s2[j] = f2_fma(d[j], f[j], s2[j]);
                }
            }
        });
        float2* out = p.part + (static_cast<long long>(n) * p.splits + rank) * p.C + c0;
        cta_group_grads<VEC>(p, vpr, rows, r, v, s1, s2, groups, p.chunk, p.gamma ? p.gamma + c0 : nullptr,
                             p.dgamma != nullptr ? out : nullptr, sm.part, running, push);
    }

    // The cluster's groups, every CTA for itself in the same order.
    if constexpr (MODE == kNormInt8)
        for (int i = threadIdx.x; i < p1 - p0; i += kResThreads) sm.top[i] = 0;
    if (p.splits > 1) {
        res_cluster_arrive();
        res_cluster_wait();
    } else {
        __syncthreads();
    }
    const float over_total = __frcp_rn(static_cast<float>(p.P) * static_cast<float>(p.cpg));
    const int wide = segment_width(p.splits), at_once = 32 / wide, k = lane & (wide - 1);
    const float cnt = k < p.splits ? static_cast<float>(p.pix_base + (k < p.pix_more)) * static_cast<float>(p.cpg) : 0.0f;
    for (int gfirst = warp * at_once; gfirst < groups; gfirst += kResThreads / 32 * at_once) {
        const int g = gfirst + lane / wide;
        const float2 o = g < groups && k < p.splits ? sm.recv[g * kResMaxCluster + k] : make_float2(0.0f, 0.0f);
        float2 res;
        if constexpr (MODE != kNormBackward) {
            const float m = segment_sum(cnt * o.x, wide) * over_total;
            const float d = o.x - m;
            const float var = segment_sum(cnt > 0.0f ? fmaf(cnt * d, d, o.y) : 0.0f, wide) * over_total;
            res = make_float2(m, __fdiv_rn(1.0f, __fsqrt_rn(var + p.eps)));
            if (rank == 0 && k == 0 && g < groups && p.mean != nullptr) {
                const int s = n * p.G + c0 / p.cpg + g;
                p.mean[s] = res.x;
                p.rstd[s] = res.y;
            }
        } else {
            res = make_float2(segment_sum(o.x, wide) * over_total, segment_sum(o.y, wide) * over_total);
        }
        if (k == 0 && g < groups) sm.result[g] = res;
    }
    __syncthreads();

    const auto result = [&](int c) { return sm.result[(c - c0) / p.cpg]; };
    if constexpr (MODE == kNormForward) {
        af.set(my_c, p.cpg, result);
        uint4* y = static_cast<uint4*>(p.y) + base;
#pragma unroll 4
        for (int i = 0; i < mine; ++i) {
            f2 f[H];
            Io::unpack(items[i * kResThreads], f);
            af.template apply<ACT>(f);
            y[i * step] = Io::pack(f);
        }
    } else if constexpr (MODE == kNormBackward) {
        GroupMeans<VEC> gm;
        gm.set(my_c, p.cpg, result);
        uint4* dx = static_cast<uint4*>(p.y) + base;
#pragma unroll 2
        for (int i = 0; i < mine; ++i) {
            f2 f[H], d[H];
            Io::unpack(items[i * kResThreads], f);
            Io::unpack(items_dy[i * kResThreads], d);
            grad.template apply<ACT>(f, d);
            gm.dx(f, d, grad);
            dx[i * step] = Io::pack(f);
        }
    } else {
        // 8-bit output (chunk = C: whole pixels here).  A pixel on 1, 2, 4, ... 32 neighbouring lanes
        // finds its largest magnitude by shuffles; any other width through shared memory.
        af.set(my_c, p.cpg, result);
        float* scales = p.scale + static_cast<long long>(n) * p.P + p0 + r;
        int8_t* q = p.q + base * VEC;
        const auto value = [&](int i, f2 (&f)[H]) {
            Io::unpack(items[i * kResThreads], f);
            af.template apply<ACT>(f);
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < H; ++j) top = magnitude(top, f[j]);
            return magnitude_bits(top);
        };
        if ((vpr & (vpr - 1)) == 0 && vpr <= 32) {
            const int turns = (p1 - p0 + rows - 1) / rows;
            constexpr int U = 4;  // pixels under way at a time: their shuffles and divisions overlap
            for (int i0 = 0; i0 < turns; i0 += U) {  // every lane of the warp takes part in the shuffles
                f2 f[U][H];
                uint32_t a[U];
#pragma unroll
                for (int u = 0; u < U; ++u) a[u] = i0 + u < mine ? value(i0 + u, f[u]) : 0u;
                if (vpr == 32) {
#pragma unroll
                    for (int u = 0; u < U; ++u) a[u] = warp_max(a[u]);
                } else {
                    for (int o = 1; o < vpr; o <<= 1)
#pragma unroll
                        for (int u = 0; u < U; ++u) a[u] = max(a[u], __shfl_xor_sync(0xffffffffu, a[u], o));
                }
                RowFactor rf[U];
                if (vpr >= U) {
                    const float own = row_factors<U>(a, v, vpr, rf);
                    if (v < U && i0 + v < mine) scales[(i0 + v) * rows] = own;
                } else {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const RowScale rs = row_scale(a[u]);
                        rf[u] = row_factor(rs.inv);
                        if (v == 0 && i0 + u < mine) scales[(i0 + u) * rows] = rs.scale;
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i0 + u < mine) quantise_store<VEC>(q + static_cast<long long>((i0 + u) * step) * VEC, f[u], rf[u]);
            }
        } else {
            for (int i = 0; i < mine; ++i) {
                f2 f[H];
                atomicMax(sm.top + r + i * rows, value(i, f));
            }
            __syncthreads();
            for (int i = 0; i < mine; ++i) {
                f2 f[H];
                value(i, f);
                const RowScale rs = row_scale(sm.top[r + i * rows]);
                quantise_store<VEC>(q + static_cast<long long>(i * step) * VEC, f, row_factor(rs.inv));
                if (v == 0) scales[i * rows] = rs.scale;
            }
        }
    }
}

// ---------------------------------------------------------------- two passes
constexpr int kTwoBatch = 4;  // vectors a thread has under way (of each tensor)

__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ uint4 load_last(const uint4* p) { return __ldcs(p); }  // not needed again
__device__ __forceinline__ void store_past(uint4* p, uint4 v) { __stcs(p, v); }

// Where a CTA of either pass stands: pixel range `s` of image n, all channels.
struct TwoRange {
    int n, s, vpr, rows, r, v, p0, p1, mine;
    long long base;  // in vectors; an image has fewer than 2^31 of them
    int step;
    __device__ __forceinline__ TwoRange(const NormParams& p, int block, int VEC) {
        n = block / p.splits;
        s = block - n * p.splits;
        vpr = p.C / VEC;
        rows = kNormThreads / vpr;
        r = threadIdx.x / vpr;
        v = threadIdx.x - r * vpr;
        pixel_range(p, s, p0, p1);
        mine = r < rows && p0 + r < p1 ? (p1 - p0 - r + rows - 1) / rows : 0;
        base = (static_cast<long long>(n) * p.P + p0 + r) * vpr + v;
        step = rows * vpr;
    }
};

// A thread's vectors of one or two tensors, in order, through slots of shared memory that only it
// writes and reads: kSlots - 1 of each are on their way at any time, whatever the arithmetic does
// (four at a time in registers, waited for together: backward 32 x 112 x 112 x 128 111 us, 97 so).
constexpr int kSlots = 8;  // a power of two

template <int TENSORS>
struct RangeStream {
    const uint4* from[TENSORS];
    uint4* slots;  // [kSlots][TENSORS][threads], from this thread's on
    long long step;
    int count;

    __device__ __forceinline__ void fetch(int i) {
        if (i < count) {
#pragma unroll
            for (int t = 0; t < TENSORS; ++t) {
                copy_async16(static_cast<uint32_t>(__cvta_generic_to_shared(&slots[((i & (kSlots - 1)) * TENSORS + t) * kNormThreads])), from[t]);
                from[t] += step;
            }
        }
        copy_commit();
    }
    __device__ __forceinline__ void start() {
#pragma unroll
        for (int i = 0; i < kSlots - 1; ++i) fetch(i);
    }
    // take(vectors, first) for each; a slot is filled again one turn after it was read.
    template <typename F>
    __device__ __forceinline__ void run(F&& take) {
#pragma unroll 2
        for (int i = 0; i < count; ++i) {
            copy_wait<kSlots - 2>();
            uint4 raw[TENSORS];
#pragma unroll
            for (int t = 0; t < TENSORS; ++t) raw[t] = slots[((i & (kSlots - 1)) * TENSORS + t) * kNormThreads];
            fetch(i + kSlots - 1);
            take(raw, i == 0);
        }
        copy_wait<0>();
    }
};

// First pass.  Forward: (mean, M2) of the range's groups; backward: (sum u gamma, sum u h gamma) of
// them and the channels' (sum u, sum u h).
template <typename T, int MODE, int ACT>
__global__ void __launch_bounds__(kNormThreads, MODE == kNormBackward ? 3 : 4) norm_range_sums_kernel(const NormParams p) {
    constexpr int VEC = 16 / sizeof(T), H = VEC / 2;
    using Io = VecIo<T, VEC>;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    float2* part = reinterpret_cast<float2*>(smem_raw);
    const TwoRange t(p, blockIdx.x, VEC);
    const int lane = threadIdx.x & 31;
    constexpr int kTensors = MODE == kNormBackward ? 2 : 1;
    RangeStream<kTensors> stream;
    stream.from[0] = static_cast<const uint4*>(p.x) + t.base;
    if constexpr (MODE == kNormBackward) stream.from[1] = static_cast<const uint4*>(p.dy) + t.base;
    stream.step = t.step;
    stream.count = t.mine;
    stream.slots = reinterpret_cast<uint4*>(smem_raw) + threadIdx.x;
    stream.start();
    launch_dependents();
    if constexpr (MODE != kNormBackward) {
        Moments<VEC> mo;
        f2 f[H];
        stream.run([&](const uint4 (&raw)[1], bool first) {
            Io::unpack(raw[0], f);
            if (first) mo.start(f);
            mo.add(f);
        });
        float mean[VEC], m2[VEC];
        mo.finish(t.mine, mean, m2);
        __syncthreads();  // the slots are the partial sums' place from here
        const auto store = [&](int g, float2 val, int wide) {
            if ((lane & (wide - 1)) == 0) p.part[(static_cast<long long>(t.n) * p.G + g) * p.splits + t.s] = val;
        };
        cta_group_moments<VEC>(p, t.p1 - t.p0, t.vpr, t.rows, t.r, t.v, t.mine, mean, m2, p.G, part, [] {}, store);
    } else {
        Grad<VEC> grad;
        grad.set(p, (t.r < t.rows ? t.v : 0) * VEC, [&](int c) { return stats_of(p, t.n, c); });
        f2 s1[H], s2[H];
#pragma unroll
        for (int j = 0; j < H; ++j) s1[j] = s2[j] = 0;
        stream.run([&](const uint4 (&raw)[2], bool) {
            f2 f[H], d[H];
            Io::unpack(raw[0], f);
            Io::unpack(raw[1], d);
            grad.template apply<ACT>(f, d);
#pragma unroll
            for (int j = 0; j < H; ++j) {
                s1[j] = f2_add(s1[j], d[j]);
                s2[j] = f2_fma(d[j], f[j], s2[j]);
            }
        });
        __syncthreads();  // the slots are the partial sums' place from here
        float2* out = p.part + (static_cast<long long>(t.n) * p.splits + t.s) * p.C;
        const auto store = [&](int g, float2 val, int wide) {
            if ((lane & (wide - 1)) == 0) p.ab[(static_cast<long long>(t.n) * p.G + g) * p.splits + t.s] = val;
        };
        cta_group_grads<VEC>(p, t.vpr, t.rows, t.r, t.v, s1, s2, p.G, p.C, p.gamma, p.dgamma != nullptr ? out : nullptr,
                             part, [] {}, store);
    }
}

// One group of an image from its ranges, by `width` threads of which this is the k-th: (mean, rstd),
// or the backward pass's (a, b).  sum() adds over those threads.
template <int MODE, typename F>
__device__ __forceinline__ float2 join_ranges(const NormParams& p, int n, int g, int k0, int width, F&& sum) {
    const float over_total = __frcp_rn(static_cast<float>(p.P) * static_cast<float>(p.cpg));
    const float2* from = (MODE == kNormBackward ? p.ab : p.part) + (static_cast<long long>(n) * p.G + g) * p.splits;
    const int end = g < p.G ? p.splits : 0;
    if constexpr (MODE == kNormBackward) {
        float a = 0.0f, b = 0.0f;
        for (int k = k0; k < end; k += width) {
            a += from[k].x;
            b += from[k].y;
        }
        a = sum(a);
        return make_float2(a * over_total, sum(b) * over_total);
    } else {
        const float each = static_cast<float>(p.pix_base) * static_cast<float>(p.cpg);
        const float one_more = static_cast<float>(p.pix_base + 1) * static_cast<float>(p.cpg);
        float m = 0.0f, q = 0.0f;
        for (int k = k0; k < end; k += width) m = fmaf(k < p.pix_more ? one_more : each, from[k].x, m);
        m = sum(m) * over_total;
        for (int k = k0; k < end; k += width) {
            const float2 o = from[k];
            const float d = o.x - m;
            q += fmaf((k < p.pix_more ? one_more : each) * d, d, o.y);
        }
        const float var = sum(q) * over_total;
        return make_float2(m, __fdiv_rn(1.0f, __fsqrt_rn(var + p.eps)));
    }
}

__device__ __forceinline__ long long norm_ab_of(const NormParams& p) { return static_cast<long long>(p.N) * p.G * p.splits; }

// Many ranges an image (few images): joined once, a CTA to each group, instead of by every CTA of the
// second pass (608 ranges of 1 x 512 x 512 x 128: 94 MB of partials read again, 48 us of 70).
template <int MODE>
__global__ void __launch_bounds__(128) norm_range_join_kernel(const NormParams p) {
    __shared__ float scratch[4];
    launch_dependents();
    wait_for_previous();
    const int n = blockIdx.x / p.G, g = blockIdx.x - n * p.G;
    const float2 res = join_ranges<MODE>(p, n, g, threadIdx.x, 128, [&](float v) { return block_sum(v, scratch); });
    if (threadIdx.x == 0) {
        if constexpr (MODE == kNormBackward) {
            p.ab[norm_ab_of(p) + blockIdx.x] = res;
        } else {
            p.mean[blockIdx.x] = res.x;
            p.rstd[blockIdx.x] = res.y;
        }
    }
}

// Second pass.  Joins the ranges of the image's groups, then writes the range backwards.  Backward:
// the first `extra` CTAs write dgamma and dbeta instead, 32 channels each.
template <typename T, int MODE, int ACT>
__global__ void __launch_bounds__(kNormThreads, MODE == kNormForward ? 4 : 3) norm_range_apply_kernel(const NormParams p, int extra) {
    constexpr int VEC = 16 / sizeof(T), H = VEC / 2;
    using Io = VecIo<T, VEC>;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    float2* joined = reinterpret_cast<float2*>(smem_raw);  // [G]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (MODE == kNormBackward && static_cast<int>(blockIdx.x) < extra) {
        wait_for_previous();
        const int c = blockIdx.x * 32 + lane;
        const long long entries = static_cast<long long>(p.N) * p.splits;
        float2 sum = make_float2(0.0f, 0.0f);
        if (c < p.C) sum = channel_sum<kNormThreads / 32>(p.part + c, warp, entries, p.C);
        joined[warp * 32 + lane] = sum;
        __syncthreads();
        if (warp == 0 && c < p.C) {
            for (int k = 1; k < kNormThreads / 32; ++k) {
                sum.x += joined[k * 32 + lane].x;
                sum.y += joined[k * 32 + lane].y;
            }
            p.dbeta[c] = sum.x;
            p.dgamma[c] = sum.y;
        }
        return;
    }
    const TwoRange t(p, blockIdx.x - (MODE == kNormBackward ? extra : 0), VEC);
    const int my_c = (t.r < t.rows ? t.v : 0) * VEC;
    const uint4* x = static_cast<const uint4*>(p.x) + t.base;
    Affine<VEC> af;
    Grad<VEC> grad;
    if constexpr (MODE == kNormBackward) grad.set(p, my_c, [&](int c) { return stats_of(p, t.n, c); });
    else af.load(p, my_c);
    wait_for_previous();
    if (p.joined) {
        for (int g = threadIdx.x; g < p.G; g += kNormThreads)
            joined[g] = MODE == kNormBackward ? p.ab[norm_ab_of(p) + t.n * p.G + g]
                                              : make_float2(p.mean[t.n * p.G + g], p.rstd[t.n * p.G + g]);
    } else {
        const int wide = segment_width(p.splits), at_once = 32 / wide;
        for (int gfirst = warp * at_once; gfirst < p.G; gfirst += kNormThreads / 32 * at_once) {
            const int g = gfirst + lane / wide;
            const float2 res = join_ranges<MODE>(p, t.n, g, lane & (wide - 1), wide, [&](float v) { return segment_sum(v, wide); });
            if ((lane & (wide - 1)) == 0 && g < p.G) {
                joined[g] = res;
                if (MODE != kNormBackward && t.s == 0 && p.mean != nullptr) {
                    p.mean[t.n * p.G + g] = res.x;
                    p.rstd[t.n * p.G + g] = res.y;
                }
            }
        }
    }
    __syncthreads();
    const auto result = [&](int c) { return joined[c / p.cpg]; };
    if constexpr (MODE == kNormForward) {
        af.set(my_c, p.cpg, result);
        uint4* y = static_cast<uint4*>(p.y) + t.base;
        const long long step = t.step;
        const auto put = [&](const uint4& raw, int i) {
            f2 f[H];
            Io::unpack(raw, f);
            af.template apply<ACT>(f);
            store_past(y + i * step, Io::pack(f));
        };
        constexpr int B = kTwoBatch;
        for (int i = t.mine; i > 0; i -= B) {
            uint4 raw[B];
#pragma unroll
            for (int k = 0; k < B; ++k)
                if (i > k) raw[k] = load_last(x + (i - 1 - k) * step);
#pragma unroll
            for (int k = 0; k < B; ++k)
                if (i > k) put(raw[k], i - 1 - k);
        }
    } else if constexpr (MODE == kNormBackward) {
        GroupMeans<VEC> gm;
        gm.set(my_c, p.cpg, result);
        const uint4* dy = static_cast<const uint4*>(p.dy) + t.base;
        uint4* dx = static_cast<uint4*>(p.y) + t.base;
        const auto put = [&](const uint4& a, const uint4& b, int i) {
            f2 f[H], d[H];
            Io::unpack(a, f);
            Io::unpack(b, d);
            grad.template apply<ACT>(f, d);
            gm.dx(f, d, grad);
            store_past(dx + static_cast<unsigned>(i * t.step), Io::pack(f));
        };
        constexpr int B = kTwoBatch / 2;
        for (int i = t.mine; i > 0; i -= B) {
            uint4 a[B], b[B];
#pragma unroll
            for (int k = 0; k < B; ++k)
                if (i > k) {
                    a[k] = load_last(x + static_cast<unsigned>((i - 1 - k) * t.step));
                    b[k] = load_last(dy + static_cast<unsigned>((i - 1 - k) * t.step));
                }
#pragma unroll
            for (int k = 0; k < B; ++k)
                if (i > k) put(a[k], b[k], i - 1 - k);
        }
    } else {
        // A pixel on 1, 2, 4, ... 32 neighbouring lanes finds its largest magnitude by shuffles, any
        // other width through shared memory; four pixels under way at a time.
        af.set(my_c, p.cpg, result);
        constexpr int U = 4;
        float* scales = p.scale + static_cast<long long>(t.n) * p.P + t.p0 + t.r;
        const bool by_lanes = (t.vpr & (t.vpr - 1)) == 0 && t.vpr <= 32;
        uint32_t* top = reinterpret_cast<uint32_t*>(joined + p.G);  // [2][U][rows]
        if (!by_lanes) {
            for (int i = threadIdx.x; i < 2 * U * t.rows; i += kNormThreads) top[i] = 0;
            __syncthreads();
        }
        const int turns = (t.p1 - t.p0 + t.rows - 1) / t.rows;
        int buf = 0;
        for (int i0 = ((turns - 1) / U) * U; i0 >= 0; i0 -= U, buf ^= 1) {
            uint4 raw[U];
            f2 f[U][H];
            uint32_t a[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u < t.mine) raw[u] = load_last(x + static_cast<unsigned>((i0 + u) * t.step));
#pragma unroll
            for (int u = 0; u < U; ++u) {
                a[u] = 0;
                if (i0 + u >= t.mine) continue;
                Io::unpack(raw[u], f[u]);
                af.template apply<ACT>(f[u]);
                float m = 0.0f;
#pragma unroll
                for (int j = 0; j < H; ++j) m = magnitude(m, f[u][j]);
                a[u] = magnitude_bits(m);
            }
            if (!by_lanes) {
                uint32_t* row = top + buf * U * t.rows + t.r;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i0 + u < t.mine) atomicMax(row + u * t.rows, a[u]);
                __syncthreads();
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i0 + u < t.mine) a[u] = row[u * t.rows];
                // the other buffer was read before this barrier: clear it for the next turn
                for (int i = threadIdx.x; i < U * t.rows; i += kNormThreads) top[(buf ^ 1) * U * t.rows + i] = 0;
                __syncthreads();
            } else if (t.vpr == 32) {
#pragma unroll
                for (int u = 0; u < U; ++u) a[u] = warp_max(a[u]);
            } else {
                for (int o = 1; o < t.vpr; o <<= 1)
#pragma unroll
                    for (int u = 0; u < U; ++u) a[u] = max(a[u], __shfl_xor_sync(0xffffffffu, a[u], o));
            }
            RowFactor rf[U];
            if (by_lanes && t.vpr >= U) {
                const float own = row_factors<U>(a, t.v, t.vpr, rf);
                if (t.v < U && i0 + t.v < t.mine) scales[(i0 + t.v) * t.rows] = own;
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const RowScale rs = row_scale(a[u]);
                    rf[u] = row_factor(rs.inv);
                    if (t.v == 0 && i0 + u < t.mine) scales[(i0 + u) * t.rows] = rs.scale;
                }
            }
            int8_t* q = p.q + t.base * VEC;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u < t.mine) quantise_store<VEC>(q + static_cast<long long>((i0 + u) * t.step) * VEC, f[u], rf[u]);
        }
    }
}

// ---------------------------------------------------------------- launch
template <typename F>
void with_types(const NormParams& p, F&& f) {
    if (p.bf16) {
        if (p.vec == 8) f(__nv_bfloat16(), std::integral_constant<int, 8>());
        else if (p.vec == 4) f(__nv_bfloat16(), std::integral_constant<int, 4>());
        else if (p.vec == 2) f(__nv_bfloat16(), std::integral_constant<int, 2>());
        else f(__nv_bfloat16(), std::integral_constant<int, 1>());
    } else {
        if (p.vec == 4) f(float(), std::integral_constant<int, 4>());
        else if (p.vec == 2) f(float(), std::integral_constant<int, 2>());
        else f(float(), std::integral_constant<int, 1>());
    }
}

template <typename F>
void with_act(int act, F&& f) {
    if (act == CONV_ACT_RELU) f(std::integral_constant<int, CONV_ACT_RELU>());
    else if (act == CONV_ACT_SILU) f(std::integral_constant<int, CONV_ACT_SILU>());
    else f(std::integral_constant<int, CONV_ACT_NONE>());
}

// Pixel ranges, and blocks of channels in two dimensions: either ends at 65,535.
dim3 stream_grid(const NormParams& p) {
    const int vecs = p.C / p.vec;
    const int cv = vecs < kNormThreads ? vecs : kNormThreads;
    const unsigned blocks = static_cast<unsigned>((vecs - 1) / cv + 1), z = (blocks + 65534) / 65535;
    return dim3(static_cast<unsigned>(p.N) * p.splits, (blocks + z - 1) / z, z);
}

}  // namespace

namespace {

// Each kernel with its one record of the shared-memory limit, which is set once, to all that a block may
// have: a limit set to each map's need, by the launches and by the occupancy query on records of their own, sank
// below what the query counted on after a smaller map had run, and between two threads below what the other launches.
template <typename T, int MODE, int ACT>
SmemLimitCache& resident_limits() {
    static SmemLimitCache limits;
    return limits;
}

template <typename T, int MODE, int ACT, typename F>
void with_limits(F&& f) {
    f(norm_resident_kernel<T, MODE, ACT>, resident_limits<T, MODE, ACT>());
}

template <typename F>
void with_resident(const NormParams& p, int mode, F&& f) {
    with_act(p.act, [&](auto act) {
        constexpr int A = decltype(act)::value;
        const auto with_mode = [&](auto t) {
            using T = decltype(t);
            if (mode == kNormForward) with_limits<T, kNormForward, A>(f);
            else if (mode == kNormInt8) with_limits<T, kNormInt8, A>(f);
            else with_limits<T, kNormBackward, A>(f);
        };
        if (p.bf16) with_mode(__nv_bfloat16());
        else with_mode(float());
    });
}

size_t resident_smem(const NormParams& p, int mode) {
    return mode == kNormForward ? res_smem_bytes<kNormForward>(p)
                                : (mode == kNormInt8 ? res_smem_bytes<kNormInt8>(p) : res_smem_bytes<kNormBackward>(p));
}

template <typename K>
cudaError_t resident_config(K* fn, SmemLimitCache& limits, const NormParams& p, int mode, cudaStream_t stream,
                            cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attr)[1]) {
    const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(fn), p.smem_optin, limits);
    cfg = cudaLaunchConfig_t();
    cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(p.N) * (p.C / p.chunk) * p.splits));
    cfg.blockDim = dim3(kResThreads);
    cfg.dynamicSmemBytes = p.smem_bytes;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.splits;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.splits > 1 ? 1 : 0;
    return e;
}

cudaError_t launch_resident(const NormParams& p, int mode, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    with_resident(p, mode, [&](auto* fn, SmemLimitCache& limits) {
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute attr[1];
        e = resident_config(fn, limits, p, mode, stream, cfg, attr);
        if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, fn, p);
    });
    return e;
}

}  // namespace

// Channels a unit takes and CTAs that share it (the 8-bit output needs whole pixels).  A map of few
// pixels takes as many channels as one CTA holds, two to an SM (backward: 64 KB of x and dy, since
// its sums a channel grow with them), while that leaves half a unit an SM: 128 x 14 x 14 x 1024
// BF16 33 us, 84 at 64 bytes a pixel; 256 x 8 x 8 x 512 17 and 68, backward 29 and 63.  A larger one
// takes up to 64 bytes a pixel (128 make clusters of 16, of which a GPC holds fewer: 32 x 112 x 112 x 256
// BF16, SiLU, took 113 us with 128, 97 with 64, 122 with 32) and the fewest CTAs that hold it
// two to an SM, then one to an SM.  More CTAs while there are fewer than SMs.
void norm_pick_resident(NormParams& p, int mode, int num_sms) {
    const int es = p.bf16 ? 2 : 4, tensors = mode == kNormBackward ? 2 : 1;
    p.chunk = 0;
    if (p.vec * es != 16 || static_cast<long long>(p.P) * (p.C / p.vec) >= (1LL << 31)) return;
    NormParams t = p;
    const auto rows_of = [&](int chunk) { return kResThreads / (chunk / p.vec); };
    const auto fits = [&](int chunk, int cluster, int limit) {
        t.chunk = chunk;
        t.splits = cluster;
        const int pixels = res_pixels(t);
        t.items = (pixels + rows_of(chunk) - 1) / rows_of(chunk);
        if (static_cast<double>(t.items) * tensors * kResThreads * 16 > limit) return false;
        t.smem_bytes = static_cast<int>(resident_smem(t, mode));
        return t.smem_bytes <= limit;
    };
    const int half = p.smem_optin / 2 - 1024;  // of an SM, less what a CTA needs besides
    int chunk = 0;
    if (mode == kNormInt8) {
        chunk = p.C;
    } else {
        const long long room = mode == kNormBackward ? 64 * 1024 : half;
        for (int g = 1; g <= p.G; ++g) {  // whole groups that divide the channels and make whole vectors
            const int c = g * p.cpg;
            if (p.G % g != 0 || c % p.vec != 0) continue;
            if (chunk != 0 && c / p.vec > kResThreads) break;
            if (chunk == 0 || c * es <= 64 ||
                (2LL * p.N * (p.C / c) >= num_sms && fits(c, 1, half) && 16LL * tensors * t.items * kResThreads <= room))
                chunk = c;
        }
    }
    if (chunk == 0 || chunk / p.vec > kResThreads) return;
    const int rows = rows_of(chunk);
    const long long units = static_cast<long long>(p.N) * (p.C / chunk);
    int best = 0;
    for (int limit : {half, p.smem_optin}) {
        for (int cluster = 1; cluster <= kResMaxCluster && best == 0; ++cluster)
            if (fits(chunk, cluster, limit)) best = cluster;
        if (best != 0) break;
    }
    if (best == 0 || units * best > 0x7fffffffLL) return;
    while (2 * best <= kResMaxCluster && units * best * 2 <= num_sms && p.P >= 2 * best * rows) best *= 2;
    fits(chunk, best, p.smem_optin);
    t.pix_base = t.P / best;
    t.pix_more = t.P % best;
    p = t;
}

// Whether the resident form (at_a_time clusters on the device) beats two passes, where both can run.
// A GPC holds few large clusters, so the last of two or three rounds of them leaves much idle,
// and two CTAs an SM of 100 KB each take long when the SMs are not full of them; two passes pay a second
// read of x, a launch and their joins.  Pairs: resident, two passes, microseconds, cold caches, BF16,
// SiLU, 32 groups.
bool norm_resident_pays(const NormParams& p, int mode, int at_a_time, int num_sms) {
    const long long units = static_cast<long long>(p.N) * (p.C / p.chunk);
    const int es = p.bf16 ? 2 : 4, tensors = mode == kNormBackward ? 2 : 1;
    const long long held = 16LL * tensors * p.items * kResThreads;  // bytes a CTA holds
    const bool one_round = units <= at_a_time;
    if (mode == kNormForward) {
        // 4 x 160 x 160 x 128 (16 CTAs, 1.1 rounds) 31 and 26, 12 x 160 x 160 x 128 (3.4) 58 and 50,
        // 8 x 200 x 200 x 128 (12 CTAs, 4.0) 74 and 51; of one round, 2 x 160 x 160 x 64 17 and 22.
        if (p.splits > 8 && !one_round) return false;
        // 16 x 96 x 96 x 128 (6 CTAs, 1.4 rounds) 33 and 32; of eight 32 x 112 x 112 x 128 (3.6) 64 and 62,
        // 32 x 112 x 112 x 256 (7.1) 106 and 111.
        return p.splits <= 4 || one_round || units > 2LL * at_a_time;
    }
    if (mode == kNormInt8) {
        // Pixel-wide units.  Up to 48 KB a CTA: 2 x 16 x 16 x 128 13 and 13, 4 x 32 x 32 x 128 15 and 16;
        // 105 KB of 10 CTAs: 1 x 32 x 32 x 512 21 and 14; 208 KB: 4 x 56 x 56 x 320 36 and 24; of 16 CTAs
        // 64 x 56 x 56 x 256 93 and 70.  Many units of at most eight CTAs: 256 x 56 x 56 x 64 91 and 105,
        // 128 x 28 x 28 x 512 95 and 103; too few of them for the SMs: 16 x 32 x 32 x 320 31 and 27.
        return held <= 48 * 1024 || (p.splits <= 8 && units * p.splits > num_sms);
    }
    // Small maps of few channels, where the joins are short: 4 x 56 x 56 x 64 17 and 17 (in a graph, x and dy in
    // L2, 10.8 and 11.6); larger, 8 x 56 x 56 x 64 FP32, 19 and 21 (10 and 15); of more channels
    // 4 x 32 x 32 x 512 19 and 22.
    if (p.C <= 128 && static_cast<double>(p.N) * p.P * p.C * es <= 4e6) return false;
    // Clusters of a dozen in one round that fills the SMs, 1 x 96 x 96 x 512 25 and 28; in 1.4 rounds 8 x 96 x 96 x 128
    // 38 and 37, of 200 KB a CTA 4 x 128 x 128 x 128 44 and 32, of sixteen 32 x 112 x 112 x 128 138 and 109.
    if (p.splits > 8) return one_round && 3 * units >= at_a_time && held > 64 * 1024 && held <= 112 * 1024;
    // Between two and three rounds 16 x 64 x 64 x 256 (2.2) 50 and 44, 32 x 64 x 64 x 128 (2.2) 52 and 42,
    // 24 x 56 x 56 x 256 (2.6) 52 and 50, 20 x 64 x 64 x 256 (2.8) 55 and 51, but 100 x 28 x 28 x 256 (2.6, single CTAs)
    // 48 and 50.  Up to two: 48 x 28 x 28 x 256 (1.3) 31 and 31 (in a graph 21 and 24), 12 x 64 x 64 x 128 FP32 (1.7)
    // 33 and 31, 16 x 56 x 56 x 256 (1.7) 40 and 37 (28 and 30).  Past three they are close: 64 x 28 x 28 x 512 (3.4)
    // 56 and 60, 32 x 56 x 56 x 256 (3.5) 61 and 58, 40 x 56 x 56 x 256 (4.3) 74 and 71, 64 x 56 x 56 x 256 (6.9) 108 and 108.
    return units <= 2LL * at_a_time || units > 3LL * at_a_time;
}

// Two passes: pixel ranges that fill the SMs once, four CTAs to each (three backward or to 8 bits).
void norm_pick_two_pass(NormParams& p, int mode, int num_sms) {
    const int vecs = p.C / p.vec;
    if (p.vec * (p.bf16 ? 2 : 4) != 16 || vecs > kNormThreads || static_cast<long long>(p.P) * vecs >= (1LL << 31)) return;
    const int rows = kNormThreads / vecs;
    long long splits = static_cast<long long>(num_sms) * (mode == kNormForward ? 4 : 3) / p.N;
    const long long most = p.P / (2LL * rows);  // two pixels a thread at least
    if (splits > most) splits = most;
    p.two_pass = 1;
    p.splits = static_cast<int>(splits < 1 ? 1 : splits);
    p.joined = p.splits > 64;
    p.pix_base = p.P / p.splits;
    p.pix_more = p.P % p.splits;
}

int norm_resident_at_a_time(const NormParams& p, int mode, int num_sms) {
    int clusters = 0;
    with_resident(p, mode, [&](auto* fn, SmemLimitCache& limits) {
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute attr[1];
        if (resident_config(fn, limits, p, mode, nullptr, cfg, attr) != cudaSuccess ||
            cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
            (p.splits > 1 && cudaOccupancyMaxActiveClusters(&clusters, fn, &cfg) != cudaSuccess)) {
            cudaGetLastError();
            clusters = 0;
        } else if (p.splits == 1) {
            clusters = 2 * num_sms;
        }
    });
    return clusters;
}

// Partials of channels (or, forward in two passes, of groups), then per group and range, then the
// statistics of the form that joins them in a kernel of its own.
size_t norm_workspace_bytes(const NormParams& p) {
    return norm_part_entries(p) * sizeof(float2) + norm_ab_entries(p) * sizeof(float2) +
           2 * static_cast<size_t>(p.N) * p.G * sizeof(float);
}

size_t norm_part_entries(const NormParams& p) { return static_cast<size_t>(p.N) * p.splits * p.C; }
size_t norm_ab_entries(const NormParams& p) { return static_cast<size_t>(p.N) * p.G * (p.two_pass ? p.splits + p.joined : 1); }

namespace {

template <int MODE>
int range_sums_smem(const NormParams& p) {
    const int vpr = p.C / p.vec, rows = kNormThreads / vpr;
    const int entries = MODE == kNormBackward ? (res_warp_rows(vpr) ? kNormThreads / 32 : rows) * p.C
                                              : rows * vpr * (p.vec / res_lump(p));
    const int slots = kSlots * (MODE == kNormBackward ? 2 : 1) * kNormThreads * 16;
    return entries * 8 > slots ? entries * 8 : slots;  // the partial sums, 16 KB at most, take the slots' place
}

template <typename T, int MODE, int ACT>
SmemLimitCache& sums_limits() {
    static SmemLimitCache limits;
    return limits;
}

template <int MODE>
cudaError_t launch_two_pass(const NormParams& p, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    const unsigned grid = static_cast<unsigned>(p.N) * p.splits;
    const int extra = MODE == kNormBackward && p.dgamma != nullptr ? (p.C + 31) / 32 : 0;
    const int vpr = p.C / p.vec, rows = kNormThreads / vpr;
    const int joined = p.G * 8 + (MODE == kNormInt8 ? 2 * 4 * rows * 4 : 0);
    const int apply_smem = joined > kNormThreads * 8 ? joined : kNormThreads * 8;
    const auto run = [&](auto* sums, SmemLimitCache& limits, auto* apply) {
        e = ensure_smem_limit(reinterpret_cast<const void*>(sums), range_sums_smem<MODE>(p), limits);
        if (e != cudaSuccess) return;
        sums<<<grid, kNormThreads, range_sums_smem<MODE>(p), stream>>>(p);
        e = cudaGetLastError();
        if (e != cudaSuccess) return;
        cudaLaunchConfig_t cfg = {};
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (p.joined) {
            cfg.gridDim = dim3(static_cast<unsigned>(p.N) * p.G);
            cfg.blockDim = dim3(128);
            e = cudaLaunchKernelEx(&cfg, norm_range_join_kernel<MODE == kNormBackward ? kNormBackward : kNormForward>, p);
            if (e != cudaSuccess) return;
        }
        cfg.gridDim = dim3(grid + extra);
        cfg.blockDim = dim3(kNormThreads);
        cfg.dynamicSmemBytes = apply_smem;
        e = cudaLaunchKernelEx(&cfg, apply, p, extra);
    };
    with_act(p.act, [&](auto act) {
        constexpr int A = decltype(act)::value;
        constexpr int SA = MODE == kNormBackward ? A : static_cast<int>(CONV_ACT_NONE);  // forward sums need no activation
        constexpr int SM = MODE == kNormBackward ? kNormBackward : kNormForward;
        if (p.bf16)
            run(norm_range_sums_kernel<__nv_bfloat16, SM, SA>, sums_limits<__nv_bfloat16, SM, SA>(), norm_range_apply_kernel<__nv_bfloat16, MODE, A>);
        else
            run(norm_range_sums_kernel<float, SM, SA>, sums_limits<float, SM, SA>(), norm_range_apply_kernel<float, MODE, A>);
    });
    return e;
}

}  // namespace

cudaError_t launch_norm_forward(const NormParams& p, int num_sms, cudaStream_t stream) {
    if (p.chunk != 0) return launch_resident(p, p.q != nullptr ? kNormInt8 : kNormForward, stream);
    if (p.two_pass) return p.q != nullptr ? launch_two_pass<kNormInt8>(p, stream) : launch_two_pass<kNormForward>(p, stream);
    const dim3 grid = stream_grid(p);
    with_types(p, [&](auto t, auto vec) {
        norm_moments_kernel<decltype(t), vec.value><<<grid, kNormThreads, 0, stream>>>(p);
    });
    norm_join_kernel<<<p.N * p.G, kJoinThreads, 0, stream>>>(p);
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

cudaError_t launch_norm_backward(const NormParams& p, cudaStream_t stream) {
    if (p.chunk != 0) {
        const cudaError_t e = launch_resident(p, kNormBackward, stream);
        if (e != cudaSuccess) return e;
        if (p.dgamma != nullptr) norm_grad_channels_kernel<<<(p.C + 31) / 32, 512, 0, stream>>>(p);
        return cudaGetLastError();
    }
    if (p.two_pass) return launch_two_pass<kNormBackward>(p, stream);
    const dim3 grid = stream_grid(p);
    with_types(p, [&](auto t, auto vec) {
        with_act(p.act, [&](auto act) {
            norm_grad_sums_kernel<decltype(t), vec.value, act.value><<<grid, kNormThreads, 0, stream>>>(p);
            norm_grad_join_kernel<<<p.N * p.G, kJoinThreads, 0, stream>>>(p);
            if (p.dgamma != nullptr) norm_grad_channels_kernel<<<(p.C + 31) / 32, 512, 0, stream>>>(p);
            norm_grad_apply_kernel<decltype(t), vec.value, act.value><<<grid, kNormThreads, 0, stream>>>(p);
        });
    });
    return cudaGetLastError();
}

}  // namespace convgb
