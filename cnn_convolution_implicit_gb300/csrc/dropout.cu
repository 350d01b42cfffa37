// dropout.cu -- y = dropped(x) / (1 - p) + residual, the mask drawn from Philox 4x32 of ten rounds.
//
// The generator is the published one (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as
// 1, 2, 3", SC 2011): a block of four words is a bijection of its counter under its key, so any
// thread finds any element's word without the others'.  A 16-byte vector takes one block (FP32) or two
// (BF16).
#include "pointwise_math.cuh"
#include "rows_internal.h"

namespace convgb {

namespace {

constexpr int kDropThreads = 256;

// One round on (c0, c1, c2, c3) takes two 32 x 32 -> 64-bit products.
__device__ __forceinline__ uint4 philox(uint4 c, uint2 key) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const unsigned long long a = static_cast<unsigned long long>(c.x) * 0xD2511F53u;
        const unsigned long long b = static_cast<unsigned long long>(c.z) * 0xCD9E8D57u;
        c = make_uint4(static_cast<uint32_t>(b >> 32) ^ c.y ^ key.x, static_cast<uint32_t>(b),
                       static_cast<uint32_t>(a >> 32) ^ c.w ^ key.y, static_cast<uint32_t>(a));
        key.x += 0x9E3779B9u;
        key.y += 0xBB67AE85u;
    }
    return c;
}

struct Draw {
    uint2 key, offset;
    uint32_t threshold;
    float scale;
    bool none_left;

    // Elements 4 i .. 4 i + 3: kept or 0, plus what is added.
    __device__ __forceinline__ void four(unsigned long long i, f2& a, f2& b, f2 ra, f2 rb) const {
        const uint4 w = philox(make_uint4(static_cast<uint32_t>(i), static_cast<uint32_t>(i >> 32), offset.x, offset.y), key);
        a = f2_make(one(w.x, f2_lo(a), f2_lo(ra)), one(w.y, f2_hi(a), f2_hi(ra)));
        b = f2_make(one(w.z, f2_lo(b), f2_lo(rb)), one(w.w, f2_hi(b), f2_hi(rb)));
    }
    __device__ __forceinline__ float one(uint32_t word, float x, float r) const {
        return word >= threshold && !none_left ? fmaf(x, scale, r) : r;
    }
};

template <typename T, bool RES>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(const DropoutParams p) {
    constexpr int V = 16 / sizeof(T), H = V / 2;
    const unsigned long long seed = p.state[0], offset = p.state[1];
    Draw d;
    d.key = make_uint2(static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32));
    d.offset = make_uint2(static_cast<uint32_t>(offset), static_cast<uint32_t>(offset >> 32));
    d.threshold = p.threshold;
    d.scale = p.scale;
    d.none_left = p.none_left != 0;
    const T* x = static_cast<const T*>(p.x);
    const T* r = static_cast<const T*>(p.r);
    T* y = static_cast<T*>(p.y);
    const unsigned long long vecs = p.n / V;
    for (unsigned long long v = blockIdx.x * static_cast<unsigned long long>(kDropThreads) + threadIdx.x; v < vecs;
         v += static_cast<unsigned long long>(gridDim.x) * kDropThreads) {
        f2 f[H], g[H] = {};
        const uint4 raw = __ldcs(reinterpret_cast<const uint4*>(x) + v);
        if constexpr (RES) VecIo<T, V>::unpack(__ldcs(reinterpret_cast<const uint4*>(r) + v), g);
        VecIo<T, V>::unpack(raw, f);
#pragma unroll
        for (int j = 0; j < H / 2; ++j) d.four(v * (V / 4) + j, f[2 * j], f[2 * j + 1], g[2 * j], g[2 * j + 1]);
        reinterpret_cast<uint4*>(y)[v] = VecIo<T, V>::pack(f);
    }
    // the last elements, fewer than a vector, one a thread
    const unsigned long long i = vecs * V + threadIdx.x;
    if (blockIdx.x == 0 && threadIdx.x < V && i < p.n) {
        f2 a, b, g = 0;
        VecIo<T, 1>::unpack(x[i], *reinterpret_cast<f2(*)[1]>(&a));
        if constexpr (RES) VecIo<T, 1>::unpack(r[i], *reinterpret_cast<f2(*)[1]>(&g));
        a = b = f2_dup(f2_lo(a));
        g = f2_dup(f2_lo(g));
        d.four(i / 4, a, b, g, g);
        const int k = static_cast<int>(i % 4);
        const f2 out[1] = {f2_dup(k == 0 ? f2_lo(a) : (k == 1 ? f2_hi(a) : (k == 2 ? f2_lo(b) : f2_hi(b))))};
        y[i] = VecIo<T, 1>::pack(out);
    }
}

template <typename T>
cudaError_t launch(const DropoutParams& p, int num_sms, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    const unsigned long long need = (p.n / V + kDropThreads - 1) / kDropThreads, most = 8ULL * num_sms;
    const unsigned grid = static_cast<unsigned>(need == 0 ? 1 : (need < most ? need : most));
    if (p.r != nullptr) dropout_kernel<T, true><<<grid, kDropThreads, 0, stream>>>(p);
    else dropout_kernel<T, false><<<grid, kDropThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dropout(const DropoutParams& p, int num_sms, cudaStream_t stream) {
    return p.bf16 ? launch<__nv_bfloat16>(p, num_sms, stream) : launch<float>(p, num_sms, stream);
}

}  // namespace convgb
