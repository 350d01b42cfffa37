// dropout.cu -- y = dropped(x) / (1 - p) + residual, the mask drawn from Philox 4x32 of ten rounds.
//
// The generator is the published one (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as
// 1, 2, 3", SC 2011): a block of four words is a bijection of its counter under its key, so any
// thread finds any element's word without the others'.  A 16-byte vector takes one block (FP32) or two
// (BF16).
//
// Bound by memory in FP32 and next to it in BF16, where ten rounds of two 64-bit products for every four values
// take about as long as the bytes (8192 x 4096 BF16 with a residual 34 us, 5.9 TB/s; without one 30 us, and 23 with a
// single round).  Hence the keys of the rounds and what of the first two does not depend on the low word of the
// counter are worked out once a thread (39 us without that), and eight CTAs an SM hide the loads.
#include "pointwise_math.cuh"
#include "rows_internal.h"

namespace convgb {

namespace {

constexpr int kDropThreads = 256;

constexpr uint32_t kMul0 = 0xD2511F53u, kMul1 = 0xCD9E8D57u, kKey0 = 0x9E3779B9u, kKey1 = 0xBB67AE85u;

__device__ __forceinline__ unsigned long long wide(uint32_t a, uint32_t b) { return static_cast<unsigned long long>(a) * b; }
__device__ __forceinline__ uint32_t high(unsigned long long v) { return static_cast<uint32_t>(v >> 32); }
__device__ __forceinline__ uint32_t low(unsigned long long v) { return static_cast<uint32_t>(v); }

// The generator for one key and offset.  A round takes (c0, c1, c2, c3) to (hi(c2 m1) ^ c1 ^ k0, lo(c2 m1),
// hi(c0 m0) ^ c3 ^ k1, lo(c0 m0)), the counter being (low, high, offset low, offset high).
struct Philox {
    uint2 key[10];
    uint32_t offset_lo, offset_hi;
    uint32_t counter_hi;            // the words below are for this one
    uint32_t lo1, hi2, lo2;         // lo(c2 m1) of round 1; hi ^ key and lo of round 2's c0 m0

    __device__ __forceinline__ void start(unsigned long long seed, unsigned long long offset) {
#pragma unroll
        for (int i = 0; i < 10; ++i) key[i] = make_uint2(low(seed) + i * kKey0, high(seed) + i * kKey1);
        offset_lo = low(offset);
        offset_hi = high(offset);
        set_counter_high(0);
    }
    __device__ __forceinline__ void set_counter_high(uint32_t h) {
        counter_hi = h;
        const unsigned long long b = wide(offset_lo, kMul1), a = wide(high(b) ^ h ^ key[0].x, kMul0);
        lo1 = low(b);
        hi2 = high(a) ^ key[1].y;
        lo2 = low(a);
    }
    __device__ __forceinline__ uint4 block(unsigned long long i) {
        if (high(i) != counter_hi) set_counter_high(high(i));
        const unsigned long long a1 = wide(low(i), kMul0), b2 = wide(high(a1) ^ offset_hi ^ key[0].y, kMul1);
        uint4 c = make_uint4(high(b2) ^ lo1 ^ key[1].x, low(b2), hi2 ^ low(a1), lo2);
#pragma unroll
        for (int r = 2; r < 10; ++r) {
            const unsigned long long a = wide(c.x, kMul0), b = wide(c.z, kMul1);
            c = make_uint4(high(b) ^ c.y ^ key[r].x, low(b), high(a) ^ c.w ^ key[r].y, low(a));
        }
        return c;
    }
};

struct Draw {
    Philox generator;
    uint32_t threshold;
    float scale;
    bool none_left;

    // Elements 4 i .. 4 i + 3: kept or 0, plus what is added.
    __device__ __forceinline__ void four(unsigned long long i, f2& a, f2& b, f2 ra, f2 rb) {
        const uint4 w = generator.block(i);
        a = f2_make(one(w.x, f2_lo(a), f2_lo(ra)), one(w.y, f2_hi(a), f2_hi(ra)));
        b = f2_make(one(w.z, f2_lo(b), f2_lo(rb)), one(w.w, f2_hi(b), f2_hi(rb)));
    }
    __device__ __forceinline__ float one(uint32_t word, float x, float r) const {
        return word >= threshold && !none_left ? fmaf(x, scale, r) : r;
    }
};

template <typename T, bool RES>
__global__ void __launch_bounds__(kDropThreads, 8) dropout_kernel(const DropoutParams p) {
    constexpr int V = 16 / sizeof(T), H = V / 2;
    Draw d;
    d.generator.start(p.state[0], p.state[1]);
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
