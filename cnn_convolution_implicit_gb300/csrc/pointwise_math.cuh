// pointwise_math.cuh -- what the normalisation and 8-bit product kernels share:
// typed vector accesses, packed FP32 arithmetic, the activations with their
// derivatives, and the 8-bit row quantiser.
//
// Two FP32 values travel as one 64-bit register pair (f2) through the packed
// add, multiply and fused multiply-add, each lane rounded as the scalar operation
// rounds it.  These kernels move about six BF16 values per clock and SM at the memory's
// rate, which leaves 21 instructions a value; packing is what keeps them below that.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "../../include/conv.h"

namespace convgb {

using f2 = unsigned long long;

__device__ __forceinline__ f2 f2_make(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ f2 f2_dup(float v) { return f2_make(v, v); }
__device__ __forceinline__ void f2_split(f2 v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ float f2_lo(f2 v) {
    float a, b;
    f2_split(v, a, b);
    return a;
}
__device__ __forceinline__ float f2_hi(f2 v) {
    float a, b;
    f2_split(v, a, b);
    return b;
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// a + b after a product that has to round by itself: the packed add may be fused with the multiply
// before it (it was: rint(x * inv) came out of the unrounded product), the scalar one is not.
__device__ __forceinline__ f2 f2_add_rounded(f2 a, f2 b) {
    return f2_make(__fadd_rn(f2_lo(a), f2_lo(b)), __fadd_rn(f2_hi(a), f2_hi(b)));
}

// VEC consecutive elements as pairs of FP32, one access of 2 to 16 bytes; VEC = 1: one pair, its
// second lane 0.
template <typename T, int VEC>
struct VecIo;

template <>
struct VecIo<__nv_bfloat16, 8> {
    using Raw = uint4;
    static __device__ __forceinline__ f2 pair(uint32_t u) {  // a BF16 is the upper half of an FP32
        return f2_make(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
    static __device__ __forceinline__ void unpack(const uint4& r, f2 (&v)[4]) {
        v[0] = pair(r.x);
        v[1] = pair(r.y);
        v[2] = pair(r.z);
        v[3] = pair(r.w);
    }
    static __device__ __forceinline__ uint32_t round(f2 v) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f2_lo(v), f2_hi(v));
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ uint4 pack(const f2 (&v)[4]) {
        return make_uint4(round(v[0]), round(v[1]), round(v[2]), round(v[3]));
    }
};

template <>
struct VecIo<float, 4> {
    using Raw = uint4;
    static __device__ __forceinline__ void unpack(const uint4& r, f2 (&v)[2]) {
        v[0] = f2_make(__uint_as_float(r.x), __uint_as_float(r.y));
        v[1] = f2_make(__uint_as_float(r.z), __uint_as_float(r.w));
    }
    static __device__ __forceinline__ uint4 pack(const f2 (&v)[2]) {
        return make_uint4(__float_as_uint(f2_lo(v[0])), __float_as_uint(f2_hi(v[0])), __float_as_uint(f2_lo(v[1])),
                          __float_as_uint(f2_hi(v[1])));
    }
};

template <>
struct VecIo<__nv_bfloat16, 4> {
    using Raw = uint2;
    static __device__ __forceinline__ void unpack(const uint2& r, f2 (&v)[2]) {
        v[0] = VecIo<__nv_bfloat16, 8>::pair(r.x);
        v[1] = VecIo<__nv_bfloat16, 8>::pair(r.y);
    }
    static __device__ __forceinline__ uint2 pack(const f2 (&v)[2]) {
        return make_uint2(VecIo<__nv_bfloat16, 8>::round(v[0]), VecIo<__nv_bfloat16, 8>::round(v[1]));
    }
};

template <>
struct VecIo<__nv_bfloat16, 2> {
    using Raw = uint32_t;
    static __device__ __forceinline__ void unpack(const uint32_t& r, f2 (&v)[1]) { v[0] = VecIo<__nv_bfloat16, 8>::pair(r); }
    static __device__ __forceinline__ uint32_t pack(const f2 (&v)[1]) { return VecIo<__nv_bfloat16, 8>::round(v[0]); }
};

template <>
struct VecIo<float, 2> {
    using Raw = uint2;
    static __device__ __forceinline__ void unpack(const uint2& r, f2 (&v)[1]) {
        v[0] = f2_make(__uint_as_float(r.x), __uint_as_float(r.y));
    }
    static __device__ __forceinline__ uint2 pack(const f2 (&v)[1]) {
        return make_uint2(__float_as_uint(f2_lo(v[0])), __float_as_uint(f2_hi(v[0])));
    }
};

template <>
struct VecIo<__nv_bfloat16, 1> {
    using Raw = __nv_bfloat16;
    static __device__ __forceinline__ void unpack(const __nv_bfloat16& r, f2 (&v)[1]) { v[0] = f2_make(__bfloat162float(r), 0.0f); }
    static __device__ __forceinline__ __nv_bfloat16 pack(const f2 (&v)[1]) { return __float2bfloat16_rn(f2_lo(v[0])); }
};

template <>
struct VecIo<float, 1> {
    using Raw = float;
    static __device__ __forceinline__ void unpack(const float& r, f2 (&v)[1]) { v[0] = f2_make(r, 0.0f); }
    static __device__ __forceinline__ float pack(const f2 (&v)[1]) { return f2_lo(v[0]); }
};

// A sum of many terms that carries its rounding along.  (What is lost next to an Inf is no number, and not carried.)
struct CarriedSum {
    float total = 0.0f, lost = 0.0f;
    __device__ __forceinline__ void add(float v) {
        const float y = v - lost, t = total + y;
        lost = isinf(t) ? 0.0f : (t - total) - y;
        total = t;
    }
};

// ------------------------------------------------------------------ activations
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN passes through
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// 1 / (1 + exp(-z)).  z = -inf gives 0, NaN stays NaN.  The rounding of z log2 e grows with |z|, and with
// it the error where exp(-z) rules: up to 3 * 2^-24 of the value for z > -3, 8 for z > -10, 27 for
// z > -30, 62 at -85 (activate() alike).  What is lost there is below 1e-11 absolute.
__device__ __forceinline__ f2 sigmoid2(f2 z) {
    const f2 t = f2_mul(z, f2_dup(-1.4426950408889634f));  // exp(-z) = 2^(-z log2 e)
    float a, b;
    f2_split(t, a, b);
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
    f2_split(f2_add(f2_make(a, b), f2_dup(1.0f)), a, b);
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
    return f2_make(a, b);
}

template <int ACT>
__device__ __forceinline__ float activate(float z) {
    if constexpr (ACT == CONV_ACT_RELU) return max_nan(z, 0.0f);
    if constexpr (ACT == CONV_ACT_SILU) return __fdividef(z, 1.0f + __expf(-z));
    return z;
}

template <int ACT>
__device__ __forceinline__ f2 activate2(f2 z) {
    if constexpr (ACT == CONV_ACT_RELU) return f2_make(max_nan(f2_lo(z), 0.0f), max_nan(f2_hi(z), 0.0f));
    if constexpr (ACT == CONV_ACT_SILU) return f2_mul(z, sigmoid2(z));
    return z;
}

// d act(z) / dz times `up`.  ReLU: 0 at z = 0; a NaN or Inf upstream stays visible.
template <int ACT>
__device__ __forceinline__ f2 activate_grad2(f2 z, f2 up) {
    if constexpr (ACT == CONV_ACT_RELU)
        return f2_mul(up, f2_make(f2_lo(z) > 0.0f ? 1.0f : 0.0f, f2_hi(z) > 0.0f ? 1.0f : 0.0f));
    if constexpr (ACT == CONV_ACT_SILU) {
        const f2 s = sigmoid2(z), one = f2_dup(1.0f);
        const f2 rest = f2_fma(s, f2_dup(-1.0f), one);  // 1 - s
        return f2_mul(up, f2_mul(s, f2_fma(z, rest, one)));
    }
    return up;
}

// ------------------------------------------------------------------ 8-bit rows
// A row's largest magnitude travels as the bits of |x|: as unsigned integers they order as the
// values do, Inf above every number and NaN above Inf, so one maximum finds both the scale and
// a row that is not finite.
__device__ __forceinline__ float max_magnitude(float a, float b) {  // |.| of the larger, its sign of no account
    float r;
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float magnitude(float top, f2 v) {
    return max_magnitude(max_magnitude(top, f2_lo(v)), f2_hi(v));
}
__device__ __forceinline__ uint32_t magnitude_bits(float top) { return __float_as_uint(top) & 0x7fffffffu; }

struct RowScale {
    float scale;  // what one step of q stands for
    float inv;    // q = rint(x * inv); 0 where every q of the row is 0
};

// scale = amax / 127, inv = 127 / amax, both rounded once.  Rows below 2^-100 count as zero
// (127 / amax would overflow); a row with a NaN or an Inf gets scale NaN and q = 0, so
// that every product of it is NaN.
__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits) {
    const float amax = __uint_as_float(amax_bits);
    if (amax_bits >= 0x7f800000u) return {__uint_as_float(0x7fc00000u), 0.0f};
    if (amax < 7.888609052e-31f) return {0.0f, 0.0f};  // 2^-100
    return {__fdiv_rn(amax, 127.0f), __fdiv_rn(127.0f, amax)};
}

struct RowFactor {
    float inv;
    uint32_t keep;  // all ones, or 0 where every q of the row is 0 (its values may be NaN)
};

__device__ __forceinline__ RowFactor row_factor(float inv) { return {inv, inv != 0.0f ? ~0u : 0u}; }

// Factors of R rows whose magnitudes every lane of a segment holds: lane r of it works out row r's
// (the two divisions once for all rows) and hands the factor round; it returns its own row's
// scale.  lane: within the segment, of `width` lanes (a power of two, R at least).
template <int R>
__device__ __forceinline__ float row_factors(const uint32_t (&top)[R], int lane, int width, RowFactor (&f)[R]) {
    uint32_t mine = top[0];
#pragma unroll
    for (int r = 1; r < R; ++r) mine = lane == r ? top[r] : mine;
    const RowScale own = row_scale(mine);
#pragma unroll
    for (int r = 0; r < R; ++r) f[r] = row_factor(__shfl_sync(0xffffffffu, own.inv, r, width));
    return own.scale;
}

// Four values to four bytes, the first in the low one.  |x * inv| <= 127 up to one rounding; adding
// 1.5 * 2^23 rounds it to an integer (ties to even), whose low byte is then the sum's.
__device__ __forceinline__ uint32_t quantise4(f2 a, f2 b, const RowFactor& r) {
    const f2 inv = f2_dup(r.inv), magic = f2_dup(12582912.0f);
    a = f2_add_rounded(f2_mul(a, inv), magic);
    b = f2_add_rounded(f2_mul(b, inv), magic);
    const uint32_t lo = __byte_perm(__float_as_uint(f2_lo(a)), __float_as_uint(f2_hi(a)), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(f2_lo(b)), __float_as_uint(f2_hi(b)), 0x0040);
    return __byte_perm(lo, hi, 0x5410) & r.keep;
}

__device__ __forceinline__ int8_t quantise1(float x, const RowFactor& r) {
    return static_cast<int8_t>(__float2int_rn(__fmul_rn(x, r.inv)) & r.keep);
}

// A vector's 8-bit values to q.
template <int VEC>
__device__ __forceinline__ void quantise_store(int8_t* q, const f2 (&v)[(VEC + 1) / 2], const RowFactor& r) {
    if constexpr (VEC == 8) *reinterpret_cast<uint2*>(q) = make_uint2(quantise4(v[0], v[1], r), quantise4(v[2], v[3], r));
    else if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(q) = quantise4(v[0], v[1], r);
    else if constexpr (VEC == 2) *reinterpret_cast<uint16_t*>(q) = static_cast<uint16_t>(quantise4(v[0], v[0], r));
    else *q = quantise1(f2_lo(v[0]), r);
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }

}  // namespace convgb
