// pointwise_math.cuh -- what the normalisation and 8-bit product kernels share:
// typed vector loads and stores, the activations with their derivatives, and the
// 8-bit row quantiser.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "../../include/conv.h"

namespace convgb {

// VEC consecutive elements as FP32.  VEC = 16 bytes of T (one 128-bit access) or 1.
template <typename T, int VEC>
struct VecIo;

template <>
struct VecIo<__nv_bfloat16, 8> {
    using Raw = uint4;
    static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[8]) {
        const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);  // a BF16 is the upper half of an FP32
            v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};

template <>
struct VecIo<float, 4> {
    using Raw = uint4;
    static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[4]) {
        v[0] = __uint_as_float(r.x);
        v[1] = __uint_as_float(r.y);
        v[2] = __uint_as_float(r.z);
        v[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
};

template <>
struct VecIo<__nv_bfloat16, 1> {
    using Raw = __nv_bfloat16;
    static __device__ __forceinline__ void unpack(const __nv_bfloat16& r, float (&v)[1]) { v[0] = __bfloat162float(r); }
    static __device__ __forceinline__ __nv_bfloat16 pack(const float (&v)[1]) { return __float2bfloat16_rn(v[0]); }
};

template <>
struct VecIo<float, 1> {
    using Raw = float;
    static __device__ __forceinline__ void unpack(const float& r, float (&v)[1]) { v[0] = r; }
    static __device__ __forceinline__ float pack(const float (&v)[1]) { return v[0]; }
};

// 1 / (1 + exp(-z)): two MUFU operations, about 2 ulp.  z = -inf gives 0, NaN stays NaN.
__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

template <int ACT>
__device__ __forceinline__ float activate(float z) {
    if constexpr (ACT == CONV_ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);  // NaN passes through
    if constexpr (ACT == CONV_ACT_SILU) return __fdividef(z, 1.0f + __expf(-z));
    return z;
}

// d act(z) / dz times `up`.  ReLU: 0 at z = 0.
template <int ACT>
__device__ __forceinline__ float activate_grad(float z, float up) {
    if constexpr (ACT == CONV_ACT_RELU) return z > 0.0f ? up : up * 0.0f;  // a NaN or Inf upstream stays visible
    if constexpr (ACT == CONV_ACT_SILU) {
        const float s = sigmoid(z);
        return up * (s * (1.0f + z * (1.0f - s)));
    }
    return up;
}

// ------------------------------------------------------------------ 8-bit rows
// A row's largest magnitude is taken over the bit patterns of |x|: as unsigned
// integers they order as the values do, and Inf and NaN come out on top, so one
// maximum finds both the scale and a row that is not finite.
__device__ __forceinline__ uint32_t magnitude_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

struct RowScale {
    float scale;  // what one step of q stands for
    float inv;    // q = rint(x * inv)
};

// scale = amax / 127, inv = 127 / amax, both rounded once.  Rows below 2^-100 count as zero
// (127 / amax would overflow); a row with a NaN or an Inf gets scale NaN and q = 0, so
// that every product of it is NaN.
__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits) {
    RowScale r;
    const float amax = __uint_as_float(amax_bits);
    if (amax_bits >= 0x7f800000u) {
        r.scale = __uint_as_float(0x7fc00000u);
        r.inv = 0.0f;
    } else if (amax < 7.888609052e-31f) {  // 2^-100
        r.scale = 0.0f;
        r.inv = 0.0f;
    } else {
        r.scale = __fdiv_rn(amax, 127.0f);
        r.inv = __fdiv_rn(127.0f, amax);
    }
    return r;
}

__device__ __forceinline__ int quantise(float x, float inv) {
    // |x * inv| <= 127 up to one rounding, and rint brings that back to 127; a row that is not
    // finite has inv = 0 (Inf * 0 is NaN, which the conversion turns into 0).
    return __float2int_rn(__fmul_rn(x, inv));
}

// Four 8-bit values in one word, the first in the low byte.
__device__ __forceinline__ uint32_t pack_int8x4(int a, int b, int c, int d) {
    return (a & 0xff) | ((b & 0xff) << 8) | ((c & 0xff) << 16) | (static_cast<uint32_t>(d) << 24);
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }

}  // namespace convgb
