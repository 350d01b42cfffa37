// int8_rows.cuh -- loads from 8-bit matrices whose rows may start on any byte.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace convgb {

// 16 bytes of a row from byte `at` of a matrix of `total` bytes, zero from `len` on (1..16 bytes
// are wanted): the one or two aligned granules that hold the bytes, shifted.  A granule that
// the matrix ends in is read byte by byte, so nothing past its last byte is touched.
__device__ __forceinline__ uint4 granule(const int8_t* base, long long g, long long total) {
    const long long at = g << 4;
    if (at + 16 <= total) return __ldg(reinterpret_cast<const uint4*>(base + at));
    uint32_t v[4] = {0, 0, 0, 0};
    for (int i = 0; i < 16; ++i)
        if (at + i < total) v[i >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(base[at + i])) << (8 * (i & 3));
    return make_uint4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ uint4 load_item(const int8_t* base, long long at, int len, long long total) {
    const long long g = at >> 4;
    const int off = static_cast<int>(at & 15);
    const uint4 a = granule(base, g, total);
    const uint4 b = off + len > 16 ? granule(base, g + 1, total) : make_uint4(0, 0, 0, 0);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    const int word = off >> 2, shift = (off & 3) * 8;
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t lo = 0, hi = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // word is 0..3: a select per word keeps w in registers
            lo = word == j ? w[i + j] : lo;
            hi = word == j ? w[i + j + 1] : hi;
        }
        const int left = len - 4 * i;
        const uint32_t v = __funnelshift_r(lo, hi, shift);
        r[i] = left >= 4 ? v : (left <= 0 ? 0u : v & ((1u << (8 * left)) - 1u));
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

}  // namespace convgb
