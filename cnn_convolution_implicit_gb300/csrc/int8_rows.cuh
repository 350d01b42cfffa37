// int8_rows.cuh -- loads from 8-bit matrices whose rows may start on any byte, and their values in FP16.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace convgb {

// Loads of an operand.  LATE: the kernel before this one, still running when this one starts
// (programmatic launch), writes it.  The non-coherent path is only for memory that nothing writes
// while the grid runs, and the compiler may move such a load across the wait for that kernel, so
// LATE data takes ordinary loads that stay behind it.
template <bool LATE>
__device__ __forceinline__ uint4 load16(const uint4* p) {
    if constexpr (!LATE) return __ldg(p);
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ float load1_late(const float* p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
    return v;
}

// 16 bytes of a row from byte `at` of a matrix of `total` bytes, zero from `len` on (1..16 bytes
// are wanted): the one or two aligned granules that hold the bytes, shifted.  A granule that
// the matrix ends in is read byte by byte, so nothing past its last byte is touched.
static __device__ __noinline__ uint4 last_granule(const int8_t* base, long long g, long long total) {
    const long long at = g << 4;
    uint32_t v[4] = {0, 0, 0, 0};
    for (int i = 0; i < 16; ++i)
        if (at + i < total) v[i >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(base[at + i])) << (8 * (i & 3));
    return make_uint4(v[0], v[1], v[2], v[3]);
}

template <bool LATE>
__device__ __forceinline__ uint4 granule(const int8_t* base, long long g, long long total) {
    if ((g << 4) + 16 <= total) return load16<LATE>(reinterpret_cast<const uint4*>(base) + g);
    return last_granule(base, g, total);
}

// 16 bytes from byte `off` of two neighbouring granules: by two words, by one, by bytes, in selects, which
// keep the words in registers.
__device__ __forceinline__ uint4 shift_granules(const uint4& a, const uint4& b, int off) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t two[6], one[5], r[4];
#pragma unroll
    for (int i = 0; i < 6; ++i) two[i] = off & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) one[i] = off & 4 ? two[i + 1] : two[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __funnelshift_r(one[i], one[i + 1], (off & 3) * 8);
    return make_uint4(r[0], r[1], r[2], r[3]);
}

__device__ __forceinline__ uint4 first_bytes(uint4 v, int len) {  // zero from len on
    if (len >= 16) return v;
    uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int left = len - 4 * i;
        r[i] = left >= 4 ? r[i] : (left <= 0 ? 0u : r[i] & ((1u << (8 * left)) - 1u));
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

template <bool LATE = false>
__device__ __forceinline__ uint4 load_item(const int8_t* base, long long at, int len, long long total) {
    const long long g = at >> 4;
    const int off = static_cast<int>(at & 15);
    uint4 a, b;
    if ((g << 4) + 32 <= total) {  // both lie in the matrix, wanted or not
        const uint4* from = reinterpret_cast<const uint4*>(base) + g;
        a = load16<LATE>(from);
        b = load16<LATE>(from + 1);
    } else {
        a = granule<LATE>(base, g, total);
        b = off + len > 16 ? granule<LATE>(base, g + 1, total) : make_uint4(0, 0, 0, 0);
    }
    return first_bytes(shift_granules(a, b, off), len);
}

// Rows of at most 32 P vectors of 16 bytes, one to a warp: lane l gets vectors l, l + 32, ... of the
// row that starts at byte `at` of the matrix.  Every granule is read once, into lane order; the next
// one's bytes come from the lane beside.  First all of a row's loads, then the shifts.
template <int P>
struct StraddlingRow {
    uint4 after;  // lane 0: the granule past the warp's 32 P
    int off, bytes;

    __device__ __forceinline__ void load(const int8_t* base, long long at, int row_bytes, long long total, int lane, uint4 (&raw)[P]) {
        off = static_cast<int>(at & 15);
        bytes = row_bytes;
        const long long first = at >> 4;
        const int granules = (off + bytes + 15) >> 4;
#pragma unroll
        for (int h = 0; h < P; ++h) raw[h] = one(base, first + lane + 32 * h, total, lane + 32 * h < granules);
        after = one(base, first + 32 * P, total, lane == 0 && 32 * P < granules);
    }

    __device__ __forceinline__ void shift(int lane, uint4 (&raw)[P]) const {
#pragma unroll
        for (int h = 0; h < P; ++h) {
            const uint4 n = h + 1 < P ? raw[h + 1 < P ? h + 1 : 0] : after;
            const uint4 give = lane == 0 ? n : raw[h];
            uint4 b;
            b.x = __shfl_sync(0xffffffffu, give.x, (lane + 1) & 31);
            b.y = __shfl_sync(0xffffffffu, give.y, (lane + 1) & 31);
            b.z = __shfl_sync(0xffffffffu, give.z, (lane + 1) & 31);
            b.w = __shfl_sync(0xffffffffu, give.w, (lane + 1) & 31);
            const int left = bytes - 16 * (lane + 32 * h);
            raw[h] = first_bytes(shift_granules(raw[h], b, off), left < 0 ? 0 : left);
        }
    }

private:
    static __device__ __forceinline__ uint4 one(const int8_t* base, long long g, long long total, bool on) {
        if (!on) return make_uint4(0, 0, 0, 0);
        if ((g << 4) + 16 <= total) return __ldcs(reinterpret_cast<const uint4*>(base) + g);
        return last_granule(base, g, total);
    }
};

// Four 8-bit integers to FP16.
__device__ __forceinline__ uint2 to_half4(uint32_t v) {
    const uint32_t u = v ^ 0x80808080u;
    uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140);  // bytes 0, 1 below 0x64
    uint32_t hi = __byte_perm(u, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(0x64806480u));  // 1152
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(0x64806480u));
    return make_uint2(lo, hi);
}

}  // namespace convgb
