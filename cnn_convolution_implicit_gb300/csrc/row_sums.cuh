// row_sums.cuh -- sums over the rows (dgamma, dbias): how long a chain of FP32 additions may get, and the join of parts.
//
// One chain of n equal terms is off by up to n / 2 * 2^-24 of its sum (10^4 of them by 1.5e-4 where measured, 512 by 5e-6), so
// a thread adds up to 512 rows: with more of them there are more CTAs, whose parts meet here.
#pragma once

#include "pointwise_math.cuh"

namespace convgb {

constexpr int kChainRows = 512;

// A kernel that keeps a thread's columns over all the rows its CTA takes, `at_once` of them side by side, `resident` CTAs at a
// time: rounds of CTAs, one where that leaves the chains short enough.
inline int chain_rounds(int M, int at_once, int resident) {
    const long long rows = static_cast<long long>(resident) * at_once * kChainRows;
    return static_cast<int>((M + rows - 1) / rows);
}

// The groups of rows of a CTA: a round has a stretch of memory of its own, which its CTAs go through side by side.  (Norm backward of
// 262144 x 4096 BF16: 959 us in one round with chains of 862 rows, 962 in two, 1041 where every round went through the whole map.)
struct GroupRange {
    int first, end, step;
    __device__ __forceinline__ GroupRange(int groups, int rounds)
        : first(static_cast<int>(blockIdx.x)), end(groups), step(static_cast<int>(gridDim.x)) {
        if (rounds == 1) return;  // no divisions ahead of the first copy
        step /= rounds;
        const int stretch = (groups + rounds - 1) / rounds, round = static_cast<int>(blockIdx.x) / step;
        first = round * stretch + static_cast<int>(blockIdx.x) - round * step;
        end = min(groups, (round + 1) * stretch);
    }
    __device__ __forceinline__ int count() const { return first < end ? (end - first - 1) / step + 1 : 0; }
};

// Parts first, first + 32, ... of column c: 256 at a time, then with the rounding carried along.
__device__ __forceinline__ float sum_of_parts(const float* part, int first, int parts, int columns, int c) {
    CarriedSum sum;
    for (int i = first; i < parts;) {
        const int end = parts - i < 32 * 256 ? parts : i + 32 * 256;
        float run = 0.0f;
#pragma unroll 4
        for (; i < end; i += 32) run += part[static_cast<long long>(i) * columns + c];
        sum.add(run);
    }
    return sum.total;
}

}  // namespace convgb
