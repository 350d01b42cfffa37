// rms_norm.cu -- root-mean-square norm of rows with the residual's addition, forward (also to 8 bits)
// and backward:
//
//   h = x + residual,  rstd = 1 / sqrt(mean(h^2) + eps),  y = h * rstd * gamma
//   n = h * rstd, d = dy * gamma:  dx = rstd * (d - n * mean(d * n)) + dh,  dgamma = sum over rows of dy * n
//
// Bound by memory: 8192 x 4096 BF16 with a residual 43 us forward (6.2 TB/s), 48 backward with dh (5.6), 40 to 8 bits
// (5.9).  A row stays in the registers of the 8 to 512 threads that hold it, so every byte
// crosses the bus once; rows past what they hold are swept twice (three times to 8 bits).
//
// A row starts at any element.  Rows off 16 bytes of up to 8,192 values have kernels of their own (rms_elements.cu); longer
// ones are handled here as the aligned 16-byte granules that they touch: all tensors of a call have the same shape, so
// a row begins at the same place of a granule in each of them; the first and last granule, shared with the
// neighbouring rows, are read and written by elements.
//
// dgamma: a backward pass that streams rows through shared memory keeps each thread's columns over all the rows that its
// CTA takes; for longer rows a kernel of its own reads dy and h by column.  Either way parts of it meet in the
// workspace and are added in one order.
#include <type_traits>

#include "rms_math.cuh"
#include "row_sums.cuh"
#include "rows_internal.h"

namespace convgb {

namespace {

// One row as granules: granule i holds columns first(i) .. first(i) + V - 1.
template <typename T, bool ALIGNED>
struct Row {
    static constexpr int V = 16 / sizeof(T), H = V / 2;
    long long granule;  // the row's first one
    int off, C, count;

    __device__ __forceinline__ Row(long long m, int C_) : C(C_) {
        const long long at = m * C_;
        granule = at / V;
        off = ALIGNED ? 0 : static_cast<int>(at % V);
        count = (off + C + V - 1) / V;
    }
    __device__ __forceinline__ int first(int i) const { return i * V - off; }
    __device__ __forceinline__ bool whole(int i) const { return ALIGNED || (first(i) >= 0 && first(i) + V <= C); }

    __device__ __forceinline__ void load(const void* base, int i, f2 (&f)[H]) const {
        const T* p = static_cast<const T*>(base) + (granule + i) * V;
        if (whole(i)) {
            VecIo<T, V>::unpack(__ldcs(reinterpret_cast<const uint4*>(p)), f);
            return;
        }
#pragma unroll
        for (int j = 0; j < H; ++j) f[j] = f2_make(element(p, i, 2 * j), element(p, i, 2 * j + 1));
    }
    __device__ __forceinline__ void store(void* base, int i, const f2 (&f)[H]) const {
        T* p = static_cast<T*>(base) + (granule + i) * V;
        if (whole(i)) {
            *reinterpret_cast<uint4*>(p) = VecIo<T, V>::pack(f);
            return;
        }
#pragma unroll
        for (int j = 0; j < H; ++j) {
            put(p, i, 2 * j, f2_lo(f[j]));
            put(p, i, 2 * j + 1, f2_hi(f[j]));
        }
    }
    __device__ __forceinline__ void store8(int8_t* base, int i, const f2 (&f)[H], const RowFactor& r) const {
        int8_t* p = base + (granule + i) * V;
        if (whole(i)) {
            quantise_store<V>(p, f, r);
            return;
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (inside(i, j)) p[j] = quantise1(j & 1 ? f2_hi(f[j / 2]) : f2_lo(f[j / 2]), r);
    }
    // gamma of the granule's columns (1 without gamma), 0 outside the row
    __device__ __forceinline__ void weights(const float* gamma, int i, f2 (&g)[H]) const {
        if (gamma == nullptr) {
#pragma unroll
            for (int j = 0; j < H; ++j) g[j] = f2_dup(1.0f);
        } else if constexpr (ALIGNED) {
#pragma unroll
            for (int j = 0; j < H; j += 2) {
                const float4 v = __ldg(reinterpret_cast<const float4*>(gamma + first(i) + 2 * j));
                g[j] = f2_make(v.x, v.y);
                g[j + 1] = f2_make(v.z, v.w);
            }
        } else {
#pragma unroll
            for (int j = 0; j < H; ++j)
                g[j] = f2_make(inside(i, 2 * j) ? __ldg(gamma + first(i) + 2 * j) : 0.0f,
                               inside(i, 2 * j + 1) ? __ldg(gamma + first(i) + 2 * j + 1) : 0.0f);
        }
    }

private:
    __device__ __forceinline__ bool inside(int i, int j) const {
        return static_cast<unsigned>(first(i) + j) < static_cast<unsigned>(C);
    }
    __device__ __forceinline__ float element(const T* p, int i, int j) const {
        return inside(i, j) ? static_cast<float>(p[j]) : 0.0f;
    }
    __device__ __forceinline__ void put(T* p, int i, int j, float v) const {
        if (inside(i, j)) p[j] = static_cast<T>(v);  // rounds to nearest even
    }
};

// Over the LANES threads of a row: a part of a warp, a warp, or a CTA; `buf` is used once.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int i = (LANES < 32 ? LANES : 32) / 2; i > 0; i >>= 1) v += __shfl_xor_sync(0xffffffffu, v, i);
    return v;
}

template <int LANES>
__device__ __forceinline__ float row_sum(float v, float* buf) {
    v = lanes_sum<LANES>(v);
    if constexpr (LANES > 32) {
        if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < LANES / 32; ++i) v += buf[i];
    }
    return v;
}

template <int LANES>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* buf) {
    if constexpr (LANES >= 32) {
        v = warp_max(v);
    } else {
#pragma unroll
        for (int i = LANES / 2; i > 0; i >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, i));
    }
    if constexpr (LANES > 32) {
        if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0;
#pragma unroll
        for (int i = 0; i < LANES / 32; ++i) v = max(v, buf[i]);
    }
    return v;
}

// A CTA: 128 threads where a warp or a part of one has a row, else a row's threads.
template <int LANES>
constexpr int kThreadsOf = LANES <= 32 ? 128 : LANES;
template <int LANES>
constexpr int kRowsOf = kThreadsOf<LANES> / LANES;

// ---------------------------------------------------------------- forward
template <typename T, bool ALIGNED, int ITEMS, int LANES, bool INT8>
__global__ void __launch_bounds__(kThreadsOf<LANES>) rms_forward_kernel(const RmsParams p) {
    using R = Row<T, ALIGNED>;
    __shared__ float sums[LANES > 32 ? LANES / 32 : 1];
    __shared__ uint32_t tops[LANES > 32 ? LANES / 32 : 1];
    const long long m = static_cast<long long>(blockIdx.x) * kRowsOf<LANES> + threadIdx.x / LANES;
    const bool live = m < p.M;
    if (LANES >= 32 && !live) return;  // whole warps; a part of one stays for the others' shuffles
    const R row(live ? m : 0, p.C);
    const int t = threadIdx.x % LANES, count = live ? row.count : 0;
    f2 v[ITEMS][R::H], square = 0;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int i = t + k * LANES;
#pragma unroll
        for (int j = 0; j < R::H; ++j) v[k][j] = 0;
        if (i < count) row.load(p.x, i, v[k]);
    }
    if (p.r != nullptr) {
        f2 r[ITEMS][R::H];
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int i = t + k * LANES;
#pragma unroll
            for (int j = 0; j < R::H; ++j) r[k][j] = 0;
            if (i < count) row.load(p.r, i, r[k]);
        }
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int i = t + k * LANES;
#pragma unroll
            for (int j = 0; j < R::H; ++j) v[k][j] = f2_add(v[k][j], r[k][j]);
            if (p.h != nullptr && i < count) row.store(p.h, i, v[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
#pragma unroll
        for (int j = 0; j < R::H; ++j) square = f2_fma(v[k][j], v[k][j], square);
    const float rstd = reciprocal_root(row_sum<LANES>(f2_lo(square) + f2_hi(square), sums), p.C, p.eps);
    if (t == 0 && live && p.rstd != nullptr) p.rstd[m] = rstd;
    const f2 factor = f2_dup(rstd);
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int i = t + k * LANES;
        if (i >= count) break;
        f2 g[R::H];
        row.weights(p.gamma, i, g);
#pragma unroll
        for (int j = 0; j < R::H; ++j) {
            v[k][j] = f2_mul(f2_mul(v[k][j], factor), g[j]);
            if constexpr (INT8) top = magnitude(top, v[k][j]);
        }
        if constexpr (!INT8) row.store(p.y, i, v[k]);
    }
    if constexpr (INT8) {
        const RowScale rs = row_scale(row_max<LANES>(magnitude_bits(top), tops));
        if (t == 0 && live) p.scale[m] = rs.scale;
        const RowFactor rf = row_factor(rs.inv);
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int i = t + k * LANES;
            if (i < count) row.store8(p.q, i, v[k], rf);
        }
    }
}

// Rows that no 512 threads hold, swept again for every step.  h is written in the last sweep: it may be the
// residual.
constexpr int kLongWarps = 16, kLongThreads = 32 * kLongWarps;

template <typename T, bool ALIGNED, bool INT8>
__global__ void __launch_bounds__(kLongThreads) rms_forward_long_kernel(const RmsParams p) {
    using R = Row<T, ALIGNED>;
    __shared__ float sums[kLongWarps];
    __shared__ uint32_t tops[kLongWarps];
    const long long m = blockIdx.x;
    const R row(m, p.C);
    const auto sum_of = [&](int i, f2(&v)[R::H]) {
        row.load(p.x, i, v);
        if (p.r == nullptr) return;
        f2 r[R::H];
        row.load(p.r, i, r);
#pragma unroll
        for (int j = 0; j < R::H; ++j) v[j] = f2_add(v[j], r[j]);
    };
    f2 square = 0;
#pragma unroll 4
    for (int i = threadIdx.x; i < row.count; i += kLongThreads) {
        f2 v[R::H];
        sum_of(i, v);
#pragma unroll
        for (int j = 0; j < R::H; ++j) square = f2_fma(v[j], v[j], square);
    }
    const float rstd = reciprocal_root(row_sum<kLongThreads>(f2_lo(square) + f2_hi(square), sums), p.C, p.eps);
    if (threadIdx.x == 0 && p.rstd != nullptr) p.rstd[m] = rstd;
    const f2 factor = f2_dup(rstd);
    const auto norm_of = [&](int i, f2(&v)[R::H]) {
        f2 g[R::H];
        row.weights(p.gamma, i, g);
#pragma unroll
        for (int j = 0; j < R::H; ++j) v[j] = f2_mul(f2_mul(v[j], factor), g[j]);
    };
    RowScale rs = {};
    if constexpr (INT8) {
        float top = 0.0f;
#pragma unroll 2
        for (int i = threadIdx.x; i < row.count; i += kLongThreads) {
            f2 v[R::H];
            sum_of(i, v);
            norm_of(i, v);
#pragma unroll
            for (int j = 0; j < R::H; ++j) top = magnitude(top, v[j]);
        }
        rs = row_scale(row_max<kLongThreads>(magnitude_bits(top), tops));
        if (threadIdx.x == 0) p.scale[m] = rs.scale;
    }
#pragma unroll 1
    for (int i = threadIdx.x; i < row.count; i += kLongThreads) {
        f2 v[R::H];
        sum_of(i, v);
        if (p.h != nullptr) row.store(p.h, i, v);
        norm_of(i, v);
        if constexpr (INT8) row.store8(p.q, i, v, row_factor(rs.inv));
        else row.store(p.y, i, v);
    }
}

// ---------------------------------------------------------------- backward
// Rows in registers: those that the ring below does not take.
template <typename T, bool ALIGNED, int ITEMS, int LANES>
__global__ void __launch_bounds__(LANES) rms_backward_kernel(const RmsParams p) {
    using R = Row<T, ALIGNED>;
    static_assert(LANES > 32, "a CTA to a row");
    __shared__ float sums[LANES / 32];
    const long long m = blockIdx.x;
    const int t = threadIdx.x;
    const R row(m, p.C);
    const f2 factor = f2_dup(p.rstd[m]);
    f2 d[ITEMS][R::H], n[ITEMS][R::H], dot = 0;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int i = t + k * LANES;
#pragma unroll
        for (int j = 0; j < R::H; ++j) d[k][j] = n[k][j] = 0;
        if (i >= row.count) continue;
        row.load(p.x, i, d[k]);
        row.load(p.h_in, i, n[k]);
    }
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int i = t + k * LANES;
        if (i >= row.count) continue;
        f2 g[R::H];
        row.weights(p.gamma, i, g);
#pragma unroll
        for (int j = 0; j < R::H; ++j) {
            n[k][j] = f2_mul(n[k][j], factor);
            d[k][j] = f2_mul(d[k][j], g[j]);
            dot = f2_fma(d[k][j], n[k][j], dot);
        }
    }
    const f2 minus = f2_dup(-__fdiv_rn(row_sum<LANES>(f2_lo(dot) + f2_hi(dot), sums), static_cast<float>(p.C)));
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int i = t + k * LANES;
        if (i >= row.count) continue;
        f2 r[R::H] = {};
        if (p.r != nullptr) row.load(p.r, i, r);
#pragma unroll
        for (int j = 0; j < R::H; ++j) d[k][j] = f2_fma(f2_fma(n[k][j], minus, d[k][j]), factor, r[j]);
        row.store(p.y, i, d[k]);
    }
}

// Rows on 16 bytes of at most 1,024 granules: a warp of its own brings them (dy, h and dh, whole rows, next to each other in
// memory) by bulk copies into a ring in shared memory, rows of 8, 16 or 32 lanes each, several to a stage, or one
// row of all warps.  Loads into registers left too few bytes under way between a row's barrier and the next row's first
// load: 8192 x 4096 BF16 with dh 83 us so, 3.2 TB/s.
constexpr int kStreamThreads = 32 * (kStreamWarps + 1);

template <typename T, int ITEMS, int LANES, bool DGAMMA>
__global__ void __launch_bounds__(kStreamThreads, ITEMS == 4 ? 1 : 2) rms_backward_stream_kernel(const RmsParams p, const Stream s) {
    using R = Row<T, true>;
    constexpr int kAtOnce = 32 * kStreamWarps / LANES;  // rows that the warps work on together
    const int rows = kAtOnce > 1 ? s.rows : 1;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ uint64_t full[kStreamMaxStages], empty[kStreamMaxStages];
    __shared__ float sums[2][kStreamWarps];
    __shared__ int abort_flag;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join of dgamma's parts
    volatile int* abort = &abort_flag;
    if (threadIdx.x == 0) {
        for (int i = 0; i < s.stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kStreamWarps);
        }
        abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    const int row_bytes = p.C * static_cast<int>(sizeof(T));
    const GroupRange range(static_cast<int>((static_cast<long long>(p.M) + rows - 1) / rows), p.rounds);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == kStreamWarps) {
        if (lane != 0) return;
        const uint8_t* from[3] = {static_cast<const uint8_t*>(p.x), static_cast<const uint8_t*>(p.h_in), static_cast<const uint8_t*>(p.r)};
        long long issued = 0;
        int st = 0;
        uint32_t ph = 0;
        for (int g = range.first; g < range.end; g += range.step) {
            if (!mbar_wait(&empty[st], ph ^ 1u, abort)) {
                record_status(p.status, kStatusTimeoutProducer, abort);
                break;
            }
            const long long m = static_cast<long long>(g) * rows;
            const int bytes = static_cast<int>(p.M - m < rows ? p.M - m : rows) * row_bytes, tensors = p.r != nullptr ? 3 : 2;
            mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(tensors * bytes));
            for (int i = 0; i < tensors; ++i)
                bulk_load(ring + st * s.stage_bytes + i * rows * row_bytes, from[i] + m * row_bytes, bytes, &full[st]);
            ++issued;
            if (++st == s.stages) {
                st = 0;
                ph ^= 1u;
            }
        }
        for (int i = 0; i < s.stages; ++i) {  // no copy in flight when the CTA leaves
            const long long fills = issued / s.stages + (i < issued % s.stages ? 1 : 0);
            if (fills && !mbar_wait(&full[i], static_cast<uint32_t>((fills - 1) & 1), nullptr)) record_status(p.status, kStatusTimeoutDrain, abort);
        }
        return;
    }
    const int t = threadIdx.x % LANES, slot = threadIdx.x / LANES, vecs = p.C / R::V;
    f2 gamma[ITEMS][R::H], total[DGAMMA ? ITEMS : 1][R::H] = {};
    const R first(0, p.C);
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int i = t + k * LANES;
        if (i < vecs) first.weights(p.gamma, i, gamma[k]);
    }
    int st = 0, turn = 0;
    uint32_t ph = 0;
    for (int g = range.first; g < range.end; g += range.step, turn ^= 1) {
        if (!mbar_wait(&full[st], ph, abort)) record_status(p.status, kStatusTimeoutTransform, abort);  // and on: every wait ends
#pragma unroll 1
        for (int at = slot; at < rows; at += kAtOnce) {  // rows is a multiple, 1 where all warps share a row
            const long long m = static_cast<long long>(g) * rows + at;
            const bool live = m < p.M;  // a dead row's lanes stay for the shuffles of others in their warp
            const float rstd = live ? __ldg(p.rstd + m) : 0.0f;
            const uint4* dy = reinterpret_cast<const uint4*>(ring + st * s.stage_bytes + at * row_bytes);
            const uint4* h = reinterpret_cast<const uint4*>(ring + st * s.stage_bytes + (rows + at) * row_bytes);
            const uint4* dh = reinterpret_cast<const uint4*>(ring + st * s.stage_bytes + (2 * rows + at) * row_bytes);
            const f2 factor = f2_dup(rstd);
            f2 d[ITEMS][R::H], n[ITEMS][R::H], dot = 0;
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) {
                const int i = t + k * LANES;
                if (i >= vecs || !live) continue;
                VecIo<T, R::V>::unpack(dy[i], d[k]);
                VecIo<T, R::V>::unpack(h[i], n[k]);
#pragma unroll
                for (int j = 0; j < R::H; ++j) {
                    n[k][j] = f2_mul(n[k][j], factor);
                    if constexpr (DGAMMA) total[k][j] = f2_fma(d[k][j], n[k][j], total[k][j]);
                    d[k][j] = f2_mul(d[k][j], gamma[k][j]);
                    dot = f2_fma(d[k][j], n[k][j], dot);
                }
            }
            float sum = lanes_sum<LANES>(f2_lo(dot) + f2_hi(dot));
            if constexpr (LANES > 32) {
                if (lane == 0) sums[turn][warp] = sum;
                sync_consumers();
                sum = 0.0f;
#pragma unroll
                for (int i = 0; i < kStreamWarps; ++i) sum += sums[turn][i];
            }
            const f2 minus = f2_dup(-__fdiv_rn(sum, static_cast<float>(p.C)));
            const R row(live ? m : 0, p.C);
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) {
                const int i = t + k * LANES;
                if (i >= vecs || !live) continue;
                f2 r[R::H] = {};
                if (p.r != nullptr) VecIo<T, R::V>::unpack(dh[i], r);
#pragma unroll
                for (int j = 0; j < R::H; ++j) d[k][j] = f2_fma(f2_fma(n[k][j], minus, d[k][j]), factor, r[j]);
                row.store(p.y, i, d[k]);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        if (++st == s.stages) {
            st = 0;
            ph ^= 1u;
        }
    }
    if constexpr (DGAMMA) {
        float* part = p.part + static_cast<long long>(blockIdx.x) * p.C;
        if constexpr (kAtOnce > 1) {  // the rows' sums, in the ring: every stage has been read
            sync_consumers();
            part = reinterpret_cast<float*>(ring) + slot * p.C;
        }
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int i = t + k * LANES;
            if (i >= vecs) continue;
#pragma unroll
            for (int j = 0; j < R::H; j += 2)
                *reinterpret_cast<float4*>(part + i * R::V + 2 * j) =
                    make_float4(f2_lo(total[k][j]), f2_hi(total[k][j]), f2_lo(total[k][j + 1]), f2_hi(total[k][j + 1]));
        }
        if constexpr (kAtOnce > 1) {
            sync_consumers();
            for (int c = threadIdx.x; c < p.C; c += 32 * kStreamWarps) {
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) sum += reinterpret_cast<const float*>(ring)[i * p.C + c];
                p.part[static_cast<long long>(blockIdx.x) * p.C + c] = sum;
            }
        }
    }
}

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kLongThreads) rms_backward_long_kernel(const RmsParams p) {
    using R = Row<T, ALIGNED>;
    __shared__ float sums[kLongWarps];
    const long long m = blockIdx.x;
    const R row(m, p.C);
    const f2 factor = f2_dup(p.rstd[m]);
    const auto scaled = [&](int i, f2(&d)[R::H], f2(&n)[R::H]) {
        row.load(p.x, i, d);
        row.load(p.h_in, i, n);
        f2 g[R::H];
        row.weights(p.gamma, i, g);
#pragma unroll
        for (int j = 0; j < R::H; ++j) {
            n[j] = f2_mul(n[j], factor);
            d[j] = f2_mul(d[j], g[j]);
        }
    };
    f2 dot = 0;
#pragma unroll 2
    for (int i = threadIdx.x; i < row.count; i += kLongThreads) {
        f2 d[R::H], n[R::H];
        scaled(i, d, n);
#pragma unroll
        for (int j = 0; j < R::H; ++j) dot = f2_fma(d[j], n[j], dot);
    }
    const f2 minus = f2_dup(-__fdiv_rn(row_sum<kLongThreads>(f2_lo(dot) + f2_hi(dot), sums), static_cast<float>(p.C)));
#pragma unroll 1
    for (int i = threadIdx.x; i < row.count; i += kLongThreads) {
        f2 d[R::H], n[R::H], r[R::H] = {};
        scaled(i, d, n);
        if (p.r != nullptr) row.load(p.r, i, r);
#pragma unroll
        for (int j = 0; j < R::H; ++j) d[j] = f2_fma(f2_fma(n[j], minus, d[j]), factor, r[j]);
        row.store(p.y, i, d);
    }
}

// dgamma by column: block (x, y) adds rows y, y + gridDim.y, ... eight at a time of 32 columns.
constexpr int kColumnRows = 8;

template <typename T>
__global__ void __launch_bounds__(256) rms_columns_kernel(const RmsParams p) {
    __shared__ float sums[kColumnRows][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const T* dy = static_cast<const T*>(p.x);
    const T* h = static_cast<const T*>(p.h_in);
    float total = 0.0f;
    if (c < p.C) {
#pragma unroll 16
        for (long long m = static_cast<long long>(blockIdx.y) * kColumnRows + warp; m < p.M;
             m += static_cast<long long>(gridDim.y) * kColumnRows)
            total = fmaf(static_cast<float>(dy[m * p.C + c]), static_cast<float>(h[m * p.C + c]) * p.rstd[m], total);
    }
    sums[warp][lane] = total;
    __syncthreads();
    if (warp == 0 && c < p.C) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kColumnRows; ++i) sum += sums[i][lane];
        p.part[static_cast<long long>(blockIdx.y) * p.C + c] = sum;
    }
}

// ---------------------------------------------------------------- launches
struct Form {
    int items, lanes;  // granules a thread holds of each tensor, and threads to a row (0: rows too long for registers)
};

Form pick_form(const RmsParams& p) {
    const int V = p.bf16 ? 8 : 4;
    const int granules = p.C % V == 0 ? p.C / V : (p.C + V - 2) / V + 1;  // the most that a row touches
    if (granules <= 8) return {1, 8};
    if (granules <= 16) return {1, 16};
    if (granules <= 32) return {1, 32};
    if (granules <= 64) return {2, 32};
    if (granules <= 128) return {4, 32};
    if (granules <= 256) return {2, 128};
    if (granules <= 512) return {4, 128};
    if (granules <= 1024) return {4, 256};
    if (granules <= 2048) return {4, 512};
    return {0, 0};
}

bool aligned_rows(const RmsParams& p) { return p.C % (p.bf16 ? 8 : 4) == 0; }

template <int N>
using Const = std::integral_constant<int, N>;

template <typename F>
void by_form(const Form& f, F&& run) {
    if (f.lanes == 8) run(Const<1>(), Const<8>());
    else if (f.lanes == 16) run(Const<1>(), Const<16>());
    else if (f.lanes == 32 && f.items == 1) run(Const<1>(), Const<32>());
    else if (f.lanes == 32 && f.items == 2) run(Const<2>(), Const<32>());
    else if (f.lanes == 32) run(Const<4>(), Const<32>());
    else if (f.lanes == 128 && f.items == 2) run(Const<2>(), Const<128>());
    else if (f.lanes == 128) run(Const<4>(), Const<128>());
    else if (f.lanes == 256) run(Const<4>(), Const<256>());
    else run(Const<4>(), Const<512>());
}

template <typename T, bool ALIGNED, bool INT8>
cudaError_t forward(const RmsParams& p, cudaStream_t stream) {
    const Form f = pick_form(p);
    if (f.lanes == 0) {
        rms_forward_long_kernel<T, ALIGNED, INT8><<<p.M, kLongThreads, 0, stream>>>(p);
    } else {
        by_form(f, [&](auto items, auto lanes) {
            constexpr int I = decltype(items)::value, N = decltype(lanes)::value;
            if constexpr (ALIGNED || (N == 512 && sizeof(T) == 2))  // other rows off 16 bytes go by elements or are longer
                rms_forward_kernel<T, ALIGNED, I, N, INT8><<<(p.M + kRowsOf<N> - 1) / kRowsOf<N>, kThreadsOf<N>, 0, stream>>>(p);
        });
    }
    return cudaGetLastError();
}

// The streaming backward form of a plan: granules a thread holds, threads to a row (0: another form), and CTAs that an
// SM runs at a time.
struct StreamForm {
    int items, lanes, ctas;
};
StreamForm stream_form(const RmsParams& p) {
    const int granules = p.C / (p.bf16 ? 8 : 4);
    if (!aligned_rows(p) || granules > 1024) return {0, 0, 0};
    const int lanes = granules <= 8 ? 8 : (granules <= 16 ? 16 : (granules <= 128 ? 32 : 32 * kStreamWarps));
    const int items = granules <= lanes ? 1 : (granules <= 2 * lanes ? 2 : 4);
    return {items, lanes, items == 4 ? 1 : 2};
}

int stream_rows_of(const RmsParams& p, const StreamForm& f, int num_sms) {
    return stream_rows(p.M, 32 * kStreamWarps / f.lanes, 3, static_cast<long long>(p.C) * (p.bf16 ? 2 : 4), f.ctas * num_sms);
}

void plan_stream(RmsParams& p, const StreamForm& f, int num_sms) {
    p.rows = stream_rows_of(p, f, num_sms);
    const long long need = (static_cast<long long>(p.M) + p.rows - 1) / p.rows;
    const int resident = f.ctas * num_sms;
    p.rounds = chain_rounds(p.M, 32 * kStreamWarps / f.lanes, resident);
    if (need <= 4) p.ctas = 1;  // a turn takes a microsecond, a join of parts and its launch four
    else if (need < resident) p.ctas = static_cast<int>(need);
    else p.ctas = p.rounds * resident;
    p.parts = p.ctas;
}

template <typename T, int ITEMS, int LANES>
cudaError_t stream_launch(const RmsParams& p, const StreamForm& f, cudaStream_t stream) {
    Stream s;
    s.rows = p.rows;
    s.stage_bytes = 3 * p.C * static_cast<int>(sizeof(T)) * s.rows;
    const int room = (f.ctas == 2 ? 113 : 226) * 1024 - 1024;  // of shared memory, barriers aside
    s.stages = room / s.stage_bytes < kStreamMaxStages ? room / s.stage_bytes : kStreamMaxStages;
    int bytes = s.stages * s.stage_bytes;
    const int sums = LANES <= 32 ? 32 * kStreamWarps / LANES * p.C * 4 : 0;  // of the rows that the warps work on together
    if (bytes < sums) bytes = sums;
    const auto run = [&](auto* kernel, SmemLimitCache& limits) {
        const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), 226 * 1024, limits);
        if (e != cudaSuccess) return e;
        kernel<<<p.ctas, kStreamThreads, bytes, stream>>>(p, s);
        return cudaGetLastError();
    };
    static SmemLimitCache with, without;
    return p.dgamma != nullptr ? run(rms_backward_stream_kernel<T, ITEMS, LANES, true>, with)
                               : run(rms_backward_stream_kernel<T, ITEMS, LANES, false>, without);
}

template <typename T>
cudaError_t stream_backward(const RmsParams& p, const StreamForm& f, cudaStream_t stream) {
    constexpr int kAll = 32 * kStreamWarps;
    if (f.lanes == 8) return stream_launch<T, 1, 8>(p, f, stream);
    if (f.lanes == 16) return stream_launch<T, 1, 16>(p, f, stream);
    if (f.lanes == 32) {
        if (f.items == 1) return stream_launch<T, 1, 32>(p, f, stream);
        return f.items == 2 ? stream_launch<T, 2, 32>(p, f, stream) : stream_launch<T, 4, 32>(p, f, stream);
    }
    if (f.items == 1) return stream_launch<T, 1, kAll>(p, f, stream);
    return f.items == 2 ? stream_launch<T, 2, kAll>(p, f, stream) : stream_launch<T, 4, kAll>(p, f, stream);
}

template <typename T, bool ALIGNED>
cudaError_t backward(const RmsParams& p, cudaStream_t stream) {
    const bool join = p.dgamma != nullptr && p.parts > 1;
    const StreamForm sf = stream_form(p);
    const Form f = pick_form(p);
    if (ALIGNED && sf.lanes != 0) {
        const cudaError_t e = stream_backward<T>(p, sf, stream);
        if (e != cudaSuccess || !join) return e;
        return launch_join_columns(p.part, p.parts, p.C, p.dgamma, true, stream);
    }
    if (p.dgamma != nullptr)  // first: dx may be dy
        rms_columns_kernel<T><<<dim3((p.C + 31) / 32, p.parts), 256, 0, stream>>>(p);
    if (f.lanes == 0) {
        rms_backward_long_kernel<T, ALIGNED><<<p.M, kLongThreads, 0, stream>>>(p);
    } else {
        by_form(f, [&](auto items, auto lanes) {
            constexpr int I = decltype(items)::value, N = decltype(lanes)::value;
            if constexpr (N == 512 && (ALIGNED || sizeof(T) == 2)) rms_backward_kernel<T, ALIGNED, I, N><<<p.M, N, 0, stream>>>(p);
        });
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !join) return e;
    return launch_join_columns(p.part, p.parts, p.C, p.dgamma, false, stream);
}

}  // namespace

void rms_plan_backward(RmsParams& p, int num_sms) {
    if (rms_by_elements(p)) {
        p.ctas = 2 * num_sms;
        rms_plan_elements(p);
        return;
    }
    const StreamForm f = stream_form(p);
    if (f.lanes != 0) {
        plan_stream(p, f, num_sms);
        return;
    }
    // dgamma by column: about four CTAs an SM, more where chains of rows would pass kChainRows (65536 x 16384 BF16 4.30 ms, 3.88 so)
    const long long columns = (p.C + 31) / 32, need = (static_cast<long long>(p.M) + 4 * kColumnRows - 1) / (4 * kColumnRows);
    const long long most = (4LL * num_sms + columns - 1) / columns;
    const long long chains = (static_cast<long long>(p.M) + kColumnRows * kChainRows - 1) / (kColumnRows * kChainRows);
    p.parts = static_cast<int>(need < most ? need : (most > chains ? most : chains));
}

cudaError_t launch_rms_forward(const RmsParams& p, cudaStream_t stream) {
    if (rms_by_elements(p)) return launch_rms_elements(p, false, stream);
    const bool aligned = aligned_rows(p);
    const auto run = [&](auto element) {
        using T = decltype(element);
        if (p.q != nullptr) return aligned ? forward<T, true, true>(p, stream) : forward<T, false, true>(p, stream);
        return aligned ? forward<T, true, false>(p, stream) : forward<T, false, false>(p, stream);
    };
    return p.bf16 ? run(__nv_bfloat16()) : run(float());
}

cudaError_t launch_rms_backward(const RmsParams& given, cudaStream_t stream) {
    RmsParams p = given;
    if (p.parts == 1) p.part = p.dgamma;
    if (rms_by_elements(p)) {
        const cudaError_t e = launch_rms_elements(p, true, stream);
        if (e != cudaSuccess || p.dgamma == nullptr || p.parts == 1) return e;
        return launch_join_columns(p.part, p.parts, p.C, p.dgamma, true, stream);
    }
    if (p.bf16) return aligned_rows(p) ? backward<__nv_bfloat16, true>(p, stream) : backward<__nv_bfloat16, false>(p, stream);
    return aligned_rows(p) ? backward<float, true>(p, stream) : backward<float, false>(p, stream);
}

}  // namespace convgb
