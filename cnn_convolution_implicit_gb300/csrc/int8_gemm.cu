// int8_gemm.cu -- the 8-bit product on tcgen05 tensor cores:
//
//   y[m][n] = act( x_scale[m] * w_scale[n] * sum_k x[m][k] * w[n][k] + bias[n] )
//
// An 8-bit integer is exact in FP16 (11 significand bits), a product of two of them
// stays below 2^15 and the FP32 accumulator holds every partial sum below 2^24
// exactly, so the FP16 MMA gives the integer sum (always for K <= 1024).  This part's
// 8-bit integer tensor rate is a small fraction of its FP16 rate.
//
// The operands stay 8-bit in memory; converter warps bring them to FP16 on their way
// into shared memory:
//   x ^ 0x80 = x + 128 as an unsigned byte u; the FP16 bit pattern 0x6400 | u is
//   1024 + u; subtracting 1152 leaves x.  One exclusive-or, two byte permutes and two
//   packed subtractions for four values.
//
// Warp roles (832 threads, one CTA per SM, persistent over tiles):
//   warps 0..15   converters, four groups that take turns by stage, so one loads, converts,
//                 publishes or waits while the others do: 8-bit rows from the raw ring to FP16
//                 values in the 128-byte-swizzle operand tiles of a stage
//   warps 16..23  epilogue: two warps per 32-row quarter of tensor memory, half of the columns
//                 each: scales, bias, activation, rounding, stores from registers
//   warp 24       tensor memory; one lane issues tcgen05.mma and commits
//   warp 25       one lane fills the raw ring by TMA: K = 64 of both operands, 8-bit, per slot
// Rows that do not start on 16 bytes (K % 16) are beyond the TMA: there the converters load
// them straight from memory (ALIGNED = false).  Loading a step ahead in registers does not
// replace the ring: the fence that publishes a stage also waits for the loads under way
// (8192 x 4096 x 4096 measured 413 us that way and 325 us with the ring).
// A stage holds K = 64 of both operands, one 128-byte FP16 row each.  Tensor memory holds two
// accumulators, so the epilogue of one tile overlaps the next one's MMAs.
//
// Columns: a lane of the epilogue reads accumulator columns 8 j + 2 q + {0, 1} of two rows
// (q = lane % 4, j = 0..7: the 16 x 256-bit shape).  The converters put weight row
// 16 q + 2 j + {0, 1} of each 64 there, so a lane holds 16 neighbouring outputs of a row, four
// lanes a 128-byte line of BF16, and a store instruction covers 8 whole lines.  (One row a
// lane, 32 lines touched per instruction, cost 38 us of 133 at 200704 x 256 -> 512; its 16-byte
// broadcast reads of the scales, four times as many as here, another 34.)
//
// PAIR: two SMs share a 256 x BN tile (tcgen05.mma.cta_group::2): each converts its own
// 128 rows of x and BN / 2 rows of w.  Shared memory bounds this kernel (written by the
// converters, read by the MMA), and a pair halves the traffic of w.
//
// Rows past M or N are neither loaded nor written: their outputs are never stored, and
// one row's operand does not reach another row's result.  Past K both operands are 0.
#include "int8_internal.h"
#include "pointwise_math.cuh"
#include "ptx.cuh"

namespace convgb {

namespace {

constexpr int kGroups = 4;       // converter groups
constexpr int kGroupWarps = 4;
constexpr int kConverterWarps = kGroups * kGroupWarps;
constexpr int kEpilogueWarps = 8;
constexpr int kMmaWarp = kConverterWarps + kEpilogueWarps;
constexpr int kLoadWarp = kMmaWarp + 1;
constexpr int kGemmThreads = 32 * (kLoadWarp + 1);
constexpr int kStepK = 64;       // K of one stage
constexpr int kRowBytes = 128;   // one FP16 operand row of a stage

template <bool PAIR, int BN, bool ALIGNED>
struct Shape {
    static constexpr int kRowsB = PAIR ? BN / 2 : BN;
    static constexpr int kTileA = 128 * kRowBytes;
    static constexpr int kStage = kTileA + kRowsB * kRowBytes;
    static constexpr int kStages = kGroups;              // one for each converter group
    static constexpr int kRaw = ALIGNED ? (128 + kRowsB) * kStepK : 0;  // one slot of the raw ring
    static constexpr int kRawSlots = ALIGNED ? (kRowsB >= 128 ? 6 : 8) : 0;  // in 227 KB beside the stages
    static constexpr int kItems = (128 + kRowsB) / 32;   // 16-byte items a converter thread moves per stage
    static constexpr int kTmemCols = 2 * BN < 32 ? 32 : 2 * BN;
    static constexpr int kSmem = kStages * kStage + kRawSlots * kRaw + 2 * 256 * 4 + 256;
};

struct Bars {
    uint64_t* rfull;
    uint64_t* rempty;
    uint64_t* full;
    uint64_t* empty;
    uint64_t* tfull;
    uint64_t* tempty;
    uint64_t* drain;
    uint64_t* esync;
    uint32_t* tmem_slot;
    int* abort;
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

__device__ __forceinline__ void store_v8(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e, uint32_t f,
                                         uint32_t g, uint32_t h) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a), "r"(b), "r"(c), "r"(d),
                 "r"(e), "r"(f), "r"(g), "r"(h)
                 : "memory");
}

// A bounded wait whose answer is the same in every lane.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}

__device__ __forceinline__ bool warp_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort) {
    return __all_sync(0xffffffffu, mbar_wait_cluster(bar, parity, abort));
}

// The epilogue warps among themselves: an mbarrier instead of a CTA barrier, so that this wait
// is bounded like every other.
__device__ __forceinline__ bool epilogue_sync(uint64_t* bar, uint32_t& phase, volatile int* abort) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
    const bool ok = warp_wait(bar, phase, abort);
    phase ^= 1u;
    return ok;
}

// Where a converter stands: its tile and K-step.
struct Walk {
    int u, k0;
    int mu, nt;
    int m0, n0;  // first row of x and of w that this CTA converts
};

// The tiles of a launch, and this CTA's way through them (no division per tile).
struct Tiles {
    int n_tiles, units, step, step_m, step_n;
    uint32_t rank;
};

template <bool PAIR, int BN>
__device__ __forceinline__ void place(const Tiles& t, Walk& w) {
    w.m0 = PAIR ? w.mu * 256 + static_cast<int>(t.rank) * 128 : w.mu * 128;
    w.n0 = w.nt * BN + (PAIR ? static_cast<int>(t.rank) * (BN / 2) : 0);
}

template <bool PAIR, int BN>
__device__ __forceinline__ Walk walk_from(const Tiles& t, int unit0) {
    Walk w;
    w.u = unit0;
    w.k0 = 0;
    w.mu = unit0 / t.n_tiles;
    w.nt = unit0 - w.mu * t.n_tiles;
    place<PAIR, BN>(t, w);
    return w;
}

__device__ __forceinline__ void next_unit(const Tiles& t, Walk& w) {
    w.u += t.step;
    w.mu += t.step_m;
    w.nt += t.step_n;
    if (w.nt >= t.n_tiles) {
        w.nt -= t.n_tiles;
        ++w.mu;
    }
}

template <bool PAIR, int BN>
__device__ __forceinline__ void advance(const Int8Params& p, const Tiles& t, Walk& w, int steps) {
    for (int i = 0; i < steps && w.u < t.units; ++i) {
        w.k0 += kStepK;
        if (w.k0 >= p.K) {
            w.k0 = 0;
            next_unit(t, w);
            place<PAIR, BN>(t, w);
        }
    }
}

template <bool PAIR, int BN>
__device__ __forceinline__ void load_stage(const Int8Params& p, const Walk& w, int r0, int c,
                                           uint4 (&item)[Shape<PAIR, BN, false>::kItems]) {
    const int k = w.k0 + 16 * c;
    const int len = p.K - k;
    const long long total_x = static_cast<long long>(p.M) * p.K, total_w = static_cast<long long>(p.N) * p.K;
#pragma unroll
    for (int i = 0; i < Shape<PAIR, BN, false>::kItems; ++i) {
        item[i] = make_uint4(0, 0, 0, 0);
        if (len <= 0) continue;
        const int n_len = len < 16 ? len : 16;
        if (i < 4) {
            const int row = w.m0 + r0 + 32 * i;
            if (row < p.M) item[i] = load_item(p.x, static_cast<long long>(row) * p.K + k, n_len, total_x);
        } else {
            const int row = w.n0 + r0 + 32 * (i - 4);
            if (row < p.N) item[i] = load_item(p.w, static_cast<long long>(row) * p.K + k, n_len, total_w);
        }
    }
}

// The stage's row (accumulator column) of weight row n: columns 16 q + 2 j + e of each 64 sit at
// 8 j + 2 q + e.  Tiles of 32 columns: the same with 8 neighbours a lane, j = 0..3.
template <int BN>
__device__ __forceinline__ int column_of(int n) {
    if constexpr (BN >= 64) return (n & ~63) | ((n & 14) << 2) | ((n & 48) >> 3) | (n & 1);
    else return ((n & 6) << 2) | ((n & 24) >> 2) | (n & 1);
}

template <bool PAIR, int BN>
__device__ __forceinline__ void store_stage(const Int8Params& p, const Walk& w, int r0, int c,
                                            const uint4 (&item)[Shape<PAIR, BN, false>::kItems], uint8_t* stage) {
    using S = Shape<PAIR, BN, false>;
#pragma unroll
    for (int i = 0; i < S::kItems; ++i) {
        int row = r0 + 32 * (i < 4 ? i : i - 4);
        if (i < 4 ? w.m0 + row >= p.M : w.n0 + row >= p.N) continue;
        const uint2 a = to_half4(item[i].x), b = to_half4(item[i].y), d = to_half4(item[i].z), e = to_half4(item[i].w);
        if (i >= 4) row = column_of<BN>(row);
        uint8_t* dst = stage + (i < 4 ? 0 : S::kTileA) + row * kRowBytes;
        const int sw = row & 7;  // eight lanes: four chunks of two rows, eight bank groups
        *reinterpret_cast<uint4*>(dst + (((2 * c) ^ sw) << 4)) = make_uint4(a.x, a.y, b.x, b.y);
        *reinterpret_cast<uint4*>(dst + (((2 * c + 1) ^ sw) << 4)) = make_uint4(d.x, d.y, e.x, e.y);
    }
}

// 16 lanes (rows) x 64 columns of tensor memory: register 4 j + 2 h + e of a lane is row
// lane / 4 + 8 h, column 8 j + 2 (lane % 4) + e.
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
          "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
          "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

// The same with 32 columns, in the first 16 registers.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
#pragma unroll
    for (int i = 16; i < 32; ++i) r[i] = 0;
}

// Scale, bias and activation of two neighbouring columns of one row, in place, as packed FP32.
template <int ACT>
__device__ __forceinline__ void finish_two(uint32_t& lo, uint32_t& hi, uint64_t xs2, uint64_t ws2, uint64_t bias2) {
    asm("{\n\t.reg .b64 t;\n\t"
        "mov.b64 t, {%0, %1};\n\t"
        "mul.rn.f32x2 t, t, %2;\n\t"
        "fma.rn.f32x2 t, t, %3, %4;\n\t"
        "mov.b64 {%0, %1}, t;\n\t}"
        : "+r"(lo), "+r"(hi)
        : "l"(xs2), "l"(ws2), "l"(bias2));
    lo = __float_as_uint(activate<ACT>(__uint_as_float(lo)));
    hi = __float_as_uint(activate<ACT>(__uint_as_float(hi)));
}

// A lane's part of 16 rows x 64 columns: 16 neighbouring columns of two rows (J = 8), or 8 of them
// where a tile has 32 columns (J = 4).
template <int ACT, int J>
__device__ __forceinline__ void finish_block(uint32_t (&v)[32], float xs_lo, float xs_hi, const float* scale,
                                             const float* bias) {
    uint64_t lo2, hi2;
    asm("mov.b64 %0, {%1, %1};" : "=l"(lo2) : "f"(xs_lo));
    asm("mov.b64 %0, {%1, %1};" : "=l"(hi2) : "f"(xs_hi));
#pragma unroll
    for (int j = 0; j < J; j += 2) {
        const ulonglong2 s = *reinterpret_cast<const ulonglong2*>(scale + 2 * j);
        const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(bias + 2 * j);
        finish_two<ACT>(v[4 * j], v[4 * j + 1], lo2, s.x, b.x);
        finish_two<ACT>(v[4 * j + 2], v[4 * j + 3], hi2, s.x, b.x);
        finish_two<ACT>(v[4 * j + 4], v[4 * j + 5], lo2, s.y, b.y);
        finish_two<ACT>(v[4 * j + 6], v[4 * j + 7], hi2, s.y, b.y);
    }
}

// 2 J neighbouring outputs of row h of a lane's two, in the widest stores that every row's start
// allows (wide: 32 or 16 bytes; 0: one by one).
template <int J>
__device__ __forceinline__ void store_row(const Int8Params& p, const uint32_t (&v)[32], int h, long long row, int n, int wide) {
    const auto at = [&](int i) { return v[4 * (i >> 1) + 2 * h + (i & 1)]; };  // column n + i
    const long long o = row * p.N + n;
    if (n + 2 * J <= p.N && wide != 0) {
        if (p.out_bf16) {
            uint32_t q[J];
#pragma unroll
            for (int i = 0; i < J; ++i) q[i] = pack_bf16x2(__uint_as_float(at(2 * i)), __uint_as_float(at(2 * i + 1)));
            __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + o;
            if (J == 8 && wide == 32) {
                store_v8(y, q[0], q[1], q[2], q[3], q[4 % J], q[5 % J], q[6 % J], q[7 % J]);
            } else {
#pragma unroll
                for (int i = 0; i < J / 4; ++i)
                    reinterpret_cast<uint4*>(y)[i] = make_uint4(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
            }
        } else {
            float* y = static_cast<float*>(p.y) + o;
            if (wide == 32) {
#pragma unroll
                for (int i = 0; i < 2 * J; i += 8)
                    store_v8(y + i, at(i), at(i + 1), at(i + 2), at(i + 3), at(i + 4), at(i + 5), at(i + 6), at(i + 7));
            } else {
#pragma unroll
                for (int i = 0; i < 2 * J; i += 4)
                    *reinterpret_cast<uint4*>(y + i) = make_uint4(at(i), at(i + 1), at(i + 2), at(i + 3));
            }
        }
        return;
    }
    if (p.out_bf16) {
        __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + o;
#pragma unroll
        for (int i = 0; i < 2 * J; ++i)
            if (n + i < p.N) y[i] = __float2bfloat16_rn(__uint_as_float(at(i)));
    } else {
        float* y = static_cast<float*>(p.y) + o;
#pragma unroll
        for (int i = 0; i < 2 * J; ++i)
            if (n + i < p.N) y[i] = __uint_as_float(at(i));
    }
}

__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {  // as idesc_bf16_f32 with FP16 operands (type 0)
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

template <bool PAIR, int BN, bool ALIGNED>
__global__ void __launch_bounds__(kGemmThreads, 1)
    int8_gemm_kernel(const Int8Params p, const __grid_constant__ CUtensorMap map_x,
                     const __grid_constant__ CUtensorMap map_w) {
    using S = Shape<PAIR, BN, ALIGNED>;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_addr(smem) & 1023u) {  // the swizzle's atoms; uniform, so no CTA waits for another
        record_status(p.status, kStatusTimeoutMma, nullptr);
        return;
    }
    Bars b;
    uint8_t* raw = smem + S::kStages * S::kStage;
    float* col_scale = reinterpret_cast<float*>(raw + S::kRawSlots * S::kRaw);  // of the tile in the epilogue
    float* col_bias = col_scale + 256;
    b.rfull = reinterpret_cast<uint64_t*>(col_bias + 256);
    b.rempty = b.rfull + S::kRawSlots;
    b.full = b.rempty + S::kRawSlots;
    b.empty = b.full + S::kStages;
    b.tfull = b.empty + S::kStages;
    b.tempty = b.tfull + 2;
    b.drain = b.tempty + 2;
    b.esync = b.drain + 1;
    b.tmem_slot = reinterpret_cast<uint32_t*>(b.esync + 1);
    b.abort = reinterpret_cast<int*>(b.tmem_slot + 1);
    volatile int* abort = b.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
    const bool leader = rank == 0;
    constexpr int kCtas = PAIR ? 2 : 1;

    Tiles tiles;
    tiles.n_tiles = (p.N + BN - 1) / BN;
    tiles.units = ((p.M + 128 * kCtas - 1) / (128 * kCtas)) * tiles.n_tiles;
    tiles.step = static_cast<int>(gridDim.x) / kCtas;
    tiles.step_m = tiles.step / tiles.n_tiles;
    tiles.step_n = tiles.step - tiles.step_m * tiles.n_tiles;
    tiles.rank = rank;
    const int unit0 = static_cast<int>(blockIdx.x) / kCtas, units = tiles.units, unit_step = tiles.step;
    const int ksteps = (p.K + kStepK - 1) / kStepK;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kRawSlots; ++s) {
            mbar_init(&b.rfull[s], 1);
            mbar_init(&b.rempty[s], kGroupWarps);
        }
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(&b.full[s], kCtas * kGroupWarps);
            mbar_init(&b.empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b.tfull[i], 1);
            mbar_init(&b.tempty[i], kCtas * kEpilogueWarps);
        }
        mbar_init(b.drain, 1);
        mbar_init(b.esync, kEpilogueWarps);
        *b.abort = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        if constexpr (PAIR) {
            tmem_alloc_pair(b.tmem_slot, S::kTmemCols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(b.tmem_slot, S::kTmemCols);
            tmem_relinquish();
        }
        tc_fence_before();
    }
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();  // the peer's barriers exist before anything signals them
    tc_fence_after();
    const uint32_t tmem = *b.tmem_slot;

    if (warp < kConverterWarps) {
        // ------------------------------------------------------------ converters
        const int group = warp / kGroupWarps;  // converts steps group, group + kGroups, ... into stage `group`
        const int t = threadIdx.x & (32 * kGroupWarps - 1);
        const int c = t & 3, r0 = t >> 2;
        Walk w = walk_from<PAIR, BN>(tiles, unit0);
        advance<PAIR, BN>(p, tiles, w, group);
        if (w.u < units) {
            uint32_t ph = 0;
            uint8_t* stage = smem + group * S::kStage;
            const auto publish = [&](uint4(&item)[S::kItems]) {
                if (!warp_wait(&b.empty[group], ph ^ 1u, abort)) {
                    record_status(p.status, kStatusTimeoutTransform, abort);
                    return false;
                }
                store_stage<PAIR, BN>(p, w, r0, c, item, stage);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR) mbar_arrive_remote(mapa_shared(smem_addr(&b.full[group]), 0));
                    else mbar_arrive(&b.full[group]);
                }
                ph ^= 1u;
                return true;
            };
            if constexpr (ALIGNED) {
                int rs = group;
                uint32_t rph = 0;
                while (w.u < units) {
                    if (!warp_wait(&b.rfull[rs], rph, abort)) {
                        record_status(p.status, kStatusTimeoutTransform, abort);
                        break;
                    }
                    uint4 item[S::kItems];
                    const uint4* src = reinterpret_cast<const uint4*>(raw + rs * S::kRaw) + t;
#pragma unroll
                    for (int i = 0; i < S::kItems; ++i) item[i] = src[i * 128];  // rows r0 + 32 i of x, then of w
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&b.rempty[rs]);
                    if (!publish(item)) break;
                    if ((rs += kGroups) >= S::kRawSlots) {  // more slots than groups: one wrap a turn at most
                        rs -= S::kRawSlots;
                        rph ^= 1u;
                    }
                    advance<PAIR, BN>(p, tiles, w, kGroups);
                }
            } else {
                while (w.u < units) {
                    uint4 item[S::kItems];
                    load_stage<PAIR, BN>(p, w, r0, c, item);
                    if (!publish(item)) break;
                    advance<PAIR, BN>(p, tiles, w, kGroups);
                }
            }
        }
    } else if (warp < kMmaWarp) {
        // ------------------------------------------------------------ epilogue
        const int quarter = warp & 3;
        const int half = (warp - kConverterWarps) >> 2;
        const int es = p.out_bf16 ? 2 : 4;
        const long long row_bytes = static_cast<long long>(p.N) * es;
        const uintptr_t y0 = reinterpret_cast<uintptr_t>(p.y);
        const int wide = row_bytes % 32 == 0 && y0 % 32 == 0 ? 32 : (row_bytes % 16 == 0 ? 16 : 0);
        int local = 0;
        uint32_t eph = 0;
        constexpr int J = BN >= 64 ? 8 : 4;        // pairs of columns a lane holds of a row
        constexpr int kCols = BN >= 128 ? BN / 2 : BN;  // columns of a warp; narrow tiles: 16 of its quarter's 32 rows
        const int col0 = BN >= 128 ? half * kCols : 0;
        for (Walk w = walk_from<PAIR, BN>(tiles, unit0); w.u < units; next_unit(tiles, w), ++local) {
            const int buf = local & 1;
            const uint32_t use = static_cast<uint32_t>(local >> 1) & 1u;
            const int nt = w.nt;
            const long long row0 = static_cast<long long>(w.mu) * 128 * kCtas + rank * 128 + quarter * 32 + (lane >> 2);
            float xs[4];  // rows row0, + 8, + 16, + 24
#pragma unroll
            for (int i = 0; i < 4; ++i) xs[i] = row0 + 8 * i < p.M ? __ldg(p.x_scale + row0 + 8 * i) : 0.0f;
            const int et = threadIdx.x - 32 * kConverterWarps;  // a column a thread, in flight while the MMAs finish
            const bool on = et < BN && nt * BN + et < p.N;
            const float cs = on ? __ldg(p.w_scale + nt * BN + et) : 0.0f;
            const float cb = on && p.bias ? __ldg(p.bias + nt * BN + et) : 0.0f;
            if (!warp_wait_cluster(&b.tfull[buf], use, abort)) {
                record_status(p.status, kStatusTimeoutEpilogue, abort);
                break;
            }
            tc_fence_after();
            bool in_step = epilogue_sync(b.esync, eph, abort);  // every warp is past the last tile's columns
            if (in_step) {
                col_scale[et] = cs;
                col_bias[et] = cb;
                in_step = epilogue_sync(b.esync, eph, abort);
            }
            if (!in_step) {
                record_status(p.status, kStatusTimeoutEpilogue, abort);
                break;
            }
            const int mine = (lane & 3) * 2 * J;  // this lane's first column of a block
#pragma unroll 1
            for (int col = col0; col < col0 + kCols; col += 8 * J) {
                if (nt * BN + col >= p.N) break;
                const int n = nt * BN + col + mine;
#pragma unroll
                for (int g = 0; g < 2; ++g) {  // 16 rows at a time
                    if (BN < 128 && g != half) continue;
                    uint32_t v[32];
                    const uint32_t at = tmem + (static_cast<uint32_t>(quarter * 32 + 16 * g) << 16) + buf * BN + col;
                    if constexpr (J == 8) tmem_ld_16x64(at, v);
                    else tmem_ld_16x32(at, v);
                    tmem_ld_wait(v);
                    const float* sc = col_scale + col + mine;
                    const float* bi = col_bias + col + mine;
                    if (p.act == CONV_ACT_RELU) finish_block<CONV_ACT_RELU, J>(v, xs[2 * g], xs[2 * g + 1], sc, bi);
                    else if (p.act == CONV_ACT_SILU) finish_block<CONV_ACT_SILU, J>(v, xs[2 * g], xs[2 * g + 1], sc, bi);
                    else finish_block<CONV_ACT_NONE, J>(v, xs[2 * g], xs[2 * g + 1], sc, bi);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const long long row = row0 + 16 * g + 8 * h;
                        if (row < p.M && n < p.N) store_row<J>(p, v, h, row, n, wide);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR) mbar_arrive_remote(mapa_shared(smem_addr(&b.tempty[buf]), 0));
                else mbar_arrive(&b.tempty[buf]);
            }
        }
    } else if (warp == kLoadWarp) {
        // ------------------------------------------------------------ raw ring
        if constexpr (ALIGNED) {
            Walk w = walk_from<PAIR, BN>(tiles, unit0);
            if (lane == 0 && w.u < units) {
                long long issued = 0;
                int rs = 0;
                uint32_t ph = 0;
                while (w.u < units) {
                    if (!mbar_wait(&b.rempty[rs], ph ^ 1u, abort)) {
                        record_status(p.status, kStatusTimeoutProducer, abort);
                        break;
                    }
                    mbar_arrive_expect_tx(&b.rfull[rs], S::kRaw);
                    uint8_t* slot = raw + rs * S::kRaw;
                    tma_load_2d(slot, &map_x, &b.rfull[rs], w.k0, w.m0);  // past the matrix: zeros
                    tma_load_2d(slot + 128 * kStepK, &map_w, &b.rfull[rs], w.k0, w.n0);
                    ++issued;
                    if (++rs == S::kRawSlots) {
                        rs = 0;
                        ph ^= 1u;
                    }
                    advance<PAIR, BN>(p, tiles, w, 1);
                }
                for (int s = 0; s < S::kRawSlots; ++s) {  // no copy in flight when the CTA leaves
                    const long long fills = issued / S::kRawSlots + (s < issued % S::kRawSlots ? 1 : 0);
                    if (fills && !mbar_wait(&b.rfull[s], static_cast<uint32_t>((fills - 1) & 1), nullptr))
                        record_status(p.status, kStatusTimeoutDrain, abort);
                }
            }
        }
    } else if (lane == 0 && leader) {
        // ------------------------------------------------------------ MMA
        constexpr uint32_t idesc = idesc_f16_f32(128 * kCtas, BN);
        int st = 0, local = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int u = unit0; u < units && ok; u += unit_step, ++local) {
            const int buf = local & 1;
            const uint32_t use = static_cast<uint32_t>(local >> 1) & 1u;
            if (!mbar_wait_cluster(&b.tempty[buf], use ^ 1u, abort)) {
                record_status(p.status, kStatusTimeoutMma, abort);
                break;
            }
            tc_fence_after();
            const uint32_t d = tmem + buf * BN;
            for (int ks = 0; ks < ksteps; ++ks) {
                if (!mbar_wait_cluster(&b.full[st], ph, abort)) {
                    record_status(p.status, kStatusTimeoutMma, abort);
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t base = smem_addr(smem + st * S::kStage);
                const int left = (p.K - ks * kStepK + 15) >> 4;
                const int mmas = left < 4 ? left : 4;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j >= mmas) break;
                    const uint64_t da = sdesc_sw128(base) + 2 * j;
                    const uint64_t db = sdesc_sw128(base + S::kTileA) + 2 * j;
                    const uint32_t acc = (ks | j) != 0 ? 1u : 0u;
                    if constexpr (PAIR) mma_bf16_pair(d, da, db, idesc, acc);  // kind::f16; idesc names the type
                    else mma_bf16(d, da, db, idesc, acc);
                }
                if constexpr (PAIR) mma_commit_pair(&b.empty[st], 3);
                else mma_commit(&b.empty[st]);
                if (++st == S::kStages) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            if (!ok) break;
            if constexpr (PAIR) mma_commit_pair(&b.tfull[buf], 3);
            else mma_commit(&b.tfull[buf]);
        }
        if constexpr (PAIR) mma_commit_pair(b.drain, 1);
        else mma_commit(b.drain);
        if (!mbar_wait_cluster(b.drain, 0, nullptr)) record_status(p.status, kStatusTimeoutDrain, abort);
    }
    __syncwarp();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();  // no CTA leaves while its peer may still signal it
    if (warp == kMmaWarp) {
        __syncwarp();
        tc_fence_after();
        if constexpr (PAIR) tmem_dealloc_pair(tmem, S::kTmemCols);
        else tmem_dealloc(tmem, S::kTmemCols);
    }
}

// [rows][K] 8-bit matrix in boxes of `box_rows` rows x 128 bytes.
bool encode_rows(CUtensorMap* map, const int8_t* base, int rows, int K, int box_rows) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K)};
    const cuuint32_t box[2] = {kStepK, static_cast<cuuint32_t>(box_rows)};
    return tensor_map_encoder_ready() &&
           encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(base), dims, strides, box,
                        CU_TENSOR_MAP_SWIZZLE_NONE) == CUDA_SUCCESS;
}

template <bool PAIR, int BN, bool ALIGNED>
cudaError_t launch_variant(const Int8Params& p, int num_sms, cudaStream_t stream) {
    using S = Shape<PAIR, BN, ALIGNED>;
    static SmemLimitCache limits;
    auto* fn = int8_gemm_kernel<PAIR, BN, ALIGNED>;
    const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(fn), S::kSmem, limits);
    if (e != cudaSuccess) return e;
    constexpr int ctas = PAIR ? 2 : 1;
    const long long units = (static_cast<long long>(p.M) + 128 * ctas - 1) / (128 * ctas) * ((p.N + BN - 1) / BN);
    const int slots = num_sms / ctas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((units < slots ? units : slots) * ctas));
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 1 : 0;
    CUtensorMap map_x = {}, map_w = {};
    if (ALIGNED && (!encode_rows(&map_x, p.x, p.M, p.K, 128) || !encode_rows(&map_w, p.w, p.N, p.K, S::kRowsB)))
        return cudaErrorInvalidValue;
    return cudaLaunchKernelEx(&cfg, fn, p, map_x, map_w);
}

template <bool PAIR, int BN>
cudaError_t launch_aligned(const Int8Params& p, int num_sms, cudaStream_t stream) {
    if (p.K % 16 == 0) return launch_variant<PAIR, BN, true>(p, num_sms, stream);
    return launch_variant<PAIR, BN, false>(p, num_sms, stream);
}

}  // namespace

bool int8_gemm_fits(const Int8Params& p) {  // tile counts and row indexes in 32 bits
    return (static_cast<long long>(p.M) + 127) / 128 * ((p.N + 31) / 32) < (1LL << 30) && p.M < (1 << 30) && p.N < (1 << 30);
}

cudaError_t launch_int8_gemm(const Int8Params& p, int num_sms, cudaStream_t stream) {
    const long long m128 = (static_cast<long long>(p.M) + 127) / 128, m256 = (m128 + 1) / 2;
    const auto tiles = [&](int bn) { return (p.N + bn - 1) / bn; };
    if (m128 > 1 && m256 * tiles(256) >= num_sms / 4) return launch_aligned<true, 256>(p, num_sms, stream);
    if (m128 * tiles(128) >= num_sms / 2) return launch_aligned<false, 128>(p, num_sms, stream);
    if (m128 * tiles(64) >= num_sms / 2) return launch_aligned<false, 64>(p, num_sms, stream);
    return launch_aligned<false, 32>(p, num_sms, stream);
}

}  // namespace convgb
