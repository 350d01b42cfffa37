// int8_gemm.cu -- the 8-bit product on tcgen05 tensor cores:
//
//   y[m][n] = act( x_scale[m] * w_scale[n] * sum_k x[m][k] * w[n][k] + bias[n] )
//
// An 8-bit integer is exact in FP16 (11 significand bits), a product of two of them
// stays below 2^15 and the FP32 accumulator holds every partial sum below 2^24
// exactly, so the FP16 MMA gives the integer sum (always for K <= 1024).  This part's
// 8-bit integer tensor rate is a small fraction of its FP16 rate.
//
// The rows of x stay 8-bit up to the SM; converter warps bring them to FP16 and into
// tensor memory, from where the MMA takes its A operand:
//   x ^ 0x80 = x + 128 as an unsigned byte u; the FP16 bit pattern 0x6400 | u is
//   1024 + u; subtracting 1152 leaves x.  One exclusive-or, two byte permutes and two
//   packed subtractions for four values.
// The weights, far fewer than what they are multiplied with, are brought to FP16 in the
// workspace by a small kernel first and come in by TMA.  (Both operands converted into
// shared memory on their way in measured 246 us at 8192 x 4096 x 4096: the fence that
// shows a thread's shared-memory writes to the tensor core took ~1,800 clocks a stage, three
// and a half times the stage's MMAs.  Tensor memory needs no such fence.)
//
// Warp roles (576 threads, one CTA per SM, persistent over tiles):
//   warps 0..7    converters, two groups that take turns by stage; a warp holds 32 rows, a lane
//                 a row: K = 64 8-bit values from the raw ring, 32 registers of FP16 pairs,
//                 one store to tensor memory
//   warps 8..15   epilogue: two warps per 32-row quarter of tensor memory, 64 columns each:
//                 scales, bias, activation, rounding, stores from registers
//   warp 16       tensor memory; one lane issues tcgen05.mma and commits
//   warp 17       one lane fills the raw ring and the weight ring by TMA, K = 64 per slot
//
// Tensor memory: three accumulator regions of HN columns and four A stages of 32 columns.  A
// tile of NH * HN columns takes NH regions in turn, so the epilogue drains one tile while the
// next accumulates; with NH = 2 the next waits for the first of its two regions only.
//
// PAIR: two SMs share a tile of 256 rows (tcgen05.mma.cta_group::2): each converts its own 128
// rows of x and brings half of the weight rows.  Shared memory moves, per K = 64 and SM, 8 KB
// of x twice and 16 KB of weights twice in the 512 clocks of the MMAs: 96 of 128 bytes a clock.
//
// Columns: a lane of the epilogue reads accumulator columns 8 j + 2 q + {0, 1} of two rows
// (q = lane % 4, j = 0..7: the 16 x 256-bit shape).  The workspace holds weight row
// 16 q + 2 j + {0, 1} of each 64 there, so a lane holds 16 neighbouring outputs of a row, four
// lanes a 128-byte line of BF16, and a store instruction covers 8 whole lines.  (One row a
// lane, 32 lines touched per instruction, cost 38 us of 133 at 200704 x 256 -> 512; its 16-byte
// broadcast reads of the scales, four times as many as here, another 34.)
#include "int8_internal.h"
#include "pointwise_math.cuh"
#include "ptx.cuh"

namespace convgb {

namespace {

constexpr int kGroups = 2;       // converter groups
constexpr int kGroupWarps = 4;   // one for each quarter of tensor memory
constexpr int kConverterWarps = kGroups * kGroupWarps;
constexpr int kEpilogueWarps = 8;
constexpr int kMmaWarp = kConverterWarps + kEpilogueWarps;
constexpr int kLoadWarp = kMmaWarp + 1;
constexpr int kGemmThreads = 32 * (kLoadWarp + 1);
constexpr int kStepK = 64;       // K of one stage
constexpr int kStagesA = 4;      // FP16 stages of x in tensor memory
constexpr int kColsA = kStepK / 2;
constexpr int kRegions = 3;      // accumulators
constexpr int kRaw = 128 * kStepK;  // one slot of 8-bit rows

// HN: columns of one MMA; NH: MMAs side by side in a tile.
template <bool PAIR, int HN, int NH>
struct Shape {
    static constexpr int kCtas = PAIR ? 2 : 1;
    static constexpr int kTileN = HN * NH;
    static constexpr int kBoxB = HN / kCtas;                 // weight rows a CTA brings for one MMA
    static constexpr int kSliceB = kBoxB * kStepK * 2;
    static constexpr int kStageB = NH * kSliceB;
    static constexpr int kStagesB = kStageB >= 32768 ? 4 : 8;
    static constexpr int kRawSlots = 8;
    static constexpr int kA0 = kRegions * HN;                // first column of the A stages
    static constexpr int kTmemCols = kA0 + kStagesA * kColsA <= 256 ? 256 : 512;
    static constexpr int kSmem = kStagesB * kStageB + kRawSlots * kRaw + 2 * 2 * HN * 4 + 512;
};

struct Bars {
    uint64_t *rfull, *rempty;  // 8-bit rows
    uint64_t *afull, *aempty;  // FP16 rows in tensor memory
    uint64_t *bfull, *bempty;  // weights
    uint64_t *tfull, *tempty;  // accumulators
    uint64_t *drain, *esync;
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

// 32 rows (lanes) x 32 columns into tensor memory.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] * B[smem]^T, FP16 operands, FP32 accumulate.
template <bool PAIR>
__device__ __forceinline__ void mma_f16_ta(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
            "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
            "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
}

__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {  // as idesc_bf16_f32 with FP16 operands (type 0)
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// A CTA's (or pair's) way through the tiles of a launch, n fastest, without a division per tile.
struct Tiles {
    int n_tiles, units, step, step_m, step_n;
};

struct Walk {
    int u, mu, nt;
};

__device__ __forceinline__ Walk walk_from(const Tiles& t, int unit0) {
    Walk w;
    w.u = unit0;
    w.mu = unit0 / t.n_tiles;
    w.nt = unit0 - w.mu * t.n_tiles;
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

// A ring slot and the phase of its barriers.
struct Slot {
    int i;
    uint32_t phase;
    __device__ __forceinline__ void next(int slots, int by = 1) {
        if ((i += by) >= slots) {
            i -= slots;
            phase ^= 1u;
        }
    }
};

// MMAs (of HN columns) that the tile's columns take.
template <int HN, int NH>
__device__ __forceinline__ int parts_of(const Int8Params& p, int nt) {
    return NH == 2 && nt * HN * NH + HN >= p.N ? 1 : NH;
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

// A lane's part of 16 rows x 64 columns: 16 neighbouring columns of two rows.
template <int ACT>
__device__ __forceinline__ void finish_block(uint32_t (&v)[32], float xs_lo, float xs_hi, const float* scale,
                                             const float* bias) {
    uint64_t lo2, hi2;
    asm("mov.b64 %0, {%1, %1};" : "=l"(lo2) : "f"(xs_lo));
    asm("mov.b64 %0, {%1, %1};" : "=l"(hi2) : "f"(xs_hi));
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const ulonglong2 s = *reinterpret_cast<const ulonglong2*>(scale + 2 * j);
        const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(bias + 2 * j);
        finish_two<ACT>(v[4 * j], v[4 * j + 1], lo2, s.x, b.x);
        finish_two<ACT>(v[4 * j + 2], v[4 * j + 3], hi2, s.x, b.x);
        finish_two<ACT>(v[4 * j + 4], v[4 * j + 5], lo2, s.y, b.y);
        finish_two<ACT>(v[4 * j + 6], v[4 * j + 7], hi2, s.y, b.y);
    }
}

// 16 neighbouring outputs of row h of a lane's two, in the widest stores that every row's start
// allows (wide: 32 or 16 bytes; 0: one by one).
__device__ __forceinline__ void store_row(const Int8Params& p, const uint32_t (&v)[32], int h, long long row, int n, int wide) {
    const auto at = [&](int i) { return v[4 * (i >> 1) + 2 * h + (i & 1)]; };  // column n + i
    const long long o = row * p.N + n;
    if (n + 16 <= p.N && wide != 0) {
        if (p.out_bf16) {
            uint32_t q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = pack_bf16x2(__uint_as_float(at(2 * i)), __uint_as_float(at(2 * i + 1)));
            __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + o;
            if (wide == 32) {
                store_v8(y, q[0], q[1], q[2], q[3], q[4], q[5], q[6], q[7]);
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    reinterpret_cast<uint4*>(y)[i] = make_uint4(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
            }
        } else {
            float* y = static_cast<float*>(p.y) + o;
            if (wide == 32) {
#pragma unroll
                for (int i = 0; i < 16; i += 8)
                    store_v8(y + i, at(i), at(i + 1), at(i + 2), at(i + 3), at(i + 4), at(i + 5), at(i + 6), at(i + 7));
            } else {
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    *reinterpret_cast<uint4*>(y + i) = make_uint4(at(i), at(i + 1), at(i + 2), at(i + 3));
            }
        }
        return;
    }
    if (p.out_bf16) {
        __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + o;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (n + i < p.N) y[i] = __float2bfloat16_rn(__uint_as_float(at(i)));
    } else {
        float* y = static_cast<float*>(p.y) + o;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (n + i < p.N) y[i] = __uint_as_float(at(i));
    }
}

template <bool PAIR, int HN, int NH>
__global__ void __launch_bounds__(kGemmThreads, 1)
    int8_gemm_kernel(const Int8Params p, const __grid_constant__ CUtensorMap map_x,
                     const __grid_constant__ CUtensorMap map_w) {
    using S = Shape<PAIR, HN, NH>;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_addr(smem) & 1023u) {  // the swizzle's atoms; uniform, so no CTA waits for another
        record_status(p.status, kStatusTimeoutMma, nullptr);
        return;
    }
    uint8_t* raw = smem + S::kStagesB * S::kStageB;
    float* col_scale = reinterpret_cast<float*>(raw + S::kRawSlots * kRaw);  // of two accumulators in turn
    float* col_bias = col_scale + 2 * HN;
    Bars b;
    b.rfull = reinterpret_cast<uint64_t*>(col_bias + 2 * HN);
    b.rempty = b.rfull + S::kRawSlots;
    b.afull = b.rempty + S::kRawSlots;
    b.aempty = b.afull + kStagesA;
    b.bfull = b.aempty + kStagesA;
    b.bempty = b.bfull + S::kStagesB;
    b.tfull = b.bempty + S::kStagesB;
    b.tempty = b.tfull + kRegions;
    b.drain = b.tempty + kRegions;
    b.esync = b.drain + 1;
    b.tmem_slot = reinterpret_cast<uint32_t*>(b.esync + 1);
    b.abort = reinterpret_cast<int*>(b.tmem_slot + 1);
    volatile int* abort = b.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
    const bool leader = rank == 0;
    constexpr int kCtas = S::kCtas;

    Tiles tiles;
    tiles.n_tiles = (p.N + S::kTileN - 1) / S::kTileN;
    tiles.units = ((p.M + 128 * kCtas - 1) / (128 * kCtas)) * tiles.n_tiles;
    tiles.step = static_cast<int>(gridDim.x) / kCtas;
    tiles.step_m = tiles.step / tiles.n_tiles;
    tiles.step_n = tiles.step - tiles.step_m * tiles.n_tiles;
    const int unit0 = static_cast<int>(blockIdx.x) / kCtas, units = tiles.units;
    const int ksteps = (p.K + kStepK - 1) / kStepK;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kRawSlots; ++s) {
            mbar_init(&b.rfull[s], 1);
            mbar_init(&b.rempty[s], kGroupWarps);
        }
        for (int s = 0; s < kStagesA; ++s) {
            mbar_init(&b.afull[s], kCtas * kGroupWarps);
            mbar_init(&b.aempty[s], 1);
        }
        for (int s = 0; s < S::kStagesB; ++s) {
            mbar_init(&b.bfull[s], 1);
            mbar_init(&b.bempty[s], 1);
        }
        for (int i = 0; i < kRegions; ++i) {
            mbar_init(&b.tfull[i], 1);
            mbar_init(&b.tempty[i], kCtas * kEpilogueWarps);
        }
        mbar_init(b.drain, 1);
        mbar_init(b.esync, kEpilogueWarps);
        *b.abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&map_x);
        tma_prefetch_desc(&map_w);
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
        const int group = warp / kGroupWarps;  // converts steps group, group + 2, ...
        const int quarter = warp & 3;
        const int my_units = unit0 < units ? (units - 1 - unit0) / tiles.step + 1 : 0;
        const long long steps = static_cast<long long>(my_units) * ksteps;
        const int row = quarter * 32 + lane;
        const uint32_t swz = static_cast<uint32_t>((row >> 1) & 3);  // 64-byte swizzle of the raw rows
        Slot rs{group, 0}, as{group, 0};
        for (long long s = group; s < steps; s += kGroups) {
            if (!warp_wait(&b.rfull[rs.i], rs.phase, abort)) {
                record_status(p.status, kStatusTimeoutTransform, abort);
                break;
            }
            const uint8_t* src = raw + rs.i * kRaw + row * kStepK;
            uint4 item[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) item[c] = *reinterpret_cast<const uint4*>(src + ((c ^ swz) << 4));
            uint32_t v[32];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t w[4] = {item[c].x, item[c].y, item[c].z, item[c].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint2 h = to_half4(w[i]);
                    v[8 * c + 2 * i] = h.x;
                    v[8 * c + 2 * i + 1] = h.y;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&b.rempty[rs.i]);
            if (!warp_wait(&b.aempty[as.i], as.phase ^ 1u, abort)) {
                record_status(p.status, kStatusTimeoutTransform, abort);
                break;
            }
            tc_fence_after();
            tmem_st32(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + S::kA0 + as.i * kColsA, v);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR) mbar_arrive_remote(mapa_shared(smem_addr(&b.afull[as.i]), 0));
                else mbar_arrive(&b.afull[as.i]);
            }
            rs.next(S::kRawSlots, kGroups);
            as.next(kStagesA, kGroups);
        }
    } else if (warp < kMmaWarp) {
        // ------------------------------------------------------------ epilogue
        const int quarter = warp & 3;
        const int half = (warp - kConverterWarps) >> 2;
        const int et = threadIdx.x - 32 * kConverterWarps;
        const int es = p.out_bf16 ? 2 : 4;
        const long long row_bytes = static_cast<long long>(p.N) * es;
        const uintptr_t y0 = reinterpret_cast<uintptr_t>(p.y);
        const int wide = row_bytes % 32 == 0 && y0 % 32 == 0 ? 32 : (row_bytes % 16 == 0 ? 16 : 0);
        // 128 columns: each warp drains 64 of them, all 32 rows; 64 columns: 16 of the rows
        const int col = HN == 128 ? 64 * half : 0;
        const int mine = col + (lane & 3) * 16;  // this lane's first column
        uint32_t eph = 0;
        int turn = 0;  // which of the two scale buffers
        Slot rg{0, 0};
        bool ok = true;
        for (Walk w = walk_from(tiles, unit0); w.u < units && ok; next_unit(tiles, w)) {
            const long long row0 = static_cast<long long>(w.mu) * 128 * kCtas + rank * 128 + quarter * 32 + (lane >> 2);
            float xs[4];  // rows row0, + 8, + 16, + 24
#pragma unroll
            for (int i = 0; i < 4; ++i) xs[i] = row0 + 8 * i < p.M ? __ldg(p.x_scale + row0 + 8 * i) : 0.0f;
            const int parts = parts_of<HN, NH>(p, w.nt);
            for (int part = 0; part < parts; ++part) {
                const int n0 = w.nt * S::kTileN + part * HN;
                // a scale or a bias a thread, on its way while the MMAs finish
                const int c = et & (HN - 1);
                const float* from = et < HN ? p.w_scale : (et < 2 * HN ? p.bias : nullptr);
                const float cv = from != nullptr && n0 + c < p.N ? __ldg(from + n0 + c) : 0.0f;
                ok = warp_wait_cluster(&b.tfull[rg.i], rg.phase, abort);
                if (ok) {
                    // Every warp passes this once it is done with the columns before last, whose buffer this is.
                    if (et < 2 * HN) (et < HN ? col_scale : col_bias)[turn * HN + c] = cv;
                    ok = epilogue_sync(b.esync, eph, abort);
                }
                if (!ok) {
                    record_status(p.status, kStatusTimeoutEpilogue, abort);
                    break;
                }
                tc_fence_after();
                if (n0 + col < p.N) {
                    const float* sc = col_scale + turn * HN + mine;
                    const float* bi = col_bias + turn * HN + mine;
                    const int n = n0 + mine;
#pragma unroll
                    for (int g = 0; g < 2; ++g) {  // 16 rows at a time
                        if (HN < 128 && g != half) continue;
                        uint32_t v[32];
                        tmem_ld_16x64(tmem + (static_cast<uint32_t>(quarter * 32 + 16 * g) << 16) + rg.i * HN + col, v);
                        tmem_ld_wait(v);
                        if (p.act == CONV_ACT_RELU) finish_block<CONV_ACT_RELU>(v, xs[2 * g], xs[2 * g + 1], sc, bi);
                        else if (p.act == CONV_ACT_SILU) finish_block<CONV_ACT_SILU>(v, xs[2 * g], xs[2 * g + 1], sc, bi);
                        else finish_block<CONV_ACT_NONE>(v, xs[2 * g], xs[2 * g + 1], sc, bi);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const long long row = row0 + 16 * g + 8 * h;
                            if (row < p.M && n < p.N) store_row(p, v, h, row, n, wide);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR) mbar_arrive_remote(mapa_shared(smem_addr(&b.tempty[rg.i]), 0));
                    else mbar_arrive(&b.tempty[rg.i]);
                }
                rg.next(kRegions);
                turn ^= 1;
            }
        }
    } else if (warp == kLoadWarp) {
        // ------------------------------------------------------------ raw rows and weights
        if (lane == 0) {
            Slot rs{0, 0}, bs{0, 0};
            long long issued = 0;
            bool ok = true;
            for (Walk w = walk_from(tiles, unit0); w.u < units && ok; next_unit(tiles, w)) {
                const int m0 = w.mu * 128 * kCtas + static_cast<int>(rank) * 128;
                const int parts = parts_of<HN, NH>(p, w.nt);
                for (int ks = 0; ks < ksteps; ++ks) {
                    ok = mbar_wait(&b.rempty[rs.i], rs.phase ^ 1u, abort) && mbar_wait(&b.bempty[bs.i], bs.phase ^ 1u, abort);
                    if (!ok) {
                        record_status(p.status, kStatusTimeoutProducer, abort);
                        break;
                    }
                    mbar_arrive_expect_tx(&b.rfull[rs.i], kRaw);
                    tma_load_2d(raw + rs.i * kRaw, &map_x, &b.rfull[rs.i], ks * kStepK, m0);  // past the matrix: zeros
                    if (leader) mbar_arrive_expect_tx(&b.bfull[bs.i], kCtas * parts * S::kSliceB);
                    for (int part = 0; part < parts; ++part) {
                        uint8_t* dst = smem + bs.i * S::kStageB + part * S::kSliceB;
                        const int n = w.nt * S::kTileN + part * HN + static_cast<int>(rank) * S::kBoxB;
                        if constexpr (PAIR)
                            tma_load_2d_pair(dst, &map_w, mapa_shared(smem_addr(&b.bfull[bs.i]), 0), ks * kStepK, n);
                        else
                            tma_load_2d(dst, &map_w, &b.bfull[bs.i], ks * kStepK, n);
                    }
                    ++issued;
                    rs.next(S::kRawSlots);
                    bs.next(S::kStagesB);
                }
            }
            // No copy of this CTA in flight when it leaves.  The pair's second CTA sees its weight
            // copies land by the MMAs' release of the slot.
            for (int s = 0; s < S::kRawSlots; ++s) {
                const long long fills = issued / S::kRawSlots + (s < issued % S::kRawSlots ? 1 : 0);
                if (fills && !mbar_wait(&b.rfull[s], static_cast<uint32_t>((fills - 1) & 1), nullptr))
                    record_status(p.status, kStatusTimeoutDrain, abort);
            }
            for (int s = 0; s < S::kStagesB; ++s) {
                const long long fills = issued / S::kStagesB + (s < issued % S::kStagesB ? 1 : 0);
                if (fills && !mbar_wait(leader ? &b.bfull[s] : &b.bempty[s], static_cast<uint32_t>((fills - 1) & 1), nullptr))
                    record_status(p.status, kStatusTimeoutDrain, abort);
            }
        }
    } else if (lane == 0 && leader) {
        // ------------------------------------------------------------ MMA
        constexpr uint32_t idesc = idesc_f16_f32(128 * kCtas, HN);
        Slot as{0, 0}, bs{0, 0}, rg{0, 0};
        bool ok = true;
        for (Walk w = walk_from(tiles, unit0); w.u < units && ok; next_unit(tiles, w)) {
            const int parts = parts_of<HN, NH>(p, w.nt);
            Slot mine[NH];
            for (int part = 0; part < NH; ++part) {
                mine[part] = rg;
                if (part < parts) {
                    ok = ok && mbar_wait_cluster(&b.tempty[rg.i], rg.phase ^ 1u, abort);
                    rg.next(kRegions);
                }
            }
            for (int ks = 0; ks < ksteps && ok; ++ks) {
                ok = mbar_wait_cluster(&b.bfull[bs.i], bs.phase, abort) && mbar_wait_cluster(&b.afull[as.i], as.phase, abort);
                if (!ok) break;
                tc_fence_after();
                const int left = (p.K - ks * kStepK + 15) >> 4;
                const int mmas = left < 4 ? left : 4;
                const uint64_t db = sdesc_sw128(smem_addr(smem + bs.i * S::kStageB));
                const uint32_t da = tmem + S::kA0 + as.i * kColsA;
#pragma unroll
                for (int part = 0; part < NH; ++part) {
                    if (part >= parts) break;
                    const uint32_t d = tmem + mine[part].i * HN;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (j >= mmas) break;
                        mma_f16_ta<PAIR>(d, da + 8 * j, db + part * (S::kSliceB >> 4) + 2 * j, idesc, (ks | j) != 0 ? 1u : 0u);
                    }
                }
                if constexpr (PAIR) {
                    mma_commit_pair(&b.aempty[as.i], 3);
                    mma_commit_pair(&b.bempty[bs.i], 3);
                } else {
                    mma_commit(&b.aempty[as.i]);
                    mma_commit(&b.bempty[bs.i]);
                }
                as.next(kStagesA);
                bs.next(S::kStagesB);
            }
            if (!ok) {
                record_status(p.status, kStatusTimeoutMma, abort);
                break;
            }
            for (int part = 0; part < parts; ++part) {
                if constexpr (PAIR) mma_commit_pair(&b.tfull[mine[part].i], 3);
                else mma_commit(&b.tfull[mine[part].i]);
            }
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

// ---------------------------------------------------------------- operands laid out
// Weights to FP16, [N rounded up to 64][pitch], rows of each 64 in the order of the accumulator's
// columns (the header comment); and, where rows of x do not start on 16 bytes, a copy of x that
// does.  One thread per 16 values; the rows and columns that only pad are not written: they
// reach no result that is stored (the TMA reads K columns, zeros after them).
__device__ __forceinline__ int column_of(int n) {
    return (n & ~63) | ((n & 14) << 2) | ((n & 48) >> 3) | (n & 1);
}

__global__ void __launch_bounds__(256) int8_layout_kernel(const Int8Params p) {
    const int chunks = (p.K + 15) >> 4;
    const long long w_items = static_cast<long long>(p.N) * chunks;
    const long long items = w_items + (p.x_rows != nullptr ? static_cast<long long>(p.M) * chunks : 0);
    for (long long i = blockIdx.x * 256LL + threadIdx.x; i < items; i += gridDim.x * 256LL) {
        const bool is_w = i < w_items;
        const long long at = is_w ? i : i - w_items;
        const long long row = at / chunks;
        const int k = static_cast<int>(at - row * chunks) * 16;
        const int len = p.K - k < 16 ? p.K - k : 16;
        const uint4 v = load_item(is_w ? p.w : p.x, row * p.K + k, len, static_cast<long long>(is_w ? p.N : p.M) * p.K);
        if (is_w) {
            uint16_t* dst = p.w_rows + static_cast<long long>(column_of(static_cast<int>(row))) * p.pitch + k;
            const uint2 a = to_half4(v.x), b = to_half4(v.y), c = to_half4(v.z), d = to_half4(v.w);
            reinterpret_cast<uint4*>(dst)[0] = make_uint4(a.x, a.y, b.x, b.y);
            reinterpret_cast<uint4*>(dst)[1] = make_uint4(c.x, c.y, d.x, d.y);
        } else {
            *reinterpret_cast<uint4*>(p.x_rows + row * p.pitch + k) = v;
        }
    }
}

// [rows][K] matrix, rows `pitch_bytes` apart, in boxes of `box_rows` rows x K = 64.
bool encode_rows(CUtensorMap* map, CUtensorMapDataType type, const void* base, long long rows, int K, size_t pitch_bytes,
                 int box_rows, CUtensorMapSwizzle swizzle) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {pitch_bytes};
    const cuuint32_t box[2] = {kStepK, static_cast<cuuint32_t>(box_rows)};
    return tensor_map_encoder_ready() &&
           encode_tiled(map, type, 2, const_cast<void*>(base), dims, strides, box, swizzle) == CUDA_SUCCESS;
}

template <bool PAIR, int HN, int NH>
cudaError_t launch_variant(const Int8Params& p, int num_sms, cudaStream_t stream) {
    using S = Shape<PAIR, HN, NH>;
    static SmemLimitCache limits;
    auto* fn = int8_gemm_kernel<PAIR, HN, NH>;
    const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(fn), S::kSmem, limits);
    if (e != cudaSuccess) return e;
    const long long units = (static_cast<long long>(p.M) + 128 * S::kCtas - 1) / (128 * S::kCtas) * ((p.N + S::kTileN - 1) / S::kTileN);
    const int slots = num_sms / S::kCtas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((units < slots ? units : slots) * S::kCtas));
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = S::kCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 1 : 0;
    CUtensorMap map_x = {}, map_w = {};
    const bool copied = p.x_rows != nullptr;
    if (!encode_rows(&map_x, CU_TENSOR_MAP_DATA_TYPE_UINT8, copied ? p.x_rows : p.x, p.M, p.K, copied ? p.pitch : p.x_pitch, 128,
                     CU_TENSOR_MAP_SWIZZLE_64B) ||
        !encode_rows(&map_w, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p.w_rows, (p.N + 63) & ~63, p.K, 2 * static_cast<size_t>(p.pitch),
                     S::kBoxB, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    return cudaLaunchKernelEx(&cfg, fn, p, map_x, map_w);
}

}  // namespace

bool int8_gemm_fits(const Int8Params& p) {  // tile counts and row indexes in 32 bits
    return (static_cast<long long>(p.M) + 127) / 128 * ((p.N + 63) / 64) < (1LL << 30) && p.M < (1 << 30) && p.N < (1 << 30);
}

cudaError_t launch_int8_layout(const Int8Params& p, int num_sms, cudaStream_t stream) {
    const long long rows = static_cast<long long>(p.N) + (p.x_rows != nullptr ? p.M : 0);
    const long long blocks = (rows * ((p.K + 15) / 16) + 255) / 256;
    int8_layout_kernel<<<static_cast<unsigned>(blocks < 8LL * num_sms ? blocks : 8LL * num_sms), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_int8_gemm(const Int8Params& p, int num_sms, cudaStream_t stream) {
    const long long m128 = (static_cast<long long>(p.M) + 127) / 128, m256 = (m128 + 1) / 2;
    const auto tiles = [&](int bn) { return (p.N + bn - 1) / bn; };
    if (m128 > 1 && m256 * tiles(256) >= num_sms / 4) return launch_variant<true, 128, 2>(p, num_sms, stream);
    if (m128 * tiles(128) >= num_sms / 2) return launch_variant<false, 128, 1>(p, num_sms, stream);
    return launch_variant<false, 64, 1>(p, num_sms, stream);
}

}  // namespace convgb
