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
//   warps 0..7    converters, four groups that take turns by stage, so one loads, converts,
//                 publishes or waits while the others do: 8-bit rows from the raw ring to FP16
//                 values in the 128-byte-swizzle operand tiles of a stage
//   warps 8..23   epilogue: four warps per 32-row quarter of tensor memory, a quarter of the
//                 columns each: scales, bias, activation, rounding, output.  (Eight warps took
//                 ~7,000 clocks a 256 x 256 tile, which at K = 256 is 1.6 times its MMAs; the
//                 converters had warps to spare.)
//   warp 24       tensor memory; one lane issues tcgen05.mma and commits
//   warp 25       one lane fills the raw ring by TMA: K = 64 of both operands, 8-bit, per slot
// Rows that do not start on 16 bytes (K % 16) are beyond the TMA: a kernel of its own copies
// them to rows that do, in the workspace, first.
// A stage holds K = 64 of both operands, one 128-byte FP16 row each.  Tensor memory holds two
// accumulators, so the epilogue of one tile overlaps the next one's MMAs.
//
// Columns: a lane of the epilogue reads accumulator columns 8 j + 2 q + {0, 1} of two rows
// (q = lane % 4, j = 0..3: the 16 x 256-bit shape).  The converters put weight row
// 8 q + 2 j + {0, 1} of each 32 there, so a lane holds 8 neighbouring outputs of a row, four
// lanes 64 bytes of BF16.  (One row a lane, 32 lines
// touched per instruction, cost 38 us of 133 at 200704 x 256 -> 512; scales read through shared
// memory, which the operands keep busy, another 34.)
//
// Measured (cold caches, launch included): 8192 x 4096 x 4096, 8-bit input, 215 us, 1,278 TFLOP/s,
// 69 % of the card's measured BF16 matrix rate: with the converters' stores left out the same
// kernel takes 174 us, so a fifth is shared memory's share (per K = 64 and SM of a pair: 16 KB
// raw in, 16 KB out, 32 KB FP16 in, 32 KB to the MMA, 768 clocks at 128 bytes against 512 of MMA).
// 200704 x 256 -> 512: 68 us, 56 % of the memory's rate over its 257 MB.  256 x 4096 -> 4096: 23 us in a graph.
//
// PAIR: two SMs share a 256 x BN tile (tcgen05.mma.cta_group::2): each converts its own
// 128 rows of x and BN / 2 rows of w.  Shared memory bounds this kernel (written by the
// converters, read by the MMA), and a pair halves the traffic of w.
//
// Few tiles: a cluster of up to 8 CTAs splits the K of one tile (p.splits).  Each leaves its sums in
// its shared memory; after a cluster barrier each finishes its share of the rows, adding the
// parts in one order.
//
// Rows past M or N are neither loaded nor written: their outputs are never stored, and
// one row's operand does not reach another row's result.  Past K both operands are 0.
#include "int8_internal.h"
#include "int8_rows.cuh"
#include "pointwise_math.cuh"
#include "ptx.cuh"

namespace convgb {

namespace {

constexpr int kGroups = 4;       // converter groups
constexpr int kGroupWarps = 2;
constexpr int kConverterWarps = kGroups * kGroupWarps;
constexpr int kEpilogueWarps = 16;
constexpr int kMmaWarp = kConverterWarps + kEpilogueWarps;
constexpr int kLoadWarp = kMmaWarp + 1;
constexpr int kGemmThreads = 32 * (kLoadWarp + 1);
constexpr int kStepK = 64;       // K of one stage
constexpr int kRowBytes = 128;   // one FP16 operand row of a stage

template <bool PAIR, int BN>
struct Shape {
    static constexpr int kRowsB = PAIR ? BN / 2 : BN;
    static constexpr int kTileA = 128 * kRowBytes;
    static constexpr int kStage = kTileA + kRowsB * kRowBytes;
    static constexpr int kStages = kGroups;              // one for each converter group
    static constexpr int kRaw = (128 + kRowsB) * kStepK;  // one slot of the raw ring
    static constexpr int kRawSlots = kRowsB >= 128 ? 4 : 8;  // in 227 KB beside the stages and the outputs
    static constexpr int kOut = 2048;                    // an epilogue warp's block of BF16 outputs
    static constexpr int kPartRow = BN + 8;              // floats of a row of partial sums (K split over a cluster)
    static constexpr int kItemsB = kRowsB / 16;          // 16-byte items of w a converter thread moves per stage (of x: 8)
    static constexpr int kTmemCols = 2 * BN < 32 ? 32 : 2 * BN;
    static constexpr int kSmem = kStages * kStage + kRawSlots * kRaw + kEpilogueWarps * kOut + 256;
};

struct Bars {
    uint64_t* rfull;
    uint64_t* rempty;
    uint64_t* full;
    uint64_t* empty;
    uint64_t* tfull;
    uint64_t* tempty;
    uint64_t* drain;
    uint32_t* tmem_slot;
    int* abort;
};

// Arrive on the pair leader's barrier.  What it announces is ordered by other means: operand
// tiles by the proxy fence before it, tensor memory by tcgen05's own fences; it orders no memory
// of its own.  With release at cluster scope it held its warp for ~1,800 clocks, three and a half
// times a stage's MMAs (8192 x 4096 x 4096: 246 us, and 217 us as it is).
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(mapa_shared(smem_addr(bar), 0)) : "memory");
}

// A bounded wait whose answer is the same in every lane.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}

__device__ __forceinline__ bool warp_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort) {
    return __all_sync(0xffffffffu, mbar_wait_cluster(bar, parity, abort));
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
    int k_begin, k_end;  // the CTA's part of K
    uint32_t rank;       // of a pair
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
    w.k0 = t.k_begin;
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
__device__ __forceinline__ void advance(const Tiles& t, Walk& w, int steps) {
    for (int i = 0; i < steps && w.u < t.units; ++i) {
        w.k0 += kStepK;
        if (w.k0 >= t.k_end) {
            w.k0 = t.k_begin;
            next_unit(t, w);
            place<PAIR, BN>(t, w);
        }
    }
}

// The stage's row (accumulator column) of weight row n: columns 8 q + 2 j + e of each 32 sit at
// 8 j + 2 q + e.
__device__ __forceinline__ int column_of(int n) { return (n & ~31) | ((n & 6) << 2) | ((n & 24) >> 2) | (n & 1); }

// COUNT items of one operand (rows r0, r0 + 16, ...) to its FP16 tile.
template <int COUNT, bool WEIGHTS>
__device__ __forceinline__ void store_items(int rows_left, int r0, int c, const uint4 (&item)[COUNT], uint8_t* tile) {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
        int row = r0 + 16 * i;
        if (row >= rows_left) continue;
        const uint2 a = to_half4(item[i].x), b = to_half4(item[i].y), d = to_half4(item[i].z), e = to_half4(item[i].w);
        if (WEIGHTS) row = column_of(row);
        uint8_t* dst = tile + row * kRowBytes;
        const int sw = row & 7;  // eight lanes: four chunks of two rows, eight bank groups
        *reinterpret_cast<uint4*>(dst + (((2 * c) ^ sw) << 4)) = make_uint4(a.x, a.y, b.x, b.y);
        *reinterpret_cast<uint4*>(dst + (((2 * c + 1) ^ sw) << 4)) = make_uint4(d.x, d.y, e.x, e.y);
    }
}

// 16 lanes (rows) x 32 columns of tensor memory: register 4 j + 2 h + e of a lane is row
// lane / 4 + 8 h, column 8 j + 2 (lane % 4) + e.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// Waits for this thread's tcgen05.ld, tied to the registers so that no use moves before it.
__device__ __forceinline__ void tmem_ld_wait16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

// Eight neighbouring FP32 values from element n of v (n a multiple of 8), zero past N or without v,
// as four packed pairs.
template <bool WHOLE>
__device__ __forceinline__ void load_pairs(const float* v, int n, int N, uint64_t (&pair)[4]) {
    if constexpr (WHOLE) {
        pair[0] = pair[1] = pair[2] = pair[3] = 0;
        if (v == nullptr) return;
        const ulonglong2 a = __ldg(reinterpret_cast<const ulonglong2*>(v + n));
        const ulonglong2 b = __ldg(reinterpret_cast<const ulonglong2*>(v + n + 4));
        pair[0] = a.x;
        pair[1] = a.y;
        pair[2] = b.x;
        pair[3] = b.y;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float lo = v != nullptr && n + 2 * j < N ? __ldg(v + n + 2 * j) : 0.0f;
            const float hi = v != nullptr && n + 2 * j + 1 < N ? __ldg(v + n + 2 * j + 1) : 0.0f;
            asm("mov.b64 %0, {%1, %2};" : "=l"(pair[j]) : "f"(lo), "f"(hi));
        }
    }
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

// A lane's part of 16 rows x 32 columns: 8 neighbouring columns of two rows.
template <int ACT>
__device__ __forceinline__ void finish_block(uint32_t (&v)[16], float xs_lo, float xs_hi, const uint64_t (&ws)[4],
                                             const uint64_t (&bias)[4]) {
    uint64_t lo2, hi2;
    asm("mov.b64 %0, {%1, %1};" : "=l"(lo2) : "f"(xs_lo));
    asm("mov.b64 %0, {%1, %1};" : "=l"(hi2) : "f"(xs_hi));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        finish_two<ACT>(v[4 * j], v[4 * j + 1], lo2, ws[j], bias[j]);
        finish_two<ACT>(v[4 * j + 2], v[4 * j + 3], hi2, ws[j], bias[j]);
    }
}

// 8 neighbouring outputs of row h of a lane's two (columns 8 q .. of row `row` of the block) to the
// warp's buffer: 64-byte rows with 64-byte swizzle (BF16) or 128 with 128 (FP32), so the eight lanes
// of a wavefront write 128 bytes.
template <bool BF16>
__device__ __forceinline__ uint8_t* block_byte(uint8_t* block, int row, int byte) {
    if constexpr (BF16) return block + row * 64 + (((byte >> 4) ^ ((row >> 1) & 3)) << 4) + (byte & 15);
    else return block + row * 128 + (((byte >> 4) ^ (row & 7)) << 4) + (byte & 15);
}

template <bool BF16>
__device__ __forceinline__ void stage_row(uint8_t* block, int row, int q, const uint32_t (&v)[16], int h) {
    const auto at = [&](int i) { return v[4 * (i >> 1) + 2 * h + (i & 1)]; };  // column 8 q + i
    if constexpr (BF16) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = pack_bf16x2(__uint_as_float(at(2 * i)), __uint_as_float(at(2 * i + 1)));
        *reinterpret_cast<uint4*>(block_byte<BF16>(block, row, 16 * q)) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
        *reinterpret_cast<uint4*>(block_byte<BF16>(block, row, 32 * q)) = make_uint4(at(0), at(1), at(2), at(3));
        *reinterpret_cast<uint4*>(block_byte<BF16>(block, row, 32 * q + 16)) = make_uint4(at(4), at(5), at(6), at(7));
    }
}

// The block's 16 rows to rows of y that start on a multiple of T's size, neighbouring lanes at
// neighbouring places.  columns: of y from the block's first on (a whole number of Ts).
template <bool BF16, typename T>
__device__ __forceinline__ void store_rows(uint8_t* y, long long row_bytes, int rows, int columns, uint8_t* block) {
    constexpr int kRow = BF16 ? 64 : 128, kLanes = kRow / static_cast<int>(sizeof(T)), kRows = kLanes >= 32 ? 1 : 32 / kLanes;
    const int lane = threadIdx.x & 31, first = lane / kLanes, byte = (lane % kLanes) * static_cast<int>(sizeof(T));
    if (byte >= columns * (BF16 ? 2 : 4)) return;
    y += first * row_bytes + byte;
    // Reads under way: of 128 columns, 2-byte stores, two 3.1 us a tile and eight 2.8; 4-byte ones of FP32 on a
    // pair 6.0 and 7.4.
    constexpr int kBatch = BF16 ? (16 / kRows < 8 ? 16 / kRows : 8) : 2;
#pragma unroll 1
    for (int i = first; i < 16; i += kBatch * kRows) {
        T v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) v[k] = *reinterpret_cast<const T*>(block_byte<BF16>(block, i + k * kRows, byte));
#pragma unroll
        for (int k = 0; k < kBatch; ++k, y += kRows * row_bytes)
            if (i + k * kRows < rows) *reinterpret_cast<T*>(y) = v[k];
    }
}

// What an epilogue warp drains of a tile: its columns in blocks of 32, 16 or 32 rows of them.
struct Drain {
    uint32_t at;  // tensor memory of its first row and column
    int n;        // this lane's first column
    float xs[4];  // scales of this lane's rows, 8 apart
    uint8_t* out;  // the warp's buffer
    const CUtensorMap* map;
    int block_n, block_m;  // the block's place in y
};

// G: 16-row groups of the quarter that this warp drains.  A block goes through shared memory: out in
// one or two bulk stores of 16 rows, which clip what lies past M and N (TMA), or, where rows
// of y do not all start on 16 bytes, in coalesced stores of as many bytes as they start on.
// Straight from registers a store touches 8 lines, of which it fills half at best (200704 x 256 -> 512,
// 8-bit input, eight epilogue warps: 86 us straight, 85 through the TMA), and in single elements an
// eighth (20763 x 170 -> 1035, 8-bit input, BF16: 104 us, 43 from the buffer).
template <int ACT, bool BF16, bool WHOLE, bool TMA, int G>
__device__ __forceinline__ void drain_block(const Int8Params& p, const Drain& d) {
    constexpr int kTurn = BF16 ? G : 1;  // groups that the buffer holds at a time
    const int lane = threadIdx.x & 31;
    uint64_t ws[4], bias[4];
#pragma unroll
    for (int t = 0; t < G; t += kTurn) {
        uint32_t v[kTurn][16];
#pragma unroll
        for (int g = 0; g < kTurn; ++g) tmem_ld_16x32(d.at + (static_cast<uint32_t>(16 * (t + g)) << 16), v[g]);
        if (t == 0) {
            load_pairs<WHOLE>(p.w_scale, d.n, p.N, ws);
            load_pairs<WHOLE>(p.bias, d.n, p.N, bias);
        }
#pragma unroll
        for (int g = 0; g < kTurn; ++g) tmem_ld_wait16(v[g]);
#pragma unroll
        for (int g = 0; g < kTurn; ++g) {
            finish_block<ACT>(v[g], d.xs[2 * (t + g)], d.xs[2 * (t + g) + 1], ws, bias);
            if (g == 0) {  // what went through the buffer before has been read
                if (TMA && lane == 0) bulk_wait_read_all();
                __syncwarp();
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) stage_row<BF16>(d.out + g * 1024, (lane >> 2) + 8 * h, lane & 3, v[g], h);
        }
        if constexpr (TMA) fence_proxy_async_smem();
        __syncwarp();
        if constexpr (TMA) {
            if (lane == 0) {
#pragma unroll
                for (int g = 0; g < kTurn; ++g)
                    if (d.block_m + 16 * (t + g) < p.M) tma_store_2d(d.map, d.out + g * 1024, d.block_n, d.block_m + 16 * (t + g));
                bulk_commit();
            }
        } else {
            constexpr int es = BF16 ? 2 : 4;
            const long long row_bytes = static_cast<long long>(p.N) * es;
#pragma unroll 1
            for (int g = 0; g < kTurn; ++g) {
                const int m = d.block_m + 16 * (t + g);
                uint8_t* y = static_cast<uint8_t*>(p.y) + m * row_bytes + static_cast<long long>(d.block_n) * es;
                const int rows = p.M - m, columns = p.N - d.block_n;
                if (row_bytes % 8 == 0) store_rows<BF16, uint2>(y, row_bytes, rows, columns, d.out + g * 1024);
                else if (row_bytes % 4 == 0) store_rows<BF16, uint32_t>(y, row_bytes, rows, columns, d.out + g * 1024);
                else if constexpr (BF16) store_rows<BF16, uint16_t>(y, row_bytes, rows, columns, d.out + g * 1024);
            }
        }
    }
}

// The sums of such a block to shared memory as they are (K split over a cluster): every operand tile
// of this CTA has been read by then.
template <int G>
__device__ __forceinline__ void leave_block(uint32_t at, float* part, int row_floats) {
    uint32_t v[G][16];
#pragma unroll
    for (int g = 0; g < G; ++g) tmem_ld_16x32(at + (static_cast<uint32_t>(16 * g) << 16), v[g]);
#pragma unroll
    for (int g = 0; g < G; ++g) tmem_ld_wait16(v[g]);
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const auto at8 = [&](int i) { return v[g][4 * (i >> 1) + 2 * h + (i & 1)]; };
            uint4* to = reinterpret_cast<uint4*>(part + (16 * g + 8 * h) * row_floats);
            to[0] = make_uint4(at8(0), at8(1), at8(2), at8(3));
            to[1] = make_uint4(at8(4), at8(5), at8(6), at8(7));
        }
}

__device__ __forceinline__ float4 peer_float4(const float* p, uint32_t cta) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(mapa_shared(smem_addr(p), cta))
                 : "memory");
    return v;
}

__device__ __forceinline__ float finish_one(const Int8Params& p, float sum, float xs, int n) {
    const float v = fmaf(sum * xs, __ldg(p.w_scale + n), p.bias ? __ldg(p.bias + n) : 0.0f);
    if (p.act == CONV_ACT_RELU) return activate<CONV_ACT_RELU>(v);
    if (p.act == CONV_ACT_SILU) return activate<CONV_ACT_SILU>(v);
    return v;
}

// This CTA's rows of the cluster's tile from the parts of all its CTAs, four columns a thread.
template <int BN>
__device__ __forceinline__ void join_parts(const Int8Params& p, const float* part, int m0, int n0, uint32_t cta, int splits) {
    constexpr int kRow = BN + 8, kQuads = BN / 4;
    const int rows = 128 / splits, first = static_cast<int>(cta) * rows;
    for (int i = threadIdx.x; i < rows * kQuads; i += kGemmThreads) {
        const int row = first + i / kQuads, q = i % kQuads, n = n0 + 4 * q;
        if (m0 + row >= p.M || n >= p.N) continue;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int k = 0; k < splits; ++k) {
            const float4 v = peer_float4(part + row * kRow + 4 * q, k);
            sum.x += v.x;
            sum.y += v.y;
            sum.z += v.z;
            sum.w += v.w;
        }
        const float xs = load1_late(p.x_scale + m0 + row);
        const float in[4] = {sum.x, sum.y, sum.z, sum.w};
        const long long o = static_cast<long long>(m0 + row) * p.N + n;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (n + j >= p.N) break;
            const float v = finish_one(p, in[j], xs, n + j);
            if (p.out_bf16) static_cast<__nv_bfloat16*>(p.y)[o + j] = __float2bfloat16_rn(v);
            else static_cast<float*>(p.y)[o + j] = v;
        }
    }
}

// The columns of a warp: `whole` of its blocks of 32 read scales in wide accesses.
template <int ACT, bool BF16, bool TMA, int G>
__device__ __forceinline__ void drain_columns(const Int8Params& p, Drain d, int blocks, int whole) {
    const auto next = [&] {
        d.at += 32;
        d.n += 32;
        d.block_n += 32;
    };
    int i = 0;
#pragma unroll 1
    for (; i < whole; ++i, next()) drain_block<ACT, BF16, true, TMA, G>(p, d);
#pragma unroll 1
    for (; i < blocks; ++i, next()) drain_block<ACT, BF16, false, TMA, G>(p, d);
}

template <bool BF16, bool TMA, int G>
__device__ __forceinline__ void drain_act(const Int8Params& p, const Drain& d, int blocks, int whole) {
    if (p.act == CONV_ACT_RELU) drain_columns<CONV_ACT_RELU, BF16, TMA, G>(p, d, blocks, whole);
    else if (p.act == CONV_ACT_SILU) drain_columns<CONV_ACT_SILU, BF16, TMA, G>(p, d, blocks, whole);
    else drain_columns<CONV_ACT_NONE, BF16, TMA, G>(p, d, blocks, whole);
}

// Whether every row of y starts on 16 bytes (y itself does).
__host__ __device__ inline bool rows_on_16(const Int8Params& p) { return p.N % (p.out_bf16 ? 8 : 4) == 0; }

__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {  // as idesc_bf16_f32 with FP16 operands (type 0)
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

template <bool PAIR, int BN>
__global__ void __launch_bounds__(kGemmThreads, 1)
    int8_gemm_kernel(const Int8Params p, const __grid_constant__ CUtensorMap map_x,
                     const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_y) {
    using S = Shape<PAIR, BN>;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_addr(smem) & 1023u) {  // the swizzle's atoms; uniform, so no CTA waits for another
        record_status(p.status, kStatusTimeoutMma, nullptr);
        return;
    }
    Bars b;
    uint8_t* raw = smem + S::kStages * S::kStage;
    uint8_t* outputs = raw + S::kRawSlots * S::kRaw;
    b.rfull = reinterpret_cast<uint64_t*>(outputs + kEpilogueWarps * S::kOut);
    b.rempty = b.rfull + S::kRawSlots;
    b.full = b.rempty + S::kRawSlots;
    b.empty = b.full + S::kStages;
    b.tfull = b.empty + S::kStages;
    b.tempty = b.tfull + 2;
    b.drain = b.tempty + 2;
    b.tmem_slot = reinterpret_cast<uint32_t*>(b.drain + 1);
    b.abort = reinterpret_cast<int*>(b.tmem_slot + 1);
    volatile int* abort = b.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t cta = cluster_ctarank();  // 0 without a cluster
    const uint32_t rank = PAIR ? cta : 0u;
    const bool leader = rank == 0;
    constexpr int kCtas = PAIR ? 2 : 1;
    const int splits = PAIR ? 1 : p.splits;

    Tiles tiles;
    tiles.n_tiles = (p.N + BN - 1) / BN;
    tiles.units = ((p.M + 128 * kCtas - 1) / (128 * kCtas)) * tiles.n_tiles;
    tiles.step = static_cast<int>(gridDim.x) / kCtas;
    tiles.step_m = tiles.step / tiles.n_tiles;
    tiles.step_n = tiles.step - tiles.step_m * tiles.n_tiles;
    tiles.rank = rank;
    int unit0 = static_cast<int>(blockIdx.x) / kCtas;
    const int units = tiles.units;
    int kfirst = 0, ksteps = (p.K + kStepK - 1) / kStepK;
    if (splits > 1) {  // one tile a cluster
        unit0 = static_cast<int>(blockIdx.x) / splits;
        tiles.step = units;
        const int all = ksteps;
        kfirst = static_cast<int>(cta) * all / splits;
        ksteps = (static_cast<int>(cta) + 1) * all / splits - kfirst;
    }
    tiles.k_begin = kfirst * kStepK;
    tiles.k_end = min(p.K, (kfirst + ksteps) * kStepK);

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
    asm volatile("griddepcontrol.wait;" ::: "memory");  // x, w or x's scales from the kernel before this one

    if (warp < kConverterWarps) {
        // ------------------------------------------------------------ converters
        const int group = warp / kGroupWarps;  // converts steps group, group + kGroups, ... into stage `group`
        const int t = threadIdx.x & (32 * kGroupWarps - 1);
        const int c = t & 3, r0 = t >> 2;
        Walk w = walk_from<PAIR, BN>(tiles, unit0);
        advance<PAIR, BN>(tiles, w, group);
        if (w.u < units) {
            uint32_t ph = 0;
            uint8_t* stage = smem + group * S::kStage;
            int rs = group;
            uint32_t rph = 0;
            while (w.u < units) {
                if (!warp_wait(&b.rfull[rs], rph, abort)) {
                    record_status(p.status, kStatusTimeoutTransform, abort);
                    break;
                }
                const uint4* src = reinterpret_cast<const uint4*>(raw + rs * S::kRaw) + t;
                uint4 x[8], wt[S::kItemsB];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = src[i * 64];  // rows r0 + 16 i of x, then of w
                if (!warp_wait(&b.empty[group], ph ^ 1u, abort)) {
                    record_status(p.status, kStatusTimeoutTransform, abort);
                    break;
                }
                store_items<8, false>(p.M - w.m0, r0, c, x, stage);
#pragma unroll
                for (int i = 0; i < S::kItemsB; ++i) wt[i] = src[(8 + i) * 64];
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.rempty[rs]);
                store_items<S::kItemsB, true>(p.N - w.n0, r0, c, wt, stage + S::kTileA);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR) arrive_leader(&b.full[group]);
                    else mbar_arrive(&b.full[group]);
                }
                ph ^= 1u;
                if ((rs += kGroups) >= S::kRawSlots) {  // at least as many slots as groups: one wrap a turn at most
                    rs -= S::kRawSlots;
                    rph ^= 1u;
                }
                advance<PAIR, BN>(tiles, w, kGroups);
            }
        }
    } else if (warp < kMmaWarp) {
        // ------------------------------------------------------------ epilogue
        const int quarter = warp & 3;
        const int part = (warp - kConverterWarps) >> 2;
        const bool wide = rows_on_16(p);
        int local = 0;
        // A warp drains a quarter of the columns of 32 rows; of 64 columns half, of 32 all (two of the four
        // warps), 16 rows.
        constexpr int kCols = BN >= 128 ? BN / 4 : 32;
        const int col0 = BN >= 128 ? part * kCols : (BN == 64 ? (part & 1) * 32 : 0);
        constexpr int G = BN >= 128 ? 2 : 1;
        const int lane0 = quarter * 32 + (BN >= 128 ? 0 : 16 * (BN == 64 ? part >> 1 : part & 1));  // its first row of the tile
        const bool idle = BN == 32 && part >= 2;
        for (Walk w = walk_from<PAIR, BN>(tiles, unit0); w.u < units; next_unit(tiles, w), ++local) {
            const int buf = local & 1;
            const uint32_t use = static_cast<uint32_t>(local >> 1) & 1u;
            const long long row0 = static_cast<long long>(w.mu) * 128 * kCtas + rank * 128 + lane0 + (lane >> 2);
            const int first = w.nt * BN + col0, left = idle ? 0 : p.N - first;
            Drain d;
            d.at = tmem + (static_cast<uint32_t>(lane0) << 16) + buf * BN + col0;
            d.n = first + (lane & 3) * 8;
            d.map = &map_y;
            d.out = outputs + (warp - kConverterWarps) * S::kOut;
            d.block_n = first;
            d.block_m = static_cast<int>(row0) - (lane >> 2);
#pragma unroll
            for (int i = 0; i < 2 * G; ++i) d.xs[i] = row0 + 8 * i < p.M ? load1_late(p.x_scale + row0 + 8 * i) : 0.0f;
            const int blocks = left <= 0 ? 0 : (left >= kCols ? kCols / 32 : (left + 31) / 32);
            const int whole = left <= 0 ? 0 : (left >= kCols ? kCols / 32 : left / 32);
            if (!warp_wait_cluster(&b.tfull[buf], use, abort)) {
                record_status(p.status, kStatusTimeoutEpilogue, abort);
                break;
            }
            tc_fence_after();
            if (splits > 1 && !idle) {
                float* part = reinterpret_cast<float*>(smem) + static_cast<size_t>(lane0 + (lane >> 2)) * S::kPartRow + (lane & 3) * 8;
                for (int c = col0; c < col0 + kCols; c += 32)
                    leave_block<G>(d.at + (c - col0), part + c, S::kPartRow);
            } else if (p.out_bf16 && wide) {
                drain_act<true, true, G>(p, d, blocks, whole);
            } else if (p.out_bf16) {
                drain_act<true, false, G>(p, d, blocks, whole);
            } else if (wide) {
                drain_act<false, true, G>(p, d, blocks, whole);
            } else {
                drain_act<false, false, G>(p, d, blocks, whole);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR) arrive_leader(&b.tempty[buf]);
                else mbar_arrive(&b.tempty[buf]);
            }
        }
        if (lane == 0) bulk_wait_all();  // none in flight when the CTA leaves
    } else if (warp == kLoadWarp) {
        // ------------------------------------------------------------ raw ring
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
                advance<PAIR, BN>(tiles, w, 1);
            }
            for (int s = 0; s < S::kRawSlots; ++s) {  // no copy in flight when the CTA leaves
                const long long fills = issued / S::kRawSlots + (s < issued % S::kRawSlots ? 1 : 0);
                if (fills && !mbar_wait(&b.rfull[s], static_cast<uint32_t>((fills - 1) & 1), nullptr))
                    record_status(p.status, kStatusTimeoutDrain, abort);
            }
        }
    } else if (lane == 0 && leader) {
        // ------------------------------------------------------------ MMA
        constexpr uint32_t idesc = idesc_f16_f32(128 * kCtas, BN);
        int st = 0, local = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int u = unit0; u < units && ok; u += tiles.step, ++local) {
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
                const int left = (p.K - (kfirst + ks) * kStepK + 15) >> 4;
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
    if (!PAIR && splits > 1) {
        cluster_sync_all();  // every part is in place
        const Walk w = walk_from<PAIR, BN>(tiles, unit0);
        join_parts<BN>(p, reinterpret_cast<const float*>(smem), w.m0, w.n0, cta, splits);
        __syncwarp();  // the aligned barrier takes a warp's lanes together
        cluster_sync_all();  // no CTA leaves while another may still read its part
    }
    if (warp == kMmaWarp) {
        __syncwarp();
        tc_fence_after();
        if constexpr (PAIR) tmem_dealloc_pair(tmem, S::kTmemCols);
        else tmem_dealloc(tmem, S::kTmemCols);
    }
}

// [rows][K] 8-bit matrix, rows `pitch` bytes apart, in boxes of `box_rows` rows x 64 bytes.
bool encode_rows(CUtensorMap* map, const int8_t* base, int rows, int K, int pitch, int box_rows) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
    const cuuint32_t box[2] = {kStepK, static_cast<cuuint32_t>(box_rows)};
    return tensor_map_encoder_ready() &&
           encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(base), dims, strides, box,
                        CU_TENSOR_MAP_SWIZZLE_NONE) == CUDA_SUCCESS;
}

template <bool PAIR, int BN>
cudaError_t launch_variant(const Int8Params& p, int num_sms, bool after_layout, cudaStream_t stream) {
    using S = Shape<PAIR, BN>;
    static SmemLimitCache limits;
    auto* fn = int8_gemm_kernel<PAIR, BN>;
    const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(fn), S::kSmem, limits);
    if (e != cudaSuccess) return e;
    constexpr int ctas = PAIR ? 2 : 1;
    const long long units = (static_cast<long long>(p.M) + 128 * ctas - 1) / (128 * ctas) * ((p.N + BN - 1) / BN);
    const int slots = num_sms / ctas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.splits > 1 ? static_cast<unsigned>(units * p.splits)
                                    : static_cast<unsigned>((units < slots ? units : slots) * ctas));
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (PAIR || p.splits > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = PAIR ? 2 : p.splits;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (after_layout) {  // its set-up overlaps the kernel before it
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    CUtensorMap map_x, map_w, map_y;
    if (rows_on_16(p)) {
        const cuuint64_t dims[2] = {static_cast<cuuint64_t>(p.N), static_cast<cuuint64_t>(p.M)};
        const cuuint64_t strides[1] = {static_cast<cuuint64_t>(p.N) * (p.out_bf16 ? 2 : 4)};
        const cuuint32_t box[2] = {32, 16};
        if (!tensor_map_encoder_ready() ||
            encode_tiled(&map_y, p.out_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, p.y, dims,
                         strides, box, p.out_bf16 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    } else {
        map_y = CUtensorMap();
    }
    if (!encode_rows(&map_x, p.x, p.M, p.K, p.x_pitch, 128) || !encode_rows(&map_w, p.w, p.N, p.K, p.w_pitch, S::kRowsB))
        return cudaErrorInvalidValue;
    return cudaLaunchKernelEx(&cfg, fn, p, map_x, map_w, map_y);
}

// Rows of K bytes to rows `pitch` apart (pitch a multiple of 16, at least K), 16 bytes a thread; the
// bytes that only pad are 0.
__global__ void __launch_bounds__(256) int8_layout_kernel(const int8_t* x, int8_t* xr, long long x_rows, const int8_t* w, int8_t* wr,
                                                          long long w_rows, int K, int pitch) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int chunks = pitch >> 4;
    const long long x_items = x_rows * chunks, items = x_items + w_rows * chunks;
    for (long long i = blockIdx.x * 256LL + threadIdx.x; i < items; i += gridDim.x * 256LL) {
        const bool is_x = i < x_items;
        const long long at = is_x ? i : i - x_items;
        const long long row = items >> 32 ? at / chunks : static_cast<uint32_t>(at) / static_cast<uint32_t>(chunks);
        const int k = static_cast<int>(at - row * chunks) * 16;
        const int len = K - k < 16 ? K - k : 16;
        const uint4 v = load_item(is_x ? x : w, row * K + k, len, (is_x ? x_rows : w_rows) * K);
        *reinterpret_cast<uint4*>((is_x ? xr : wr) + row * pitch + k) = v;
    }
}

}  // namespace

bool int8_gemm_fits(const Int8Params& p) {  // tile counts and row indexes in 32 bits
    return (static_cast<long long>(p.M) + 127) / 128 * ((p.N + 31) / 32) < (1LL << 30) && p.M < (1 << 30) && p.N < (1 << 30);
}

cudaError_t launch_int8_layout(const int8_t* x, int8_t* xr, long long x_rows, const int8_t* w, int8_t* wr, long long w_rows,
                               int K, int pitch, int num_sms, cudaStream_t stream) {
    const long long blocks = ((x_rows + w_rows) * (pitch / 16) + 255) / 256;
    int8_layout_kernel<<<static_cast<unsigned>(blocks < 8LL * num_sms ? blocks : 8LL * num_sms), 256, 0, stream>>>(
        x, xr, x_rows, w, wr, w_rows, K, pitch);
    return cudaGetLastError();
}

namespace {

// Tile shapes and what they cost, in microseconds on a 152-SM part at ~1.9 GHz (repeated launches
// in a graph, 8-bit input, whole rounds of tiles): a K = 64 step and what a tile takes besides, the
// least it takes (its epilogue), both again where rows of y start off 16 bytes, the launch, and what
// joining the parts adds where a cluster splits K.  From K = 64 / 256 / 1024, BF16 output:
// 1.1 / 2.0 / 6.9 us a tile of 32 columns, 1.3 / 2.2 / 7.3 of 64, 1.8 / 2.8 / 8.2 of 128, 3.1 / 3.8 / 8.8 on a pair.
// 65 x 4096 -> 4096 (64 steps): 29.2 us as 128 tiles of 32 columns, 20.5 as 64 tiles of 64 split
// in two, 15.7 as 32 tiles of 128 split in four; 256 rows 31.6 as 128 tiles of 64, 23.4 as 64 of 128
// split in two; 1000 rows 62 in tiles of 128 x 128 and 35 on pairs.
struct Tile {
    int rows, columns;
    double step, besides, least, off_besides, off_least, launch, join;
};
constexpr Tile kTiles[4] = {{128, 32, 0.415, 0.25, 1.15, 0.40, 1.45, 4.4, 1.9},
                            {128, 64, 0.42, 0.45, 1.35, 0.70, 1.80, 4.7, 2.4},
                            {128, 128, 0.46, 0.90, 1.85, 1.8, 3.0, 5.0, 3.8},
                            {256, 256, 0.45, 1.60, 3.05, 3.0, 5.5, 5.8, 0.0}};

// Clusters of this kernel's CTAs (one an SM) that the part holds at a time, by CTAs in a cluster: a
// 152-SM part holds 76 of 2, 36 of 4 and 15 of 8.
int clusters_at_a_time(int num_sms, int ctas) {
    return ctas == 1 ? num_sms : (ctas == 2 ? num_sms / 2 : (ctas == 4 ? num_sms * 36 / 152 : num_sms * 15 / 152));
}

}  // namespace

// The tile shape and split of K that cost least by those figures.
Int8Tile int8_pick_tile(const Int8Params& p, int num_sms) {
    const long long steps = (p.K + kStepK - 1) / kStepK;
    const bool on_16 = rows_on_16(p);
    double best = 0.0;
    Int8Tile pick = {};
    for (int i = 0; i < 4; ++i) {
        const Tile& t = kTiles[i];
        const long long units = (static_cast<long long>(p.M) + t.rows - 1) / t.rows * ((p.N + t.columns - 1) / t.columns);
        for (int splits = 1; splits <= (i < 3 ? 8 : 1); splits *= 2) {
            const long long at_a_time = clusters_at_a_time(num_sms, i == 3 ? 2 : splits);
            if (splits > 1 && (units > at_a_time || steps < 2 * splits)) break;
            const double each = static_cast<double>((steps + splits - 1) / splits) * t.step + (on_16 ? t.besides : t.off_besides);
            const double least = on_16 ? t.least : t.off_least;
            const double cost = t.launch + static_cast<double>((units + at_a_time - 1) / at_a_time) * (each > least ? each : least) +
                                (splits > 1 ? t.join : 0.0);
            if (pick.rows == 0 || cost < best) {
                best = cost;
                pick = {t.rows, t.columns, splits};
            }
        }
    }
    return pick;
}

cudaError_t launch_int8_gemm(const Int8Params& given, int num_sms, bool after_layout, cudaStream_t stream) {
    Int8Params p = given;
    const Int8Tile tile = int8_pick_tile(p, num_sms);
    p.splits = tile.splits;
    if (tile.columns == 256) return launch_variant<true, 256>(p, num_sms, after_layout, stream);
    if (tile.columns == 128) return launch_variant<false, 128>(p, num_sms, after_layout, stream);
    if (tile.columns == 64) return launch_variant<false, 64>(p, num_sms, after_layout, stream);
    return launch_variant<false, 32>(p, num_sms, after_layout, stream);
}

}  // namespace convgb
