// linear_gemm.cu -- the linear layer's products on tcgen05 tensor cores:
//
//   y[m][n] = act( sum_k a(m, k) * b(n, k) + bias[n] ) + r[m][n]
//
// One kernel for the forward product (both operands by row: K-major) and the two gradients, whose
// operands lie the other way round: dx = u w reads w, and dw = u^T x both operands, as rows along K
// (MN-major: the TMA brings 64 x 64 boxes, whose 128-byte rows run along m or n).  Both gradients go in one launch:
// their tiles fill the SMs' rounds together.
//
// Warp roles (one CTA per SM, persistent over units; a unit is a tile, or a part of its K):
//   the first 8 or 16   epilogue: a warp drains 32 rows of tensor memory, 64 columns at a time; in two groups that
//                       take the units in turn where a CTA has several, so that one's residuals and sums arrive
//                       while the other works
//   next                tensor memory; the whole warp walks the stages and one elected lane issues tcgen05.mma
//                       and commits.  (A loop of one lane only, its operands in the registers of a divergent
//                       thread, took 95 clocks an MMA and 700 a stage of 512 clocks of MMAs: 19456 x 4096 x 4096
//                       376 us, and 328 as it is, 1,988 TFLOP/s.)
//   last                fills the ring of (A, B) stages, K = 64 or 128 each, by TMA
// Tensor memory holds two accumulators, so the epilogue of one unit overlaps the next one's MMAs.
//
// PAIR: two SMs share a 256 x 256 tile (tcgen05.mma.cta_group::2): each loads its own 128 rows of A and
// 128 of B.
//
// The epilogue keeps the sum in FP32 to the end.  The residual comes by TMA into the warp's output
// buffer while the MMAs run; every thread adds its row's part and writes the result in the same
// place, from where the TMA stores it (so y may be the residual).  Rows of y off 16 bytes (N % 8) are
// beyond the TMA: they move between buffer and memory as the aligned granules that they lie in.
//
// Measured (repeated launches in a graph): 8192 x 4096 x 4096 142 us, 1,933 TFLOP/s, the rate of the card's library product;
// bound by the tensor cores (89 % of their cycles) and, in long streams of calls, by power.  200704 x 256 -> 512 with bias,
// ReLU and a residual 84 us, 6.1 TB/s; bound by memory.  dx and dw of 8192 x 1024 -> 4096 80 us, 1,720 TFLOP/s.
//
// Few tiles: the K of each is shared by `splits` units.  Of the forward product two, four or eight of them are a cluster:
// each leaves its FP32 sums in its shared memory, and after a cluster barrier each finishes its share of the rows from
// all of them, added in one order.  Otherwise they leave parts in the workspace, and a kernel of its own adds and finishes them.
#include "int8_rows.cuh"
#include "linear_internal.h"
#include "pointwise_math.cuh"
#include "ptx.cuh"
#include "row_sums.cuh"

namespace convgb {

namespace {

constexpr int kBlockCols = 64, kBlockBytes = 32 * 128;  // 32 rows x 64 columns of outputs
constexpr int kEdgeBytes = 5 * 1024;                       // room for them where rows start off 16 bytes
constexpr int kStepK = 64;       // K of a step: 128 bytes of a row
constexpr int kTileA = 128 * 128;  // bytes of A in a stage: 128 rows

// What a launch fixes besides the operands.
struct Ring {
    int stages;  // of operands
    int warps;   // of the epilogue that work
    int groups;  // of them: 1, or 2 that take the units in turn
    int cluster;  // CTAs that share the K of a tile and join it themselves; 1: none
};

constexpr int kBox = 64 * 128;   // bytes of an MN-major box: 64 of K, 64 of m or n

template <bool PAIR, int BN, bool TMA>
struct Shape {
    static constexpr int kCtas = PAIR ? 2 : 1;
    static constexpr int kRowsB = BN / kCtas;            // of B in this CTA
    static constexpr int kStage = kTileA + kRowsB * 128;  // of K = 64
    // Such stages that share a barrier: a turn of the MMA warp costs 300 clocks besides its MMAs, which those of K = 64 hide on a
    // pair (512 clocks) and not in smaller tiles (a step of K = 64 0.24 us there, 0.15 with two to a turn); where only two
    // turns would fit, one.
    static constexpr int kSteps = !PAIR && (BN == 64 || TMA) ? 2 : 1;
    static constexpr int kEpilogueWarps = BN == 256 ? 16 : 8;
    static constexpr int kThreads = 32 * (kEpilogueWarps + 2);
    static constexpr int kTmemCols = 2 * BN;
    // Each epilogue warp that works has room for a block of outputs; the ring takes the rest.
    static constexpr int kBarBytes = 512 + kEpilogueWarps * 128;  // barriers, the warps' biases
    static constexpr int kOut = TMA ? kBlockBytes : kEdgeBytes;
    static constexpr int stages(int warps) { return (232448 - kBarBytes - warps * kOut) / (kSteps * kStage); }
    static constexpr int kMaxStages = stages(8);
    static_assert((2 * kMaxStages + 5 + kEpilogueWarps) * 8 + 8 <= 512, "barriers");
};

struct Bars {
    uint64_t* full;
    uint64_t* empty;
    uint64_t* tfull;
    uint64_t* tempty;
    uint64_t* drain;
    uint64_t* res;  // one for each epilogue warp
    float* bias;    // 32 values for each of them
    uint32_t* tmem_slot;
    int* abort;
};

// Arrive on the pair leader's barrier; tensor memory's contents are ordered by tcgen05's own fences.
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(mapa_shared(smem_addr(bar), 0)) : "memory");
}

// A bounded wait whose answer is the same in every lane.  (The first look by itself: the loop behind it is rarely entered.)
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    if (__all_sync(0xffffffffu, mbar_try_wait(smem_addr(bar), parity))) return true;
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}
__device__ __forceinline__ bool warp_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort) {
    if (__all_sync(0xffffffffu, mbar_try_wait_cluster(smem_addr(bar), parity))) return true;
    return __all_sync(0xffffffffu, mbar_wait_cluster(bar, parity, abort));
}

// The same one lane of a converged warp at every call: MMAs and their commits are one thread's.
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t* bar) {
    if constexpr (PAIR) mma_commit_pair(bar, 3);
    else mma_commit(bar);
}

// What a unit is: its tile, in order of groups of kGroupM tile rows (neighbouring units share rows of A and
// columns of B, which then come from L2), and its steps of K.
constexpr int kGroupM = 8;

// One product of a launch.
struct Job {
    CUtensorMap map_a, map_b, map_y, map_z, map_r, map_part;
    int M, N, K, splits;
    int m_tiles, n_tiles, tiles, ksteps;
    int first;  // its first unit
    int a_by_k, act;
    const float* bias;
    const __nv_bfloat16* r;
    __nv_bfloat16* y;
    __nv_bfloat16* z;
};

struct Launch {
    Job job[2];
    int jobs, units;
    Ring ring;
    ColumnJoin join;
    unsigned* status;
};

struct Unit {
    int mt, nt, split, k_first, k_count;
};

// The forward product comes alone, the gradients (SEVERAL) in twos.
template <bool SEVERAL>
__device__ __forceinline__ const Job& job_of(const Launch& L, int u) {
    if constexpr (!SEVERAL) return L.job[0];
    return L.job[L.jobs > 1 && u >= L.job[1].first ? 1 : 0];
}

template <bool SEVERAL>
__device__ __forceinline__ Unit unit_at(const Job& t, int u) {
    Unit w;
    if constexpr (SEVERAL) u -= t.first;
    w.split = u / t.tiles;
    const int i = u - w.split * t.tiles;
    const int per_group = kGroupM * t.n_tiles, g = i / per_group, rest = i - g * per_group;
    const int rows = min(kGroupM, t.m_tiles - g * kGroupM);
    w.nt = rest / rows;
    w.mt = g * kGroupM + rest - w.nt * rows;
    w.k_first = static_cast<int>(static_cast<long long>(w.split) * t.ksteps / t.splits);
    w.k_count = static_cast<int>(static_cast<long long>(w.split + 1) * t.ksteps / t.splits) - w.k_first;
    return w;
}

// Shared-memory descriptor of an MN-major operand: boxes of 64 (K) rows of 128 bytes in the 128-byte swizzle,
// 8 rows of K 1,024 bytes apart (stride offset), the next 64 of m or n a box further (leading offset).
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(kBox >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}

// ROWS rows of an operand from row `row`, K = 64 from k, to a stage.
template <bool PAIR, int ROWS>
__device__ __forceinline__ void load_operand(bool by_k, uint8_t* dst, const CUtensorMap* map, uint64_t* bar, uint32_t bar_leader, int row, int k) {
    if (by_k) {
#pragma unroll
        for (int i = 0; i < ROWS / 64; ++i) {
            if constexpr (PAIR) tma_load_2d_pair(dst + i * kBox, map, bar_leader, row + 64 * i, k);
            else tma_load_2d(dst + i * kBox, map, bar, row + 64 * i, k);
        }
    } else {
        if constexpr (PAIR) tma_load_2d_pair(dst, map, bar_leader, k, row);
        else tma_load_2d(dst, map, bar, k, row);
    }
}

// K = 16 j .. 16 j + 15 of a stage: 2,048 bytes, or 32, further for each.
__device__ __forceinline__ uint64_t operand_desc(bool by_k, uint32_t base, int j) {
    return by_k ? sdesc_mn(base) + 128 * j : sdesc_sw128(base) + 2 * j;
}

// ---------------------------------------------------------------- epilogue of a block: 32 rows x 64 columns
// A thread has one row of it: 128 bytes, in the 128-byte swizzle that the TMA reads and writes.
__device__ __forceinline__ uint4* block_chunk(uint8_t* block, int row, int j) {
    return reinterpret_cast<uint4*>(block + row * 128 + ((j ^ (row & 7)) << 4));
}

// Eight columns of a row: act(v + bias) + r, each operation rounded by itself.  bias: the columns' in shared memory,
// the same for every lane.
template <int ACT>
__device__ __forceinline__ uint4 finish_chunk(const uint32_t* v, const float4* bias, const uint4* r) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[i]);
    if (bias != nullptr) {
        const float4 lo = bias[0], hi = bias[1];
        const float add[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __fadd_rn(f[i], add[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = activate<ACT>(f[i]);
    if (r != nullptr) {
        const uint4 q = *r;
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __fadd_rn(f[2 * i], __uint_as_float(u[i] << 16));
            f[2 * i + 1] = __fadd_rn(f[2 * i + 1], __uint_as_float(u[i] & 0xffff0000u));
        }
    }
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// Rows of y that start on 2 bytes only: a block's part of a row lies across 9 aligned granules of 16 bytes at most.  A row of
// the buffer holds them as they lie in memory (144 bytes from row to row: eight lanes' 16-byte accesses fall on 32 banks),
// so whole granules move in wide accesses of neighbouring lanes, nine loads of the residual under way a lane, and
// only the ends of a row go by elements.  (Two-byte accesses throughout: 40000 x 515 -> 777 with a residual 139 us.)
constexpr int kEdgePitch = 144, kGranules = 9;

__device__ __forceinline__ void edge_load(uint8_t* block, const __nv_bfloat16* r, int m, int n, int M, int N) {
    const int8_t* base = reinterpret_cast<const int8_t*>(r);
    const long long total = static_cast<long long>(M) * N * 2;
    const int lane = threadIdx.x & 31, bytes = 2 * min(kBlockCols, N - n);
    uint4 v[kGranules];
#pragma unroll
    for (int i = 0; i < kGranules; ++i) {
        const int at = i * 32 + lane, row = at / kGranules, g = at - row * kGranules;
        const long long first = (static_cast<long long>(m + row) * N + n) * 2, from = (first & ~15LL) + 16 * g;
        v[i] = make_uint4(0, 0, 0, 0);
        if (m + row < M && from < first + bytes) v[i] = granule<true>(base, from >> 4, total);  // ordinary loads: y may be the residual
    }
#pragma unroll
    for (int i = 0; i < kGranules; ++i) {
        const int at = i * 32 + lane, row = at / kGranules, g = at - row * kGranules;
        *reinterpret_cast<uint4*>(block + row * kEdgePitch + 16 * g) = v[i];
    }
    __syncwarp();
}

// Byte of the block's part of a row in its first granule (32 bits do).
__device__ __forceinline__ int edge_offset(int row, int n, int N) {
    return static_cast<int>((static_cast<uint32_t>(row) * static_cast<uint32_t>(N) + static_cast<uint32_t>(n)) * 2u & 15u);
}

__device__ __forceinline__ void edge_store(const uint8_t* block, __nv_bfloat16* y, int m, int n, int M, int N) {
    uint8_t* first = reinterpret_cast<uint8_t*>(y) + (static_cast<long long>(m) * N + n) * 2;  // the block's first byte
    const long long pitch = 2LL * N;
    const int lane = threadIdx.x & 31, rows = min(32, M - m), bytes = 2 * min(kBlockCols, N - n);
    __syncwarp();
    // Whole granules: the (lane % 8)th of rows lane / 8, lane / 8 + 4, ...
    {
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = i * 4 + (lane >> 3), off = edge_offset(m + row, n, N), g = (lane & 7) + (off != 0);
            v[i] = *reinterpret_cast<const uint4*>(block + row * kEdgePitch + 16 * g);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = i * 4 + (lane >> 3), off = edge_offset(m + row, n, N), at = 16 * ((lane & 7) + (off != 0)) - off;
            if (row < rows && at + 16 <= bytes) *reinterpret_cast<uint4*>(first + row * pitch + at) = v[i];
        }
    }
    if (bytes == 2 * kBlockCols) {  // eight elements of a row, or none, lie before the first of them and behind the last
        uint16_t v[8];
        int at[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = i * 4 + (lane >> 3), off = edge_offset(m + row, n, N), k = lane & 7;
            at[i] = off == 0 || row >= rows ? -1 : (2 * k < 16 - off ? 2 * k : 2 * k + 112);
            v[i] = *reinterpret_cast<const uint16_t*>(block + row * kEdgePitch + off + max(at[i], 0));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (at[i] >= 0) *reinterpret_cast<uint16_t*>(first + (i * 4 + (lane >> 3)) * pitch + at[i]) = v[i];
    } else {  // the last columns of y: up to seven before the first whole granule, up to seven behind the last
#pragma unroll 8
        for (int i = 0; i < 16; ++i) {
            const int row = i * 2 + (lane >> 4), off = edge_offset(m + row, n, N), k = lane & 7;
            const int inner = (16 - off) & 15, outer = bytes - ((bytes + off) & 15);
            const int at = (lane & 8 ? max(inner, outer) : 0) + 2 * k;
            if (row < rows && at < (lane & 8 ? bytes : min(inner, bytes)))
                *reinterpret_cast<uint16_t*>(first + row * pitch + at) = *reinterpret_cast<const uint16_t*>(block + row * kEdgePitch + off + at);
        }
    }
    __syncwarp();
}

// A lane's share of the bias of a block: columns lane and 32 + lane.
struct LaneBias {
    float* row;  // the warp's 32 values in shared memory; nullptr: no bias
    float v[2];
    __device__ __forceinline__ void load(const float* bias, int n, int N) {
        if (row == nullptr) return;
        const int c = n + static_cast<int>(threadIdx.x & 31);
        v[0] = c < N ? __ldg(bias + c) : 0.0f;
        v[1] = c + 32 < N ? __ldg(bias + c + 32) : 0.0f;
    }
};

// One pass over a block's sums: y (with the residual that lies in `block`), or z, takes its place there and goes out.
// The bias reaches the lanes through shared memory: read from global memory by every lane, 16 bytes at a time, it
// was what the epilogue waited for (200704 x 256 -> 512 with ReLU 73 us, 55 without a bias).
template <int ACT, bool TMA>
__device__ __forceinline__ void block_pass(const Job& p, const CUtensorMap* map, __nv_bfloat16* to, bool with_r, uint32_t at,
                                           uint8_t* block, const LaneBias& bias, int m, int n) {
    const int lane = threadIdx.x & 31;
    uint4* own = reinterpret_cast<uint4*>(block + lane * kEdgePitch);  // off 16 bytes: the row's granules
    const int off = TMA ? 0 : edge_offset(m + lane, n, p.N);
    uint4 r = make_uint4(0, 0, 0, 0), before = r;
    if (!TMA && with_r) r = own[0];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t v[32];
        tmem_ld32(at + 32 * half, v);
        if (bias.row != nullptr) {
            __syncwarp();  // every lane has read what was there
            bias.row[lane] = bias.v[half];
            __syncwarp();
        }
        tmem_ld_wait(v);
        const float4* row = reinterpret_cast<const float4*>(bias.row);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4* b = row != nullptr ? row + 2 * j : nullptr;
            if constexpr (TMA) {
                uint4* chunk = block_chunk(block, lane, 4 * half + j);
                *chunk = finish_chunk<ACT>(v + 8 * j, b, with_r ? chunk : nullptr);
            } else {  // eight columns lie across two granules, for the residual and for what takes its place
                const int g = 4 * half + j;
                uint4 add = r;
                if (with_r) {
                    r = own[g + 1];
                    add = shift_granules(add, r, off);
                }
                const uint4 now = finish_chunk<ACT>(v + 8 * j, b, with_r ? &add : nullptr);
                own[g] = off == 0 ? now : shift_granules(before, now, 16 - off);
                before = now;
            }
        }
    }
    if constexpr (TMA) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_2d(map, block, n, m);
            bulk_commit();
        }
    } else {
        if (off != 0) own[kGranules - 1] = shift_granules(before, make_uint4(0, 0, 0, 0), 16 - off);
        edge_store(block, to, m, n, p.M, p.N);
    }
}

// PLAIN: y is the sums, rounded.
template <bool TMA, bool PLAIN>
__device__ __forceinline__ void finish_block(const Job& p, uint32_t at,
                                             uint8_t* block, const LaneBias& bias, int m, int n) {
    if constexpr (PLAIN) {
        block_pass<CONV_ACT_NONE, TMA>(p, &p.map_y, p.y, false, at, block, LaneBias(), m, n);
        return;
    }
    const bool with_r = p.r != nullptr;
    if (p.act == CONV_ACT_RELU) block_pass<CONV_ACT_RELU, TMA>(p, &p.map_y, p.y, with_r, at, block, bias, m, n);
    else if (p.act == CONV_ACT_SILU) block_pass<CONV_ACT_SILU, TMA>(p, &p.map_y, p.y, with_r, at, block, bias, m, n);
    else block_pass<CONV_ACT_NONE, TMA>(p, &p.map_y, p.y, with_r, at, block, bias, m, n);
    if (p.z != nullptr) {  // a second pass: tensor memory still has the sums
        if (TMA && (threadIdx.x & 31) == 0) bulk_wait_read_all();
        __syncwarp();
        block_pass<CONV_ACT_NONE, TMA>(p, &p.map_z, p.z, false, at, block, bias, m, n);
    }
}

// The sums of a block as they are to the workspace, half a block at a time: 128-byte rows in the 128-byte swizzle.
__device__ __forceinline__ void leave_block(const CUtensorMap* map, uint32_t at, uint8_t* buffer, int m, int n, int N, int split) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        if (n + 32 * half >= N) break;
        uint32_t v[32];
        tmem_ld32(at + 32 * half, v);
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
        tmem_ld_wait(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) *block_chunk(buffer, lane, j) = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_3d(map, buffer, n + 32 * half, m, split);
            bulk_commit();
        }
    }
}

// Four neighbouring outputs from their whole sums.
template <typename P>
__device__ __forceinline__ void finish_four(const P& p, const float4& s, long long m, int n) {
    float z[4] = {s.x, s.y, s.z, s.w}, y[4];
    const long long o = m * p.N + n;
    const int count = min(4, p.N - n);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (p.bias != nullptr && j < count) z[j] = __fadd_rn(z[j], __ldg(p.bias + n + j));
        y[j] = p.act == CONV_ACT_RELU ? activate<CONV_ACT_RELU>(z[j]) : (p.act == CONV_ACT_SILU ? activate<CONV_ACT_SILU>(z[j]) : z[j]);
    }
    if (p.N % 4 == 0) {
        if (p.z != nullptr) *reinterpret_cast<uint2*>(p.z + o) = make_uint2(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]));
        if (p.r != nullptr) {  // ordinary loads: y may be the residual
            const uint2 r = *reinterpret_cast<const uint2*>(p.r + o);
            y[0] = __fadd_rn(y[0], __uint_as_float(r.x << 16));
            y[1] = __fadd_rn(y[1], __uint_as_float(r.x & 0xffff0000u));
            y[2] = __fadd_rn(y[2], __uint_as_float(r.y << 16));
            y[3] = __fadd_rn(y[3], __uint_as_float(r.y & 0xffff0000u));
        }
        *reinterpret_cast<uint2*>(p.y + o) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (j >= count) break;
        if (p.z != nullptr) p.z[o + j] = __float2bfloat16_rn(z[j]);
        p.y[o + j] = __float2bfloat16_rn(p.r != nullptr ? __fadd_rn(y[j], __bfloat162float(p.r[o + j])) : y[j]);
    }
}

// ---------------------------------------------------------------- a K shared by a cluster
// The sums of 32 rows x 64 columns to shared memory: rows BN + 4 floats apart (16-byte accesses of eight rows fall on 32 banks).
__device__ __forceinline__ void keep_block(uint32_t at, float* part, int pitch) {
    float* row = part + static_cast<int>(threadIdx.x & 31) * pitch;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t v[32];
        tmem_ld32(at + 32 * half, v);
        tmem_ld_wait(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) reinterpret_cast<uint4*>(row + 32 * half)[j] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
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

// This CTA's rows of the cluster's tile from the parts of all its CTAs, eight accesses of a thread in flight.
template <int BN, int SPLITS>
__device__ __forceinline__ void join_cluster(const Job& p, const float* part, int m0, int n0, uint32_t cta) {
    constexpr int kPitch = BN + 4, kQuads = BN / 4, kRows = 128 / SPLITS, kAtOnce = 8 / SPLITS;
    const int first = static_cast<int>(cta) * kRows, threads = static_cast<int>(blockDim.x);
    for (int i = threadIdx.x; i < kRows * kQuads; i += threads * kAtOnce) {
        float4 v[kAtOnce][SPLITS];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int q = min(i + j * threads, kRows * kQuads - 1);
#pragma unroll
            for (int k = 0; k < SPLITS; ++k) v[j][k] = peer_float4(part + (first + q / kQuads) * kPitch + q % kQuads * 4, k);
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int q = i + j * threads, m = m0 + first + q / kQuads, n = n0 + q % kQuads * 4;
            if (q >= kRows * kQuads || m >= p.M || n >= p.N) continue;
            float4 s = v[j][0];
#pragma unroll
            for (int k = 1; k < SPLITS; ++k) {
                s.x += v[j][k].x;
                s.y += v[j][k].y;
                s.z += v[j][k].z;
                s.w += v[j][k].w;
            }
            finish_four(p, s, m, n);
        }
    }
}

// Sums over rows that the kernel before left in parts, a warp to a column: lane i adds parts i, i + 32, ..., as
// launch_join_columns' warps do, and the lanes' sums meet in its order.
__device__ __forceinline__ void join_columns(const ColumnJoin& j, int first, int step) {
    const int lane = threadIdx.x & 31;
    for (int c = first; c < j.columns; c += step) {
        float total = sum_of_parts(j.part, lane, j.parts, j.columns, c);
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) total += __shfl_xor_sync(0xffffffffu, total, i);
        if (lane == 0) j.out[c] = total;
    }
}

// TMA: rows of y start on 16 bytes (of their own, lest the other path's registers spill this one's: 200704 x 256 -> 512 with
// a residual 94 us together, 84 apart).
template <bool PAIR, int BN, bool B_BY_K, bool TMA>
__global__ void __launch_bounds__(Shape<PAIR, BN, TMA>::kThreads, 1) linear_gemm_kernel(const __grid_constant__ Launch L) {
    using S = Shape<PAIR, BN, TMA>;
    constexpr int kMmaWarp = S::kEpilogueWarps, kLoadWarp = kMmaWarp + 1, kCtas = S::kCtas;
    const Ring ring = L.ring;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join of parts that may follow
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_addr(smem) & 1023u) {  // the swizzle's atoms; uniform, so no CTA waits for another
        record_status(L.status, kStatusTimeoutMma, nullptr);
        return;
    }
    Bars b;
    uint8_t* outputs = smem + ring.stages * S::kSteps * S::kStage;
    b.full = reinterpret_cast<uint64_t*>(outputs + ring.warps * S::kOut);
    b.empty = b.full + S::kMaxStages;
    b.tfull = b.empty + S::kMaxStages;
    b.tempty = b.tfull + 2;
    b.drain = b.tempty + 2;
    b.res = b.drain + 1;
    b.bias = reinterpret_cast<float*>(outputs + ring.warps * S::kOut + 512);
    b.tmem_slot = reinterpret_cast<uint32_t*>(b.res + S::kEpilogueWarps);
    b.abort = reinterpret_cast<int*>(b.tmem_slot + 1);
    volatile int* abort = b.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
    const bool leader = rank == 0;

    const int units = L.units;
    constexpr bool kClusters = !PAIR && !B_BY_K;
    const bool joins = kClusters && ring.cluster > 1;  // then a CTA has one unit: its part of the cluster's tile
    const uint32_t cta = joins ? cluster_ctarank() : 0u;
    const int unit0 = joins ? static_cast<int>(cta) * L.job[0].tiles + static_cast<int>(blockIdx.x) / ring.cluster : static_cast<int>(blockIdx.x) / kCtas;
    const int unit_step = joins ? units : static_cast<int>(gridDim.x) / kCtas;

    if (threadIdx.x == 0) {
        for (int s = 0; s < ring.stages; ++s) {
            mbar_init(&b.full[s], 1);
            mbar_init(&b.empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b.tfull[i], 1);
            mbar_init(&b.tempty[i], kCtas * ring.warps / ring.groups);
        }
        mbar_init(b.drain, 1);
        for (int i = 0; i < S::kEpilogueWarps; ++i) mbar_init(&b.res[i], 1);
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
    asm volatile("griddepcontrol.wait;" ::: "memory");  // operands from the kernel before this one

    if (warp < ring.warps) {
        // ------------------------------------------------------------ epilogue
        const int per_group = ring.warps / ring.groups, group = warp / per_group;
        const int quarter = warp & 3, cols = BN * 4 / per_group, part = (warp - group * per_group) >> 2;
        uint8_t* block = outputs + warp * S::kOut;
        uint64_t* res = b.res + warp;
        float* bias_row = b.bias + 32 * warp;
        if (B_BY_K && L.join.out != nullptr) join_columns(L.join, static_cast<int>(blockIdx.x) * ring.warps + warp, static_cast<int>(gridDim.x) * ring.warps);
        uint32_t res_phase = 0;
        int local = group;
        bool ok = true;
        for (int u = unit0 + group * unit_step; u < units && ok; u += ring.groups * unit_step, local += ring.groups) {
            const Job& p = job_of<B_BY_K>(L, u);
            const Unit w = unit_at<B_BY_K>(p, u);
            const bool by_tma = TMA && !B_BY_K && p.r != nullptr && p.splits == 1;
            const int buf = local & 1;
            const uint32_t use = static_cast<uint32_t>(local >> 1) & 1u;
            const int m = w.mt * 128 * kCtas + static_cast<int>(rank) * 128 + quarter * 32, n = w.nt * BN + part * cols;
            const int blocks = m >= p.M ? 0 : min(cols / kBlockCols, (p.N - n + kBlockCols - 1) / kBlockCols);  // 0 or less: none
            const auto fetch = [&](int i) {  // block i of the residual, once what was in the buffer has left
                if (lane == 0) {
                    bulk_wait_read_all();
                    mbar_arrive_expect_tx(res, kBlockBytes);
                    tma_load_2d(block, &p.map_r, res, n + kBlockCols * i, m);
                }
                __syncwarp();
            };
            LaneBias bias = {};
            if constexpr (!B_BY_K) {
                bias.row = p.bias != nullptr ? bias_row : nullptr;
                bias.load(p.bias, n, p.N);
            }
            if (by_tma && blocks > 0) fetch(0);
            const auto fetch_rows = [&](int i) {
                edge_load(block, p.r, m, n + kBlockCols * i, p.M, p.N);
            };
            const bool by_rows = !TMA && !B_BY_K && p.splits == 1 && p.r != nullptr;
            if (by_rows && blocks > 0) fetch_rows(0);
            if (!warp_wait_cluster(&b.tfull[buf], use, abort)) {
                record_status(L.status, kStatusTimeoutEpilogue, abort);
                ok = false;
            }
            tc_fence_after();
#pragma unroll 1
            for (int i = 0; i < blocks && (ok || i == 0); ++i) {
                if (by_tma) {  // the first also after a wait that gave up: no copy may be in flight when the CTA leaves
                    if (i > 0) fetch(i);
                    if (!warp_wait(res, res_phase, nullptr)) {
                        record_status(L.status, kStatusTimeoutEpilogue, abort);
                        ok = false;
                    }
                    res_phase ^= 1u;
                } else if (TMA ? p.splits == 1 : B_BY_K) {  // off 16 bytes too: the unit before may have left parts of the other product
                    if (lane == 0) bulk_wait_read_all();
                    __syncwarp();
                } else if (by_rows && i > 0 && ok) {
                    fetch_rows(i);
                }
                if (!ok) continue;
                if (!B_BY_K && i > 0) bias.load(p.bias, n + kBlockCols * i, p.N);
                const uint32_t at = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + buf * BN + part * cols + kBlockCols * i;
                if (joins) keep_block(at, reinterpret_cast<float*>(smem) + quarter * 32 * (BN + 4) + part * cols + kBlockCols * i, BN + 4);  // operands are done with
                else if (p.splits > 1) leave_block(&p.map_part, at, block, m, n + kBlockCols * i, p.N, w.split);
                else finish_block<TMA, B_BY_K>(p, at, block, bias, m, n + kBlockCols * i);
            }
            if (!ok) break;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR) arrive_leader(&b.tempty[buf]);
                else mbar_arrive(&b.tempty[buf]);
            }
        }
        if (lane == 0) bulk_wait_all();  // none in flight when the CTA leaves
    } else if (warp == kLoadWarp) {
        // ------------------------------------------------------------ operands
        long long issued = 0;
        const bool issuer = elect_one();
        int st = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int u = unit0; u < units && ok; u += unit_step) {
            const Job& p = job_of<B_BY_K>(L, u);
            const Unit w = unit_at<B_BY_K>(p, u);
            const int m = w.mt * 128 * kCtas + static_cast<int>(rank) * 128, n = w.nt * BN + static_cast<int>(rank) * S::kRowsB;
            const bool a_by_k = B_BY_K && p.a_by_k != 0;  // the forward product's operands both lie by row
            for (int ks = 0; ks < w.k_count; ks += S::kSteps) {
                if (!warp_wait(&b.empty[st], ph ^ 1u, abort)) {
                    record_status(L.status, kStatusTimeoutProducer, abort);
                    ok = false;
                    break;
                }
                if (issuer) {
                    const int steps = min(S::kSteps, w.k_count - ks);
                    if (leader) mbar_arrive_expect_tx(&b.full[st], kCtas * S::kStage * steps);
                    const uint32_t bar = PAIR ? mapa_shared(smem_addr(&b.full[st]), 0) : 0u;
#pragma unroll
                    for (int i = 0; i < S::kSteps; ++i) {
                        if (i >= steps) break;
                        uint8_t* dst = smem + (st * S::kSteps + i) * S::kStage;
                        const int k = (w.k_first + ks + i) * kStepK;  // past the matrix: zeros
                        load_operand<PAIR, 128>(a_by_k, dst, &p.map_a, &b.full[st], bar, m, k);
                        load_operand<PAIR, S::kRowsB>(B_BY_K, dst + kTileA, &p.map_b, &b.full[st], bar, n, k);
                    }
                }
                __syncwarp();
                ++issued;
                if (++st == ring.stages) {
                    st = 0;
                    ph ^= 1u;
                }
            }
        }
        if (lane == 0) {
            for (int s = 0; s < ring.stages; ++s) {  // no copy in flight when the CTA leaves
                const long long fills = issued / ring.stages + (s < issued % ring.stages ? 1 : 0);
                if (fills == 0) continue;
                const uint32_t par = static_cast<uint32_t>((fills - 1) & 1);
                // the peer of a pair sees the MMAs release each slot, which needs its copies landed
                if (!(leader ? mbar_wait(&b.full[s], par, nullptr) : mbar_wait(&b.empty[s], par, nullptr)))
                    record_status(L.status, kStatusTimeoutDrain, abort);
            }
        }
    } else if (warp == kMmaWarp && leader) {
        // ------------------------------------------------------------ MMA
        const uint32_t base0 = smem_addr(smem);
        const bool issuer = elect_one();
        int st = 0, local = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int u = unit0; u < units && ok; u += unit_step, ++local) {
            const Job& p = job_of<B_BY_K>(L, u);
            const Unit w = unit_at<B_BY_K>(p, u);
            const int buf = local & 1;
            const uint32_t use = static_cast<uint32_t>(local >> 1) & 1u;
            if (!warp_wait_cluster(&b.tempty[buf], use ^ 1u, abort)) {
                record_status(L.status, kStatusTimeoutMma, abort);
                break;
            }
            tc_fence_after();
            const bool a_by_k = B_BY_K && p.a_by_k != 0;
            const uint32_t idesc = idesc_bf16_f32(128 * kCtas, BN) | (a_by_k ? 1u << 15 : 0u) | (B_BY_K ? 1u << 16 : 0u);
            const int k16 = (p.K - w.k_first * kStepK + 15) >> 4;  // steps of K = 16 to the end of the matrix
            for (int ks = 0; ks < w.k_count; ks += S::kSteps) {
                if (!warp_wait_cluster(&b.full[st], ph, abort)) {
                    record_status(L.status, kStatusTimeoutMma, abort);
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t base = base0 + st * S::kSteps * S::kStage;
                if (issuer) {
                    const int mmas = min(4 * min(S::kSteps, w.k_count - ks), k16 - 4 * ks);
#pragma unroll
                    for (int j = 0; j < 4 * S::kSteps; ++j) {
                        if (j >= mmas) break;
                        const uint32_t at = base + j / 4 * S::kStage;
                        const uint64_t da = operand_desc(a_by_k, at, j % 4), db = operand_desc(B_BY_K, at + kTileA, j % 4);
                        const uint32_t acc = (ks | j) != 0 ? 1u : 0u;
                        if constexpr (PAIR) mma_bf16_pair(tmem + buf * BN, da, db, idesc, acc);
                        else mma_bf16(tmem + buf * BN, da, db, idesc, acc);
                    }
                    commit<PAIR>(&b.empty[st]);
                }
                __syncwarp();
                if (++st == ring.stages) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            if (!ok) break;
            if (issuer) commit<PAIR>(&b.tfull[buf]);
            __syncwarp();
        }
        if (elect_one()) {
            if constexpr (PAIR) mma_commit_pair(b.drain, 1);
            else mma_commit(b.drain);
            if (!mbar_wait_cluster(b.drain, 0, nullptr)) record_status(L.status, kStatusTimeoutDrain, abort);
        }
    }
    __syncwarp();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();  // no CTA leaves while its peer may still signal it
    if constexpr (kClusters) {
        if (joins) {
            cluster_sync_all();  // every part is in place
            const Job& p = L.job[0];
            const Unit w = unit_at<false>(p, unit0);
            const float* part = reinterpret_cast<const float*>(smem);
            if (ring.cluster == 2) join_cluster<BN, 2>(p, part, w.mt * 128, w.nt * BN, cta);
            else if (ring.cluster == 4) join_cluster<BN, 4>(p, part, w.mt * 128, w.nt * BN, cta);
            else join_cluster<BN, 8>(p, part, w.mt * 128, w.nt * BN, cta);
            __syncwarp();  // the aligned barrier takes a warp's lanes together
            cluster_sync_all();  // no CTA leaves while another may still read its part
        }
    }
    if (warp == kMmaWarp) {
        __syncwarp();
        tc_fence_after();
        if constexpr (PAIR) tmem_dealloc_pair(tmem, S::kTmemCols);
        else tmem_dealloc(tmem, S::kTmemCols);
    }
}

// ---------------------------------------------------------------- parts of K
// Four neighbouring outputs to L threads, which add the parts l, l + L, ... each; their sums meet in order, then comes the
// epilogue.  (One thread to them all: 64 parts of 83 x 48 outputs 21 us.)
constexpr int kJoinThreads = 256;

template <int L>
__global__ void __launch_bounds__(kJoinThreads) linear_join_kernel(const GemmParams p, int splits) {
    constexpr int kQuads = kJoinThreads / L;
    __shared__ float4 sums[L][kQuads];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int quads = (p.N + 3) / 4, l = threadIdx.x / kQuads, q = threadIdx.x % kQuads;
    const long long i = static_cast<long long>(blockIdx.x) * kQuads + q, m = i / quads, all = static_cast<long long>(p.M) * quads;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const auto add = [&](const float4& v) {
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    };
    if (i < all) {
        const float4* from = reinterpret_cast<const float4*>(p.part) + i;
#pragma unroll 4
        for (int k = l; k < splits; k += L) add(from[k * all]);
    }
    if constexpr (L > 1) {
        sums[l][q] = s;
        __syncthreads();
        if (l != 0) return;
#pragma unroll
        for (int k = 1; k < L; ++k) add(sums[k][q]);
    }
    if (i < all) finish_four(p, s, m, static_cast<int>(i - m * quads) * 4);
}

// ---------------------------------------------------------------- launches
constexpr int part_pitch(int N) { return (N + 3) / 4 * 4; }

// [rows][inner] BF16 matrix in boxes of box_rows x box_inner.
bool encode_matrix(CUtensorMap* map, const void* base, long long rows, long long inner, long long pitch, int box_rows, int box_inner,
                   CUtensorMapSwizzle swizzle) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch) * 2};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_rows)};
    return tensor_map_encoder_ready() && encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
                                                      swizzle) == CUDA_SUCCESS;
}

bool encode_operand(CUtensorMap* map, const __nv_bfloat16* base, bool by_k, int rows, int K, int pitch, int box_rows) {
    return by_k ? encode_matrix(map, base, K, rows, pitch, kStepK, 64, CU_TENSOR_MAP_SWIZZLE_128B)
                : encode_matrix(map, base, rows, K, pitch, box_rows, kStepK, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <bool PAIR, int BN, bool TMA>
bool make_job(Job& j, const GemmParams& p, int splits, bool joins, int first) {
    using S = Shape<PAIR, BN, TMA>;
    j.M = p.M;
    j.N = p.N;
    j.K = p.K;
    j.splits = splits;
    j.m_tiles = (p.M + 128 * S::kCtas - 1) / (128 * S::kCtas);
    j.n_tiles = (p.N + BN - 1) / BN;
    j.tiles = j.m_tiles * j.n_tiles;
    j.ksteps = (p.K + kStepK - 1) / kStepK;
    j.first = first;
    j.a_by_k = p.a_by_k;
    j.act = p.act;
    j.bias = p.bias;
    j.r = p.r;
    j.y = p.y;
    j.z = p.z;
    if (!encode_operand(&j.map_a, p.a, p.a_by_k, p.M, p.K, p.a_pitch, 128) ||
        !encode_operand(&j.map_b, p.b, p.b_by_k, p.N, p.K, p.b_pitch, S::kRowsB))
        return false;
    if (joins) return true;
    if (splits > 1) {
        const cuuint64_t pitch = static_cast<cuuint64_t>(part_pitch(p.N)) * 4;
        const cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.N), static_cast<cuuint64_t>(p.M), static_cast<cuuint64_t>(splits)};
        const cuuint64_t strides[2] = {pitch, pitch * static_cast<cuuint64_t>(p.M)};
        const cuuint32_t box[3] = {32, 32, 1};
        return encode_tiled(&j.map_part, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, p.part, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) == CUDA_SUCCESS;
    }
    if (p.N % 8 != 0) return true;
    const auto rows = [&](CUtensorMap* map, const void* base) {
        return base == nullptr || encode_matrix(map, base, p.M, p.N, p.N, 32, kBlockCols, CU_TENSOR_MAP_SWIZZLE_128B);
    };
    return rows(&j.map_y, p.y) && rows(&j.map_z, p.z) && rows(&j.map_r, p.r);
}

template <bool PAIR, int BN, bool B_BY_K, bool TMA>
cudaError_t launch_variant(const GemmParams* p, int count, const GemmTile& t, const ColumnJoin& sums, int num_sms, bool after_other,
                           cudaStream_t stream) {
    using S = Shape<PAIR, BN, TMA>;
    static SmemLimitCache limits;
    auto* fn = linear_gemm_kernel<PAIR, BN, B_BY_K, TMA>;
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(fn), 232448, limits);  // all that a block may have, once
    if (e != cudaSuccess) return e;
    const bool joins = !PAIR && !B_BY_K && gemm_joins_in_cluster(t);
    Launch L;
    L.jobs = count;
    L.units = 0;
    L.join = sums;
    L.status = p[0].status;
    int longest = 0;
    for (int i = 0; i < count; ++i) {
        if (!make_job<PAIR, BN, TMA>(L.job[i], p[i], t.splits[i], joins, L.units)) return cudaErrorInvalidValue;
        L.units += L.job[i].tiles * t.splits[i];
        longest = p[i].K > longest ? p[i].K : longest;
    }
    const int slots = num_sms / S::kCtas;
    // Sixteen epilogue warps where units are short; their buffers cost a stage, which long ones miss (8192 x 4096 x 4096
    // 147 us with five stages, 142 with six).  Two groups where CTAs have several units; of 64 columns a group has all.
    L.ring.warps = longest >= 1024 ? 8 : S::kEpilogueWarps;
    L.ring.groups = BN == 64 || (L.units > slots && L.ring.warps == S::kEpilogueWarps) ? 2 : 1;
    L.ring.stages = S::stages(L.ring.warps);
    L.ring.cluster = joins ? t.splits[0] : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(joins ? L.units : (L.units < slots ? L.units : slots) * S::kCtas));
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = L.ring.stages * S::kSteps * S::kStage + L.ring.warps * S::kOut + S::kBarBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    if (PAIR || joins) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = PAIR ? 2 : t.splits[0];
        attr[cfg.numAttrs].val.clusterDim.y = 1;
        attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    if (after_other) {  // its set-up overlaps the kernel before it
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
        ++cfg.numAttrs;
    }
    cfg.attrs = attr;
    e = cudaLaunchKernelEx(&cfg, fn, L);
    bool early = true;  // a second join comes behind the first, which lets nothing start early
    for (int i = 0; i < count && e == cudaSuccess; ++i) {
        if (t.splits[i] == 1 || joins) continue;
        cudaLaunchConfig_t join = {};
        const long long quads = static_cast<long long>(p[i].M) * ((p[i].N + 3) / 4);
        const int threads = t.splits[i] <= 4 ? 1 : (t.splits[i] <= 16 ? 4 : 16), at_once = kJoinThreads / threads;
        join.gridDim = dim3(static_cast<unsigned>((quads + at_once - 1) / at_once));
        join.blockDim = dim3(kJoinThreads);
        join.stream = stream;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        join.attrs = attr;
        join.numAttrs = early ? 1 : 0;
        early = false;
        auto* kernel = threads == 1 ? linear_join_kernel<1> : (threads == 4 ? linear_join_kernel<4> : linear_join_kernel<16>);
        e = cudaLaunchKernelEx(&join, kernel, p[i], t.splits[i]);
    }
    return e;
}

template <bool B_BY_K, bool TMA>
cudaError_t launch_shape(const GemmParams* p, int count, const GemmTile& t, const ColumnJoin& join, int num_sms, bool after_other,
                            cudaStream_t stream) {
    if (t.columns == 256) return launch_variant<true, 256, B_BY_K, TMA>(p, count, t, join, num_sms, after_other, stream);
    if (t.columns == 128) return launch_variant<false, 128, B_BY_K, TMA>(p, count, t, join, num_sms, after_other, stream);
    return launch_variant<false, 64, B_BY_K, TMA>(p, count, t, join, num_sms, after_other, stream);
}

}  // namespace

bool gemm_fits(int M, int N) { return (static_cast<long long>(M) + 127) / 128 * ((N + 63) / 64) < (1LL << 29); }

bool gemm_joins_in_cluster(const GemmTile& t) { return t.columns <= 128 && (t.splits[0] == 2 || t.splits[0] == 4 || t.splits[0] == 8); }

size_t gemm_part_bytes(int splits, int M, int N) {
    return splits > 1 ? static_cast<size_t>(splits) * M * part_pitch(N) * sizeof(float) : 0;
}

// Clusters of this kernel's CTAs (one an SM) that the part holds at a time, by CTAs in a cluster: a 152-SM part holds
// 76 of 2, 36 of 4 and 15 of 8.
static int clusters_at_a_time(int num_sms, int ctas) {
    return ctas == 2 ? num_sms / 2 : (ctas == 4 ? num_sms * 36 / 152 : num_sms * 15 / 152);
}

// The tile shape and split of K that cost least by these figures, in microseconds on a 152-SM part (repeated launches in a
// graph): the launch with a short tile, a K = 64 step, what a tile takes besides, and the least it takes (its epilogue).
// From one tile on every SM, K = 64 / 256 / 1024 / 4096: 6.5 / 7.4 / 10.8 / 23.4 us of 256 x 256 on pairs, 4.9 / 5.6 / 7.7 / 15.7
// of 128 x 128, 4.3 / 4.8 / 6.8 / 13.9 of 128 x 64; the least is what the epilogue takes where y goes to memory.  A join in a
// cluster takes 4.0 / 3.1 / 2.3 us of 128 columns by 2 / 4 / 8, 2.6 / 2.2 / 2.0 of 64; of parts in the workspace 2 and their way
// through memory, and the second launch 4 of a call where the host is what bounds it, nothing in a graph: half is counted.
// Rows of y off 16 bytes: the last tile's epilogue takes 2 to 4 longer, a cluster's or the join kernel's shares of it 1 to 3.
// Rows of K off 64 bytes: a box's part of a row lies in two lines of L2, and a step takes 0.42 / 0.38 / 0.29 instead of 0.27 /
// 0.20 / 0.155 (4000 x 1000 -> 1000, 1101 x 2504 -> 1544; 8192 x 4096 -> 4096 145 us, 4128 150, 4104 195).
// The gradients' operands come in smaller boxes, and their steps take longer in small tiles when all SMs run: dx and dw of
// 3935 x 2648 -> 1656 82 us in 256 x 256 and 111 in 128 x 128.
// 1000 x 2048 -> 96: 9.4 us whole in a graph, by four in a cluster 7.6, by six through the workspace 7.5.
GemmTile gemm_pick_tile(const GemmSize* products, int count, bool forward, int num_sms) {
    struct Cost {
        int rows, columns;
        double launch, step, besides, least;
    };
    constexpr Cost kForward[3] = {{256, 256, 5.6, 0.27, 0.8, 3.0}, {128, 128, 4.35, 0.20, 0.6, 2.0}, {128, 64, 3.7, 0.155, 0.4, 1.2}};
    constexpr Cost kAcrossLines[3] = {{256, 256, 5.6, 0.42, 0.8, 3.0}, {128, 128, 4.35, 0.38, 0.6, 2.0}, {128, 64, 3.7, 0.29, 0.4, 1.2}};
    constexpr Cost kGradients[3] = {{256, 256, 5.9, 0.29, 1.0, 3.0}, {128, 128, 4.5, 0.235, 0.7, 2.0}, {128, 64, 4.2, 0.22, 0.6, 1.2}};
    constexpr int kSplits[14] = {1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 16, 24, 32, 64};
    double best = 0.0;
    GemmTile pick = {};
    const bool lines = products[0].K % 32 == 0 || (products[0].K % 8 != 0 && products[0].K >= 256);  // laid out on 128 bytes
    for (const Cost& c : !forward ? kGradients : (lines ? kForward : kAcrossLines)) {
        const long long slots = c.rows == 256 ? num_sms / 2 : num_sms;
        const auto tiles = [&](const GemmSize& p) {
            return (static_cast<long long>(p.M) + c.rows - 1) / c.rows * ((p.N + c.columns - 1) / c.columns);
        };
        const auto each = [&](const GemmSize& p, int splits) {
            const long long steps = (static_cast<long long>(p.K) + kStepK - 1) / kStepK;
            const double step = c.columns == 128 && p.N % 8 != 0 && c.step < 0.235 ? 0.235 : c.step;  // one to a turn (kSteps)
            const double t = static_cast<double>((steps + splits - 1) / splits) * step + c.besides;
            return t > c.least ? t : c.least;
        };
        const auto in_cluster = [&](int splits) { return forward && gemm_joins_in_cluster({c.rows, c.columns, {splits, 1}}); };
        const auto allowed = [&](const GemmSize& p, int splits) {
            return splits == 1 || (splits <= (p.K + kStepK - 1) / kStepK &&
                                   (in_cluster(splits) ? tiles(p) <= clusters_at_a_time(num_sms, splits) : tiles(p) * splits <= slots));
        };
        const auto finish = [&](const GemmSize& p, int splits) {
            if (splits == 1) return forward && p.N % 8 != 0 ? 1.2 : 0.0;
            if (in_cluster(splits)) return 1.7 + 0.036 * c.columns / splits + (p.N % 4 != 0 ? 1.0 : 0.0);
            return 3.8 + static_cast<double>(p.M) * p.N * splits * 1e-6;
        };
        for (int s0 : kSplits) {
            if (!allowed(products[0], s0)) continue;
            for (int s1 : kSplits) {
                if (count == 1 ? s1 != 1 : !allowed(products[1], s1)) continue;
                // units are dealt out in turn, the first product's before the second's: the CTA with most to do
                const long long u0 = tiles(products[0]) * s0, u1 = count == 1 ? 0 : tiles(products[1]) * s1;
                const double e0 = each(products[0], s0), e1 = count == 1 ? 0.0 : each(products[1], s1);
                double longest = 0.0;
                for (long long i = 0; i < slots; ++i) {
                    const long long n0 = u0 > i ? (u0 - i - 1) / slots + 1 : 0, all = u0 + u1 > i ? (u0 + u1 - i - 1) / slots + 1 : 0;
                    const double t = static_cast<double>(n0) * e0 + static_cast<double>(all - n0) * e1;
                    longest = t > longest ? t : longest;
                }
                const double cost = c.launch + longest + finish(products[0], s0) + (count == 1 ? 0.0 : finish(products[1], s1));
                if (pick.rows == 0 || cost < best) {
                    best = cost;
                    pick = {c.rows, c.columns, {s0, s1}};
                }
            }
        }
    }
    return pick;
}

cudaError_t launch_gemm(const GemmParams* p, int count, const GemmTile& t, const ColumnJoin& join, int num_sms, bool after_other,
                        cudaStream_t stream) {
    const bool tma = p[0].N % 8 == 0;  // both products of a launch have the same N
    if (p[0].b_by_k)
        return tma ? launch_shape<true, true>(p, count, t, join, num_sms, after_other, stream)
                   : launch_shape<true, false>(p, count, t, join, num_sms, after_other, stream);
    return tma ? launch_shape<false, true>(p, count, t, join, num_sms, after_other, stream)
               : launch_shape<false, false>(p, count, t, join, num_sms, after_other, stream);
}

}  // namespace convgb
