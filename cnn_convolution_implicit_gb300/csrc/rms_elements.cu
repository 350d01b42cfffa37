// rms_elements.cu -- the root-mean-square norm of rows that do not start on 16 bytes, up to 8,192 values: forward, to
// 8 bits, and backward (the formulas stand in rms_norm.cu).
//
// Bound by memory like the aligned forms.  Rows are next to each other in memory, so a group of them is one run of
// bytes whose whole 16-byte granules move by bulk copies, both ways, whatever the rows' starts; in shared memory a
// thread takes single values, neighbouring lanes neighbouring ones, and keeps the same columns in every row (gamma and
// the sums of dgamma stay in registers).  Handled as granules in registers, with gamma and dgamma's columns read apart,
// 8192 x 4099 BF16 took 106 us forward and 322 backward; it takes 46 and 68 so, 58 to 8 bits.
//
// Warps: eight work on rows (eight rows of one warp each, or one row of all), one brings groups into the ring, one
// sends results, which replace their inputs there, back.  The first and last granule of a group, shared with the
// neighbouring groups, are written by elements; what of the tensor's last granule is not the tensor's is not read.
#include "rms_math.cuh"
#include "row_sums.cuh"
#include "rows_internal.h"

namespace convgb {

namespace {

enum Mode { kForward, kForwardInt8, kBackward };

constexpr int kThreads = 32 * (kStreamWarps + 2);

__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(reinterpret_cast<uint64_t>(dst)), "r"(smem_addr(src)),
                 "r"(bytes)
                 : "memory");
}

// A group of rows as bytes of its tensor: [start, end), from granule `base` on; [inner, outer) are whole granules of its own.
struct Run {
    long long start, end, base, inner, outer;
    __device__ __forceinline__ Run(long long m, int rows, long long row_bytes) {
        start = m * row_bytes;
        end = start + rows * row_bytes;
        base = start & ~15LL;
        inner = (start + 15) & ~15LL;
        outer = end & ~15LL;
    }
};

template <typename T, int E, int WARPS, int MODE>
__global__ void __launch_bounds__(kThreads, 2) rms_element_kernel(const RmsParams p, const Stream s) {
    constexpr bool kBack = MODE == kBackward;
    constexpr int kStride = 32 * WARPS, es = static_cast<int>(sizeof(T));
    const int rows = WARPS > 1 ? 1 : s.rows;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ uint64_t full[kStreamMaxStages], done[kStreamMaxStages], empty[kStreamMaxStages];
    __shared__ float sums[2][kStreamWarps];
    __shared__ uint32_t tops[2][kStreamWarps];
    __shared__ int abort_flag;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join of dgamma's parts
    volatile int* abort = &abort_flag;
    if (threadIdx.x == 0) {
        for (int i = 0; i < s.stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&done[i], kStreamWarps);
            mbar_init(&empty[i], 1);
        }
        abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    const long long row_bytes = static_cast<long long>(p.C) * es;
    const int tile_bytes = (rows * p.C * es + 14 + 15) & ~15;  // of one tensor, from the granule that holds its first byte
    const GroupRange range(static_cast<int>((static_cast<long long>(p.M) + rows - 1) / rows), kBack ? p.rounds : 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const auto run_of = [&](int g) {
        const long long m = static_cast<long long>(g) * rows;
        return Run(m, static_cast<int>(p.M - m < rows ? p.M - m : rows), row_bytes);
    };
    int st = 0;
    uint32_t ph = 0;
    const auto next = [&] {
        if (++st == s.stages) {
            st = 0;
            ph ^= 1u;
        }
    };
    if (warp == kStreamWarps) {
        // ------------------------------------------------------------ groups into the ring
        if (lane != 0) return;
        const uint8_t* from[3] = {static_cast<const uint8_t*>(p.x), static_cast<const uint8_t*>(kBack ? p.h_in : p.r),
                                  static_cast<const uint8_t*>(kBack ? p.r : nullptr)};
        const int tensors = kBack ? (p.r != nullptr ? 3 : 2) : (p.r != nullptr ? 2 : 1);
        const long long last = p.M * row_bytes;
        long long issued = 0;
        for (int g = range.first; g < range.end; g += range.step) {
            if (!mbar_wait(&empty[st], ph ^ 1u, abort)) {
                record_status(p.status, kStatusTimeoutProducer, abort);
                break;
            }
            const Run run = run_of(g);
            const long long up = (run.end + 15) & ~15LL, copied = up <= last ? up : last & ~15LL;  // to where whole granules go
            uint8_t* stage = ring + st * s.stage_bytes;
            for (int i = 0; i < tensors; ++i)
                for (long long b = copied > run.start ? copied : run.start; b < run.end; b += es)
                    *reinterpret_cast<T*>(stage + i * tile_bytes + (b - run.base)) = *reinterpret_cast<const T*>(from[i] + b);
            const uint32_t bytes = copied > run.base ? static_cast<uint32_t>(copied - run.base) : 0u;
            mbar_arrive_expect_tx(&full[st], tensors * bytes);
            for (int i = 0; i < tensors && bytes != 0; ++i) bulk_load(stage + i * tile_bytes, from[i] + run.base, bytes, &full[st]);
            ++issued;
            next();
        }
        for (int i = 0; i < s.stages; ++i) {  // no copy in flight when the CTA leaves
            const long long fills = issued / s.stages + (i < issued % s.stages ? 1 : 0);
            if (fills && !mbar_wait(&full[i], static_cast<uint32_t>((fills - 1) & 1), nullptr)) record_status(p.status, kStatusTimeoutDrain, abort);
        }
        return;
    }
    if (warp == kStreamWarps + 1) {
        // ------------------------------------------------------------ results to memory
        const auto send = [&](void* to, const uint8_t* tile, const Run& run) {  // whole granules by one lane, the edges by elements
            uint8_t* out = static_cast<uint8_t*>(to);
            const long long head = run.inner < run.end ? run.inner : run.end, tail = run.outer > head ? run.outer : head;
            const long long at = lane < 16 ? run.start + lane * es : tail + (lane - 16) * es;
            if (at < (lane < 16 ? head : run.end)) *reinterpret_cast<T*>(out + at) = *reinterpret_cast<const T*>(tile + (at - run.base));
            if (lane == 0 && run.outer > run.inner) bulk_store(out + run.inner, tile + (run.inner - run.base), static_cast<uint32_t>(run.outer - run.inner));
        };
        for (int g = range.first; g < range.end; g += range.step) {
            if (!__all_sync(0xffffffffu, mbar_wait(&done[st], ph, abort))) {
                record_status(p.status, kStatusTimeoutEpilogue, abort);
                break;
            }
            const Run run = run_of(g);
            const uint8_t* stage = ring + st * s.stage_bytes;
            if constexpr (MODE != kForwardInt8) send(p.y, stage, run);
            if (!kBack && p.h != nullptr) send(p.h, stage + tile_bytes, run);
            if (lane == 0) {
                bulk_commit();
                bulk_wait_read_all();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
            next();
        }
        if (lane == 0) bulk_wait_all();
        return;
    }
    // ---------------------------------------------------------------- rows
    const int t = WARPS == 1 ? lane : static_cast<int>(threadIdx.x), slot = WARPS == 1 ? warp : 0;
    float gamma[E], total[kBack ? E : 1] = {};
#pragma unroll
    for (int k = 0; k < E; ++k) {
        const int c = t + k * kStride;
        gamma[k] = c < p.C ? (p.gamma != nullptr ? __ldg(p.gamma + c) : 1.0f) : 0.0f;
    }
    int turn = 0;
    const auto row_total = [&](float v) {
        v = warp_sum(v);
        if constexpr (WARPS > 1) {
            if (lane == 0) sums[turn][warp] = v;
            sync_consumers();
            v = 0.0f;
#pragma unroll
            for (int i = 0; i < WARPS; ++i) v += sums[turn][i];
        }
        return v;
    };
    const bool with_r = p.r != nullptr;
    for (int g = range.first; g < range.end; g += range.step, turn ^= 1) {
        if (!mbar_wait(&full[st], ph, abort)) record_status(p.status, kStatusTimeoutTransform, abort);  // and on: every wait ends
        const Run run = run_of(g);
#pragma unroll 1
        for (int at = slot; at < rows; at += kStreamWarps) {  // once, where all warps share a row
            const long long m = static_cast<long long>(g) * rows + at;
            if (m >= p.M) break;
            T* own0 = reinterpret_cast<T*>(ring + st * s.stage_bytes + (run.start - run.base)) + at * p.C;  // results take their inputs' place
            T* own1 = reinterpret_cast<T*>(reinterpret_cast<uint8_t*>(own0) + tile_bytes);
            if constexpr (!kBack) {
                float v[E], square = 0.0f;
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    const int c = t + k * kStride;
                    v[k] = 0.0f;
                    if (c >= p.C) continue;
                    v[k] = static_cast<float>(own0[c]);
                    if (with_r) v[k] = __fadd_rn(v[k], static_cast<float>(own1[c]));
                    square = fmaf(v[k], v[k], square);
                }
                const float rstd = reciprocal_root(row_total(square), p.C, p.eps);
                if (t == 0 && p.rstd != nullptr) p.rstd[m] = rstd;
                float top = 0.0f;
                const bool with_h = p.h != nullptr;
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    const int c = t + k * kStride;
                    if (c >= p.C) continue;
                    if (with_h) own1[c] = static_cast<T>(v[k]);
                    v[k] = __fmul_rn(__fmul_rn(v[k], rstd), gamma[k]);
                    if constexpr (MODE == kForward) own0[c] = static_cast<T>(v[k]);
                    else top = max_magnitude(top, v[k]);
                }
                if constexpr (MODE == kForwardInt8) {
                    uint32_t bits = warp_max(magnitude_bits(top));
                    if constexpr (WARPS > 1) {
                        if (lane == 0) tops[turn][warp] = bits;
                        sync_consumers();
#pragma unroll
                        for (int i = 0; i < WARPS; ++i) bits = max(bits, tops[turn][i]);
                    }
                    const RowScale rs = row_scale(bits);
                    const RowFactor rf = row_factor(rs.inv);
                    if (t == 0) p.scale[m] = rs.scale;
                    int8_t* q = p.q + m * p.C;
#pragma unroll
                    for (int k = 0; k < E; ++k) {
                        const int c = t + k * kStride;
                        if (c < p.C) q[c] = quantise1(v[k], rf);
                    }
                }
            } else {
                const T* own2 = reinterpret_cast<const T*>(reinterpret_cast<const uint8_t*>(own1) + tile_bytes);
                const float rstd = __ldg(p.rstd + m);
                float dot = 0.0f;
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    const int c = t + k * kStride;
                    if (c >= p.C) continue;
                    const float dy = static_cast<float>(own0[c]), n = __fmul_rn(static_cast<float>(own1[c]), rstd);
                    total[k] = fmaf(dy, n, total[k]);
                    dot = fmaf(__fmul_rn(dy, gamma[k]), n, dot);
                }
                const float mean = __fdiv_rn(row_total(dot), static_cast<float>(p.C));
#pragma unroll
                for (int k = 0; k < E; ++k) {  // from shared memory again: registers are scarcer
                    const int c = t + k * kStride;
                    if (c >= p.C) continue;
                    const float n = __fmul_rn(static_cast<float>(own1[c]), rstd), d = __fmul_rn(static_cast<float>(own0[c]), gamma[k]);
                    own0[c] = static_cast<T>(fmaf(fmaf(n, -mean, d), rstd, with_r ? static_cast<float>(own2[c]) : 0.0f));
                }
            }
        }
        fence_proxy_async_smem();  // before the bulk copies out, and the next group's into the same place
        __syncwarp();
        if (lane == 0) mbar_arrive(&done[st]);
        next();
    }
    if constexpr (kBack) {
        if (p.dgamma == nullptr) return;
        float* part = p.part + static_cast<long long>(blockIdx.x) * p.C;
        float* warps = reinterpret_cast<float*>(ring);
        if constexpr (WARPS == 1) {  // the warps' sums, in the ring once every stage has left it
            const int mine = range.count();
            for (int i = 0; i < s.stages; ++i) {
                const int fills = mine / s.stages + (i < mine % s.stages ? 1 : 0);
                if (fills && !mbar_wait(&empty[i], static_cast<uint32_t>((fills - 1) & 1), abort)) record_status(p.status, kStatusTimeoutTransform, abort);
            }
            sync_consumers();
            part = warps + warp * p.C;
        }
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const int c = t + k * kStride;
            if (c < p.C) part[c] = total[k];
        }
        if constexpr (WARPS == 1) {
            sync_consumers();
            for (int c = threadIdx.x; c < p.C; c += 32 * kStreamWarps) {
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < kStreamWarps; ++i) sum += warps[i * p.C + c];
                p.part[static_cast<long long>(blockIdx.x) * p.C + c] = sum;
            }
        }
    }
}

// Values a thread holds, warps to a row.
struct Form {
    int values, warps;
};
Form form_of(int C) {
    const int warps = C <= 1024 ? 1 : kStreamWarps, per = C / (32 * warps) + (C % (32 * warps) != 0);
    return {per <= 8 ? 8 : (per <= 16 ? 16 : (per <= 24 ? 24 : 32)), warps};
}

template <typename T, int E, int WARPS, int MODE>
cudaError_t launch(const RmsParams& p, cudaStream_t stream) {
    constexpr bool kBack = MODE == kBackward;
    static SmemLimitCache limits;
    auto* kernel = rms_element_kernel<T, E, WARPS, MODE>;
    const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), 225 * 1024, limits);
    if (e != cudaSuccess) return e;
    const int tensors = (kBack ? 2 : 1) + (p.r != nullptr ? 1 : 0);
    Stream s;
    s.rows = stream_rows(p.M, WARPS == 1 ? kStreamWarps : 1, kBack ? 3 : 2, static_cast<long long>(p.C) * sizeof(T), p.ctas);
    s.stage_bytes = tensors * ((s.rows * p.C * static_cast<int>(sizeof(T)) + 14 + 15) & ~15);
    s.stages = 112 * 1024 / s.stage_bytes;  // two CTAs an SM
    if (s.stages == 0) s.stages = 225 * 1024 / s.stage_bytes;
    if (s.stages > kStreamMaxStages) s.stages = kStreamMaxStages;
    const long long need = (static_cast<long long>(p.M) + s.rows - 1) / s.rows;
    const long long ctas = kBack && p.dgamma != nullptr ? p.parts : (need < p.ctas ? need : p.ctas);
    RmsParams q = p;
    if (p.dgamma == nullptr) q.rounds = 1;
    kernel<<<static_cast<unsigned>(ctas), kThreads, s.stages * s.stage_bytes, stream>>>(q, s);
    return cudaGetLastError();
}

template <typename T, int WARPS, int MODE>
cudaError_t by_values(const RmsParams& p, int values, cudaStream_t stream) {
    if (values == 8) return launch<T, 8, WARPS, MODE>(p, stream);
    if (values == 16) return launch<T, 16, WARPS, MODE>(p, stream);
    return values == 24 ? launch<T, 24, WARPS, MODE>(p, stream) : launch<T, 32, WARPS, MODE>(p, stream);
}

template <typename T, int MODE>
cudaError_t by_form(const RmsParams& p, cudaStream_t stream) {
    const Form f = form_of(p.C);
    return f.warps == 1 ? by_values<T, 1, MODE>(p, f.values, stream) : by_values<T, kStreamWarps, MODE>(p, f.values, stream);
}

template <typename T>
cudaError_t by_mode(const RmsParams& p, bool backward, cudaStream_t stream) {
    if (backward) return by_form<T, kBackward>(p, stream);
    return p.q != nullptr ? by_form<T, kForwardInt8>(p, stream) : by_form<T, kForward>(p, stream);
}

}  // namespace

bool rms_by_elements(const RmsParams& p) { return p.C % (p.bf16 ? 8 : 4) != 0 && p.C <= 8192; }

void rms_plan_elements(RmsParams& p) {
    const int at_once = form_of(p.C).warps == 1 ? kStreamWarps : 1;
    const int rows = stream_rows(p.M, at_once, 3, static_cast<long long>(p.C) * (p.bf16 ? 2 : 4), p.ctas);
    const long long need = (static_cast<long long>(p.M) + rows - 1) / rows;
    p.rounds = chain_rounds(p.M, at_once, p.ctas);
    if (need <= 4) p.parts = 1;  // as plan_stream
    else if (need < p.ctas) p.parts = static_cast<int>(need);
    else p.parts = p.rounds * p.ctas;
}

cudaError_t launch_rms_elements(const RmsParams& p, bool backward, cudaStream_t stream) {
    return p.bf16 ? by_mode<__nv_bfloat16>(p, backward, stream) : by_mode<float>(p, backward, stream);
}

}  // namespace convgb
