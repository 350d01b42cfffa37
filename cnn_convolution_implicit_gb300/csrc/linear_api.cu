// linear_api.cu -- C ABI of the linear layer (conv_linear_* in include/conv.h): checks, launch
// configuration and the calls.
#include <new>

#include "../../include/conv.h"
#include "int8_internal.h"
#include "linear_internal.h"
#include "status_slots.h"

using namespace convgb;

struct conv_linear_plan {
    int M, N, K, act;
    bool few;                  // the forward product runs in the kernel of few rows
    GemmTile forward, backward;  // tiles of the product, and of the gradients' (the longer sums first; alone they keep the same
                                 // tiles and splits, so that what else a call asks for does not change their bits)
    bool dw_first;
    int device;
    int num_sms;
    unsigned* status;
    int status_slot;  // index of the plan's own status word, -1: the library-wide word, or none
};

namespace {

template <typename... P>
bool all_aligned16(const P*... ptr) {
    return ((reinterpret_cast<uintptr_t>(ptr) | ...) & 15u) == 0;
}

conv_status check_device(const conv_linear_plan* pl) {
    if (pl->device < 0) return CONV_ERR_CUDA;  // host-only plan
    int cur = -1;
    if (cudaGetDevice(&cur) != cudaSuccess) {
        cudaGetLastError();
        return CONV_ERR_CUDA;
    }
    return cur == pl->device ? CONV_OK : CONV_ERR_INVALID_ARG;
}

// A buffer of a call, to tell whether two share memory (nullptr shares none).
struct Span {
    uintptr_t at;
    size_t bytes;
    template <typename T>
    Span(const T* p, size_t n) : at(reinterpret_cast<uintptr_t>(p)), bytes(p == nullptr ? 0 : n) {}
    bool meets(const Span& o) const { return bytes != 0 && o.bytes != 0 && at < o.at + o.bytes && o.at < at + bytes; }
    bool is(const Span& o) const { return at == o.at; }
};

template <typename... S>
bool meets_any(const Span& a, const S&... others) {
    return (a.meets(others) || ...);
}

conv_status launched(cudaError_t e) {
    if (e == cudaSuccess) return CONV_OK;
    cudaGetLastError();
    return CONV_ERR_CUDA;
}

size_t up(size_t v, size_t to) { return (v + to - 1) / to * to; }

// Elements of a row laid out: on 128 bytes (a box's 128 bytes of a row are then one line of L2, not two) unless that lengthens
// a short row.
int pitch_of(int n) { return static_cast<int>(up(n, n < 256 ? 8 : 64)); }

// Workspaces: rows off 16 bytes laid out on them, u, parts of sums.
struct Workspace {
    size_t x, w, u, part, part2, sums, bytes;  // offsets, and bytes in all
};

size_t rows_bytes(long long rows, int n) { return up(static_cast<size_t>(rows) * pitch_of(n) * 2, 256); }

Workspace forward_space(const conv_linear_plan* pl) {
    Workspace ws = {};
    if (pl->few) return ws;
    const bool lay_out = pl->K % 8 != 0;
    ws.w = lay_out ? rows_bytes(pl->M, pl->K) : 0;
    ws.part = ws.w + (lay_out ? rows_bytes(pl->N, pl->K) : 0);
    ws.bytes = ws.part + (gemm_joins_in_cluster(pl->forward) ? 0 : gemm_part_bytes(pl->forward.splits[0], pl->M, pl->N));
    return ws;
}

Workspace backward_space(const conv_linear_plan* pl) {
    Workspace ws = {};
    const bool lay_out = pl->K % 8 != 0;
    ws.w = lay_out ? rows_bytes(pl->M, pl->K) : 0;
    ws.u = ws.w + (lay_out ? rows_bytes(pl->N, pl->K) : 0);
    ws.sums = ws.u + (pl->act != CONV_ACT_NONE || pl->N % 8 != 0 ? rows_bytes(pl->M, pl->N) : 0);
    const int sums = linear_grad_parts(pl->M, pl->N, pl->num_sms);
    ws.part = ws.sums + (sums > 1 ? up(static_cast<size_t>(sums) * pl->N * sizeof(float), 256) : 0);
    ws.part2 = ws.part + up(gemm_part_bytes(pl->backward.splits[pl->dw_first ? 1 : 0], pl->M, pl->K), 256);  // dw's, behind dx's
    ws.bytes = ws.part2 + gemm_part_bytes(pl->backward.splits[pl->dw_first ? 0 : 1], pl->N, pl->K);
    return ws;
}

// Rows of a and of b (either may have none) to rows on 16 bytes.
cudaError_t lay_out(const void* a, void* to_a, long long rows_a, const void* b, void* to_b, long long rows_b, int n, int num_sms,
                    cudaStream_t stream) {
    return launch_int8_layout(static_cast<const int8_t*>(a), static_cast<int8_t*>(to_a), rows_a, static_cast<const int8_t*>(b),
                              static_cast<int8_t*>(to_b), rows_b, 2 * n, 2 * pitch_of(n), num_sms, stream);
}

}  // namespace

extern "C" {

conv_status conv_linear_plan_create(conv_linear_plan** out, int M, int N, int K, conv_act act) {
    if (out == nullptr) return CONV_ERR_INVALID_ARG;
    *out = nullptr;
    if (M <= 0 || N <= 0 || K <= 0) return CONV_ERR_INVALID_ARG;
    if (act != CONV_ACT_NONE && act != CONV_ACT_RELU && act != CONV_ACT_SILU) return CONV_ERR_INVALID_ARG;
    const long long most = 1LL << 40;
    const int side = 1 << 29;
    if (M >= side || N >= side || K >= side || static_cast<long long>(M) * K > most ||
        static_cast<long long>(N) * K > most || static_cast<long long>(M) * N > most)
        return CONV_ERR_UNSUPPORTED;
    if (!gemm_fits(M, N) || !gemm_fits(M, K) || !gemm_fits(N, K)) return CONV_ERR_UNSUPPORTED;
    conv_linear_plan* pl = new (std::nothrow) conv_linear_plan();
    if (pl == nullptr) return CONV_ERR_NO_MEMORY;
    pl->M = M;
    pl->N = N;
    pl->K = K;
    pl->act = act;
    pl->status_slot = -1;
    int ndev = 0;
    if (cudaGetDeviceCount(&ndev) != cudaSuccess || ndev == 0) {
        cudaGetLastError();
        pl->device = -1;
        pl->num_sms = 152;
    } else if (cudaGetDevice(&pl->device) != cudaSuccess ||
               cudaDeviceGetAttribute(&pl->num_sms, cudaDevAttrMultiProcessorCount, pl->device) != cudaSuccess ||
               acquire_status_word(pl->device, &pl->status, &pl->status_slot) != cudaSuccess) {
        cudaGetLastError();
        delete pl;
        return CONV_ERR_CUDA;
    }
    pl->few = linear_use_few(M, N, K);
    const GemmSize forward = {M, N, K}, dx = {M, K, N}, dw = {N, K, M};
    pl->forward = gemm_pick_tile(&forward, 1, true, pl->num_sms);
    pl->dw_first = M > N;
    const GemmSize both[2] = {pl->dw_first ? dw : dx, pl->dw_first ? dx : dw};
    pl->backward = gemm_pick_tile(both, 2, false, pl->num_sms);
    *out = pl;
    return CONV_OK;
}

conv_status conv_linear_workspace(const conv_linear_plan* p, unsigned long long* forward, unsigned long long* backward) {
    if (p == nullptr) return CONV_ERR_INVALID_ARG;
    if (forward != nullptr) *forward = forward_space(p).bytes;
    if (backward != nullptr) *backward = backward_space(p).bytes;
    return CONV_OK;
}

conv_status conv_linear_forward(conv_linear_plan* pl, const void* x, const void* w, const float* bias,
                                const void* residual, void* y, void* z, void* workspace, void* stream) {
    if (pl == nullptr || x == nullptr || w == nullptr || y == nullptr) return CONV_ERR_INVALID_ARG;
    const Workspace ws = forward_space(pl);
    if (workspace == nullptr && ws.bytes != 0) return CONV_ERR_INVALID_ARG;
    if (!all_aligned16(x, w, bias, residual, y, z, workspace)) return CONV_ERR_MISALIGNED;
    const conv_status s = check_device(pl);
    if (s != CONV_OK) return s;
    const size_t M = pl->M, N = pl->N, K = pl->K;
    const Span sx(x, 2 * M * K), sw(w, 2 * N * K), sb(bias, 4 * N), sr(residual, 2 * M * N), sy(y, 2 * M * N), sz(z, 2 * M * N);
    if (meets_any(sy, sx, sw, sb, sz) || meets_any(sz, sx, sw, sb, sr) || (sy.meets(sr) && !sy.is(sr))) return CONV_ERR_INVALID_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (pl->few) {
        const FewParams f = {pl->M, pl->N, pl->K, static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(w), bias,
                             static_cast<const __nv_bfloat16*>(residual), static_cast<__nv_bfloat16*>(y),
                             static_cast<__nv_bfloat16*>(z), pl->act};
        return launched(launch_linear_few(f, st));
    }
    uint8_t* base = static_cast<uint8_t*>(workspace);
    GemmParams p = {};
    p.M = pl->M;
    p.N = pl->N;
    p.K = pl->K;
    p.a = static_cast<const __nv_bfloat16*>(x);
    p.b = static_cast<const __nv_bfloat16*>(w);
    p.a_pitch = p.b_pitch = p.K;
    const bool laid_out = p.K % 8 != 0;
    if (laid_out) {
        const cudaError_t e = lay_out(x, base + ws.x, p.M, w, base + ws.w, p.N, p.K, pl->num_sms, st);
        if (e != cudaSuccess) return launched(e);
        p.a = reinterpret_cast<const __nv_bfloat16*>(base + ws.x);
        p.b = reinterpret_cast<const __nv_bfloat16*>(base + ws.w);
        p.a_pitch = p.b_pitch = pitch_of(p.K);
    }
    p.act = pl->act;
    p.bias = bias;
    p.r = static_cast<const __nv_bfloat16*>(residual);
    p.y = static_cast<__nv_bfloat16*>(y);
    p.z = static_cast<__nv_bfloat16*>(z);
    p.part = reinterpret_cast<float*>(base + ws.part);
    p.status = pl->status;
    return launched(launch_gemm(&p, 1, pl->forward, ColumnJoin(), pl->num_sms, laid_out, st));
}

conv_status conv_linear_backward(conv_linear_plan* pl, const void* dy, const void* x, const void* w, const void* z,
                                 void* dx, void* dw, float* dbias, void* workspace, void* stream) {
    if (pl == nullptr || dy == nullptr || (dx == nullptr && dw == nullptr && dbias == nullptr) ||
        (dx != nullptr && w == nullptr) || (dw != nullptr && x == nullptr) || (pl->act != CONV_ACT_NONE && z == nullptr))
        return CONV_ERR_INVALID_ARG;
    const Workspace ws = backward_space(pl);
    if (workspace == nullptr && ws.bytes != 0) return CONV_ERR_INVALID_ARG;
    if (!all_aligned16(dy, x, w, z, dx, dw, dbias, workspace)) return CONV_ERR_MISALIGNED;
    const conv_status s = check_device(pl);
    if (s != CONV_OK) return s;
    const size_t M = pl->M, N = pl->N, K = pl->K;
    const Span sy(dy, 2 * M * N), sx(x, 2 * M * K), sw(w, 2 * N * K), sz(z, 2 * M * N);
    const Span gx(dx, 2 * M * K), gw(dw, 2 * N * K), gb(dbias, 4 * N);
    if (meets_any(gx, sy, sx, sw, sz, gw, gb) || meets_any(gw, sy, sx, sw, sz, gb) || meets_any(gb, sy, sx, sw, sz)) return CONV_ERR_INVALID_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint8_t* base = static_cast<uint8_t*>(workspace);
    const bool products = dx != nullptr || dw != nullptr;
    const __nv_bfloat16* u = static_cast<const __nv_bfloat16*>(dy);
    int u_pitch = pl->N;
    ColumnJoin join = {};  // dbias's parts, left to the products' launch
    const bool copy = products && (pl->act != CONV_ACT_NONE || pl->N % 8 != 0);
    cudaError_t e = cudaSuccess;
    bool early = false;  // the kernel before the products lets them start early
    if (copy || dbias != nullptr) {
        early = products;
        LinearGradParams g = {};
        g.M = pl->M;
        g.N = pl->N;
        g.dy = u;
        g.z = static_cast<const __nv_bfloat16*>(z);
        if (copy) {
            g.u = reinterpret_cast<__nv_bfloat16*>(base + ws.u);
            u = g.u;
            u_pitch = pitch_of(pl->N);
        }
        g.u_pitch = u_pitch;
        g.part = reinterpret_cast<float*>(base + ws.sums);
        g.dbias = dbias;
        g.act = pl->act;
        e = launch_linear_grad(g, pl->num_sms, !products, st);
        const int parts = linear_grad_parts(pl->M, pl->N, pl->num_sms);
        if (products && dbias != nullptr && parts > 1) join = {g.part, dbias, parts, pl->N};
    }
    const __nv_bfloat16* xs = static_cast<const __nv_bfloat16*>(x);
    const __nv_bfloat16* wt = static_cast<const __nv_bfloat16*>(w);
    int k_pitch = pl->K;
    if (e == cudaSuccess && products && pl->K % 8 != 0) {
        early = true;
        e = lay_out(x, base + ws.x, dw != nullptr ? pl->M : 0, w, base + ws.w, dx != nullptr ? pl->N : 0, pl->K, pl->num_sms, st);
        xs = reinterpret_cast<const __nv_bfloat16*>(base + ws.x);
        wt = reinterpret_cast<const __nv_bfloat16*>(base + ws.w);
        k_pitch = pitch_of(pl->K);
    }
    if (e != cudaSuccess || !products) return launched(e);
    GemmParams p[2] = {};
    GemmTile tile = pl->backward;
    const auto product = [&](GemmParams& g, int M, int K, const __nv_bfloat16* b, void* y, size_t part) {
        g.M = M;
        g.N = pl->K;
        g.K = K;
        g.a = u;
        g.a_pitch = u_pitch;
        g.b = b;
        g.b_pitch = k_pitch;
        g.b_by_k = true;
        g.y = static_cast<__nv_bfloat16*>(y);
        g.part = reinterpret_cast<float*>(base + part);
        g.status = pl->status;
    };
    const int at_dx = pl->dw_first ? 1 : 0, at_dw = 1 - at_dx;  // in tile's order
    if (dx != nullptr) product(p[at_dx], pl->M, pl->N, wt, dx, ws.part);
    if (dw != nullptr) {
        product(p[at_dw], pl->N, pl->M, xs, dw, ws.part2);
        p[at_dw].a_by_k = true;
    }
    const int only = dx == nullptr ? at_dw : (dw == nullptr ? at_dx : -1);
    if (only == 1) {
        p[0] = p[1];
        tile.splits[0] = tile.splits[1];
    }
    return launched(launch_gemm(p, only < 0 ? 2 : 1, tile, join, pl->num_sms, early, st));
}

conv_status conv_linear_plan_info(const conv_linear_plan* p, conv_linear_info* info) {
    if (p == nullptr || info == nullptr) return CONV_ERR_INVALID_ARG;
    *info = conv_linear_info();
    info->kernel = p->few ? CONV_LINEAR_FEW_ROWS : CONV_LINEAR_TILES;
    if (!p->few) {
        info->rows = p->forward.rows;
        info->columns = p->forward.columns;
        info->splits = p->forward.splits[0];
    }
    info->grad_rows = p->backward.rows;
    info->grad_columns = p->backward.columns;
    info->dx_splits = p->backward.splits[p->dw_first ? 1 : 0];
    info->dw_splits = p->backward.splits[p->dw_first ? 0 : 1];
    return CONV_OK;
}

conv_status conv_linear_plan_device_status(const conv_linear_plan* p, void* stream, int* code) {
    if (p == nullptr || code == nullptr) return CONV_ERR_INVALID_ARG;
    *code = 0;
    if (p->device < 0) return CONV_ERR_CUDA;  // host-only plan
    if (p->status == nullptr) {  // no kernel of the plan writes one: clean, once the stream is done
        const conv_status s = check_device(p);
        if (s != CONV_OK) return s;
        return launched(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)));
    }
    return read_status_word(p->device, p->status, stream, code);
}

conv_status conv_linear_plan_destroy(conv_linear_plan* p) {
    if (p != nullptr) release_status_word(p->device, p->status_slot);
    delete p;
    return CONV_OK;
}

}  // extern "C"
