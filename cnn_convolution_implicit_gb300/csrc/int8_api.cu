// int8_api.cu -- C ABI of the 8-bit product and of the row quantiser
// (conv_int8_*, conv_quantize_rows in include/conv.h): checks, launch
// configuration and the calls.
#include <new>

#include "../../include/conv.h"
#include "int8_internal.h"
#include "status_slots.h"

using namespace convgb;

struct conv_int8_plan {
    Int8Params ip;
    int device;
    int num_sms;
    int status_slot;  // index of the plan's own status word, -1: the library-wide word, or none
};

namespace {

constexpr int kMaxK = 131071;  // 128 * 128 * K stays below 2^31

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

conv_status check_device(const conv_int8_plan* pl) {
    if (pl->device < 0) return CONV_ERR_CUDA;  // host-only plan
    int cur = -1;
    if (cudaGetDevice(&cur) != cudaSuccess) {
        cudaGetLastError();
        return CONV_ERR_CUDA;
    }
    return cur == pl->device ? CONV_OK : CONV_ERR_INVALID_ARG;
}

size_t up(size_t v, size_t to) { return (v + to - 1) / to * to; }

// Workspace of the tensor-core forms: rows of x that they quantise, with their scales; for many rows also
// those of x and w that do not start on 16 bytes.
struct Workspace {
    int pitch;                // bytes between rows
    size_t x, w, scales;      // offsets
    size_t forward, quantize; // bytes of either call
};

Workspace workspace_of(const Int8Params& p) {
    Workspace ws = {};
    if (!int8_use_gemm(p) && !int8_use_mid(p)) return ws;
    ws.pitch = static_cast<int>(up(p.K, 16));
    const size_t x = up(static_cast<size_t>(p.M) * ws.pitch, 256);
    const size_t w = p.K % 16 != 0 && int8_use_gemm(p) ? up(static_cast<size_t>(p.N) * ws.pitch, 256) : 0;
    ws.w = x;
    ws.scales = x + w;
    ws.forward = w != 0 ? x + w : 0;
    ws.quantize = ws.scales + static_cast<size_t>(p.M) * sizeof(float);
    return ws;
}

conv_status launched(cudaError_t e) {
    if (e == cudaSuccess) return CONV_OK;
    cudaGetLastError();
    return CONV_ERR_CUDA;
}

}  // namespace

extern "C" {

conv_status conv_int8_plan_create(conv_int8_plan** out, int M, int N, int K, conv_dtype out_dtype, conv_act act) {
    if (out == nullptr) return CONV_ERR_INVALID_ARG;
    *out = nullptr;
    if (M <= 0 || N <= 0 || K <= 0) return CONV_ERR_INVALID_ARG;
    if (out_dtype != CONV_F32 && out_dtype != CONV_BF16) return CONV_ERR_INVALID_ARG;
    if (act != CONV_ACT_NONE && act != CONV_ACT_RELU && act != CONV_ACT_SILU) return CONV_ERR_INVALID_ARG;
    const long long most = 1LL << 40;
    if (K > kMaxK || static_cast<long long>(M) * K > most || static_cast<long long>(N) * K > most ||
        static_cast<long long>(M) * N > most)
        return CONV_ERR_UNSUPPORTED;
    conv_int8_plan* pl = new (std::nothrow) conv_int8_plan();
    if (pl == nullptr) return CONV_ERR_NO_MEMORY;
    Int8Params& p = pl->ip;
    p = Int8Params();
    p.M = M;
    p.N = N;
    p.K = K;
    p.out_bf16 = out_dtype == CONV_BF16;
    p.act = act;
    if (int8_use_gemm(p) && !int8_gemm_fits(p)) {
        delete pl;
        return CONV_ERR_UNSUPPORTED;
    }
    pl->status_slot = -1;
    int ndev = 0;
    if (cudaGetDeviceCount(&ndev) != cudaSuccess || ndev == 0) {
        cudaGetLastError();
        pl->device = -1;
        pl->num_sms = 152;
    } else if (cudaGetDevice(&pl->device) != cudaSuccess ||
               cudaDeviceGetAttribute(&pl->num_sms, cudaDevAttrMultiProcessorCount, pl->device) != cudaSuccess ||
               // the kernels of few rows wait for nothing: no word of the pool for them
               (int8_use_gemm(p) && acquire_status_word(pl->device, &p.status, &pl->status_slot) != cudaSuccess)) {
        cudaGetLastError();
        delete pl;
        return CONV_ERR_CUDA;
    }
    *out = pl;
    return CONV_OK;
}

conv_status conv_int8_forward(conv_int8_plan* pl, const void* x, const float* x_scale, const void* w,
                              const float* w_scale, const float* bias, void* y, void* workspace, void* stream) {
    if (pl == nullptr || x == nullptr || x_scale == nullptr || w == nullptr || w_scale == nullptr || y == nullptr)
        return CONV_ERR_INVALID_ARG;
    const Workspace ws = workspace_of(pl->ip);
    if (workspace == nullptr && ws.forward != 0) return CONV_ERR_INVALID_ARG;
    for (const void* ptr : {x, static_cast<const void*>(x_scale), w, static_cast<const void*>(w_scale),
                            static_cast<const void*>(bias), static_cast<const void*>(y),
                            static_cast<const void*>(workspace)})
        if (ptr != nullptr && !aligned16(ptr)) return CONV_ERR_MISALIGNED;
    const conv_status s = check_device(pl);
    if (s != CONV_OK) return s;
    Int8Params p = pl->ip;
    p.x = static_cast<const int8_t*>(x);
    p.x_scale = x_scale;
    p.w = static_cast<const int8_t*>(w);
    p.w_scale = w_scale;
    p.bias = bias;
    p.y = y;
    p.x_pitch = p.w_pitch = p.K;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (int8_use_mid(p)) return launched(launch_int8_mid(p, false, st));
    if (!int8_use_gemm(p)) return launched(launch_int8_few(p, st));
    if (ws.forward != 0) {
        int8_t* base = static_cast<int8_t*>(workspace);
        const cudaError_t e = launch_int8_layout(p.x, base + ws.x, p.M, p.w, base + ws.w, p.N, p.K, ws.pitch, pl->num_sms, st);
        if (e != cudaSuccess) return launched(e);
        p.x = base + ws.x;
        p.w = base + ws.w;
        p.x_pitch = p.w_pitch = ws.pitch;
    }
    return launched(launch_int8_gemm(p, pl->num_sms, ws.forward != 0, st));
}

conv_status conv_int8_workspace(const conv_int8_plan* p, unsigned long long* forward, unsigned long long* quantize) {
    if (p == nullptr) return CONV_ERR_INVALID_ARG;
    const Workspace ws = workspace_of(p->ip);
    if (forward) *forward = ws.forward;
    if (quantize) *quantize = ws.quantize;
    return CONV_OK;
}

conv_status conv_int8_forward_quantize(conv_int8_plan* pl, const void* x, conv_dtype x_dtype, const void* w,
                                       const float* w_scale, const float* bias, void* y, void* workspace,
                                       void* stream) {
    if (pl == nullptr || x == nullptr || w == nullptr || w_scale == nullptr || y == nullptr ||
        (workspace == nullptr && workspace_of(pl->ip).quantize != 0))
        return CONV_ERR_INVALID_ARG;
    if (x_dtype != CONV_F32 && x_dtype != CONV_BF16) return CONV_ERR_INVALID_ARG;
    for (const void* ptr : {x, w, static_cast<const void*>(w_scale), static_cast<const void*>(bias),
                            static_cast<const void*>(y), static_cast<const void*>(workspace)})
        if (ptr != nullptr && !aligned16(ptr)) return CONV_ERR_MISALIGNED;
    const conv_status s = check_device(pl);
    if (s != CONV_OK) return s;
    Int8Params p = pl->ip;
    p.w = static_cast<const int8_t*>(w);
    p.w_scale = w_scale;
    p.bias = bias;
    p.y = y;
    if (!int8_use_gemm(p) && !int8_use_mid(p))
        return launched(launch_int8_few_quantize(p, x, x_dtype == CONV_BF16, static_cast<cudaStream_t>(stream)));
    const Workspace ws = workspace_of(p);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    int8_t* base = static_cast<int8_t*>(workspace);
    float* scale = reinterpret_cast<float*>(base + ws.scales);
    p.w_pitch = p.K;
    cudaError_t e = cudaSuccess;
    if (p.K % 16 != 0 && int8_use_gemm(p)) {
        e = launch_int8_layout(nullptr, nullptr, 0, p.w, base + ws.w, p.N, p.K, ws.pitch, pl->num_sms, st);
        p.w = base + ws.w;
        p.w_pitch = ws.pitch;
    }
    if (e == cudaSuccess)
        e = launch_quantize_rows(x, x_dtype == CONV_BF16, p.M, p.K, ws.pitch, base + ws.x, scale, pl->num_sms, st);
    if (e != cudaSuccess) return launched(e);
    p.x = base + ws.x;
    p.x_pitch = ws.pitch;
    p.x_scale = scale;
    if (int8_use_mid(p)) return launched(launch_int8_mid(p, true, st));
    return launched(launch_int8_gemm(p, pl->num_sms, true, st));
}

conv_status conv_int8_plan_info(const conv_int8_plan* p, int* kernel, int* tile_rows, int* tile_columns, int* splits) {
    if (p == nullptr) return CONV_ERR_INVALID_ARG;
    const bool gemm = int8_use_gemm(p->ip);
    const Int8Tile t = gemm ? int8_pick_tile(p->ip, p->num_sms) : Int8Tile();
    if (kernel) *kernel = gemm ? CONV_INT8_TILES : (int8_use_mid(p->ip) ? CONV_INT8_MID_ROWS : CONV_INT8_FEW_ROWS);
    if (tile_rows) *tile_rows = t.rows;
    if (tile_columns) *tile_columns = t.columns;
    if (splits) *splits = t.splits;
    return CONV_OK;
}

conv_status conv_int8_plan_device_status(const conv_int8_plan* p, void* stream, int* code) {
    if (p == nullptr || code == nullptr) return CONV_ERR_INVALID_ARG;
    *code = 0;
    if (p->device < 0) return CONV_ERR_CUDA;  // host-only plan
    if (p->ip.status == nullptr) {  // no kernel of the plan writes one: clean, once the stream is done
        const conv_status s = check_device(p);
        if (s != CONV_OK) return s;
        return launched(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)));
    }
    return read_status_word(p->device, p->ip.status, stream, code);
}

conv_status conv_int8_plan_destroy(conv_int8_plan* p) {
    if (p != nullptr) release_status_word(p->device, p->status_slot);
    delete p;
    return CONV_OK;
}

conv_status conv_quantize_rows(const void* x, conv_dtype dtype, int M, int K, void* q, float* scale, void* stream) {
    if (x == nullptr || q == nullptr || scale == nullptr || M <= 0 || K <= 0) return CONV_ERR_INVALID_ARG;
    if (dtype != CONV_F32 && dtype != CONV_BF16) return CONV_ERR_INVALID_ARG;
    if (static_cast<long long>(M) * K > (1LL << 40)) return CONV_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(q) || !aligned16(scale)) return CONV_ERR_MISALIGNED;
    int dev = -1, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return CONV_ERR_CUDA;
    }
    return launched(launch_quantize_rows(x, dtype == CONV_BF16, M, K, K, static_cast<int8_t*>(q), scale, sms,
                                         static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
