// linear_api.cu -- C ABI of the linear layer (conv_linear_* in include/conv.h): checks, launch
// configuration and the calls.
#include <new>

#include "../../include/conv.h"
#include "linear_internal.h"
#include "status_slots.h"

using namespace convgb;

struct conv_linear_plan {
    int M, N, K, act;
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

conv_status launched(cudaError_t e) {
    if (e == cudaSuccess) return CONV_OK;
    cudaGetLastError();
    return CONV_ERR_CUDA;
}

size_t up(size_t v, size_t to) { return (v + to - 1) / to * to; }

size_t backward_bytes(const conv_linear_plan* pl) {
    return pl->act != CONV_ACT_NONE ? up(static_cast<size_t>(pl->M) * pl->N * 2, 256) : 0;
}

}  // namespace

extern "C" {

conv_status conv_linear_plan_create(conv_linear_plan** out, int M, int N, int K, conv_act act) {
    if (out == nullptr) return CONV_ERR_INVALID_ARG;
    *out = nullptr;
    if (M <= 0 || N <= 0 || K <= 0) return CONV_ERR_INVALID_ARG;
    if (act != CONV_ACT_NONE && act != CONV_ACT_RELU && act != CONV_ACT_SILU) return CONV_ERR_INVALID_ARG;
    const long long most = 1LL << 40;
    const int side = 1 << 30;
    if (M >= side || N >= side || K >= side || static_cast<long long>(M) * K > most ||
        static_cast<long long>(N) * K > most || static_cast<long long>(M) * N > most)
        return CONV_ERR_UNSUPPORTED;
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
               cudaDeviceGetAttribute(&pl->num_sms, cudaDevAttrMultiProcessorCount, pl->device) != cudaSuccess) {
        cudaGetLastError();
        delete pl;
        return CONV_ERR_CUDA;
    }
    *out = pl;
    return CONV_OK;
}

conv_status conv_linear_workspace(const conv_linear_plan* p, unsigned long long* forward, unsigned long long* backward) {
    if (p == nullptr) return CONV_ERR_INVALID_ARG;
    if (forward != nullptr) *forward = 0;
    if (backward != nullptr) *backward = backward_bytes(p);
    return CONV_OK;
}

conv_status conv_linear_forward(conv_linear_plan* pl, const void* x, const void* w, const float* bias,
                                const void* residual, void* y, void* z, void* workspace, void* stream) {
    if (pl == nullptr || x == nullptr || w == nullptr || y == nullptr) return CONV_ERR_INVALID_ARG;
    if (!all_aligned16(x, w, bias, residual, y, z, workspace)) return CONV_ERR_MISALIGNED;
    const conv_status s = check_device(pl);
    if (s != CONV_OK) return s;
    ProductParams p = {};
    p.M = pl->M;
    p.N = pl->N;
    p.K = pl->K;
    p.a = static_cast<const __nv_bfloat16*>(x);
    p.b = static_cast<const __nv_bfloat16*>(w);
    p.a_m = p.b_n = p.K;
    p.a_k = p.b_k = 1;
    p.bias = bias;
    p.r = static_cast<const __nv_bfloat16*>(residual);
    p.y = static_cast<__nv_bfloat16*>(y);
    p.z = static_cast<__nv_bfloat16*>(z);
    p.act = pl->act;
    return launched(launch_product(p, static_cast<cudaStream_t>(stream)));
}

conv_status conv_linear_backward(conv_linear_plan* pl, const void* dy, const void* x, const void* w, const void* z,
                                 void* dx, void* dw, float* dbias, void* workspace, void* stream) {
    if (pl == nullptr || dy == nullptr || (dx == nullptr && dw == nullptr && dbias == nullptr) ||
        (dx != nullptr && w == nullptr) || (dw != nullptr && x == nullptr) || (pl->act != CONV_ACT_NONE && z == nullptr) ||
        (workspace == nullptr && backward_bytes(pl) != 0))
        return CONV_ERR_INVALID_ARG;
    if (!all_aligned16(dy, x, w, z, dx, dw, dbias, workspace)) return CONV_ERR_MISALIGNED;
    const conv_status s = check_device(pl);
    if (s != CONV_OK) return s;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const __nv_bfloat16* u = static_cast<const __nv_bfloat16*>(dy);
    cudaError_t e = cudaSuccess;
    if (pl->act != CONV_ACT_NONE || dbias != nullptr) {
        LinearGradParams g = {};
        g.M = pl->M;
        g.N = pl->N;
        g.dy = u;
        g.z = static_cast<const __nv_bfloat16*>(z);
        if (pl->act != CONV_ACT_NONE) u = g.u = static_cast<__nv_bfloat16*>(workspace);
        g.dbias = dbias;
        g.act = pl->act;
        e = launch_linear_grad(g, st);
    }
    ProductParams p = {};
    if (e == cudaSuccess && dx != nullptr) {
        p.M = pl->M;
        p.N = pl->K;
        p.K = pl->N;
        p.a = u;
        p.a_m = pl->N;
        p.a_k = 1;
        p.b = static_cast<const __nv_bfloat16*>(w);
        p.b_n = 1;
        p.b_k = pl->K;
        p.y = static_cast<__nv_bfloat16*>(dx);
        e = launch_product(p, st);
    }
    if (e == cudaSuccess && dw != nullptr) {
        p.M = pl->N;
        p.N = pl->K;
        p.K = pl->M;
        p.a = u;
        p.a_m = 1;
        p.a_k = pl->N;
        p.b = static_cast<const __nv_bfloat16*>(x);
        p.b_n = 1;
        p.b_k = pl->K;
        p.y = static_cast<__nv_bfloat16*>(dw);
        e = launch_product(p, st);
    }
    return launched(e);
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
