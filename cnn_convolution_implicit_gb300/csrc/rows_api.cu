// rows_api.cu -- C ABI of the root-mean-square norm and of dropout (conv_rms_norm_*, conv_dropout in
// include/conv.h): checks, launch configuration and the calls.
#include <atomic>
#include <cmath>
#include <new>

#include "../../include/conv.h"
#include "rows_internal.h"

using namespace convgb;

struct conv_rms_norm_plan {
    RmsParams rp;
    int device;
};

namespace {

template <typename... P>
bool all_aligned16(const P*... ptr) {
    return ((reinterpret_cast<uintptr_t>(ptr) | ...) & 15u) == 0;
}

conv_status check_device(const conv_rms_norm_plan* pl) {
    if (pl->device < 0) return CONV_ERR_CUDA;  // host-only plan
    int cur = -1;
    if (cudaGetDevice(&cur) != cudaSuccess) {
        cudaGetLastError();
        return CONV_ERR_CUDA;
    }
    return cur == pl->device ? CONV_OK : CONV_ERR_INVALID_ARG;
}

// Of the current device.
conv_status sm_count(int& sms) {
    static std::atomic<int> known[64];
    int dev = -1;
    if (cudaGetDevice(&dev) == cudaSuccess) {
        sms = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
        if (sms != 0) return CONV_OK;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) {
            if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
            return CONV_OK;
        }
    }
    cudaGetLastError();
    return CONV_ERR_CUDA;
}

unsigned long long part_bytes(const conv_rms_norm_plan* pl) {
    return pl->rp.parts > 1 ? static_cast<unsigned long long>(pl->rp.parts) * pl->rp.C * sizeof(float) : 0;
}

conv_status launched(cudaError_t e) {
    if (e == cudaSuccess) return CONV_OK;
    cudaGetLastError();
    return CONV_ERR_CUDA;
}

conv_status forward(conv_rms_norm_plan* pl, const void* x, const void* residual, const float* gamma, void* y, void* q,
                    float* q_scale, void* h, float* rstd, void* stream) {
    if (pl == nullptr || x == nullptr || (h != nullptr && residual == nullptr)) return CONV_ERR_INVALID_ARG;
    if (!all_aligned16(x, residual, gamma, y, q, q_scale, h, rstd)) return CONV_ERR_MISALIGNED;
    const conv_status s = check_device(pl);
    if (s != CONV_OK) return s;
    RmsParams p = pl->rp;
    p.x = x;
    p.r = residual;
    p.gamma = gamma;
    p.y = y;
    p.q = static_cast<int8_t*>(q);
    p.scale = q_scale;
    p.h = h;
    p.rstd = rstd;
    return launched(launch_rms_forward(p, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

conv_status conv_rms_norm_plan_create(conv_rms_norm_plan** out, int M, int C, float eps, conv_dtype dtype) {
    if (out == nullptr) return CONV_ERR_INVALID_ARG;
    *out = nullptr;
    if (M <= 0 || C <= 0 || !(eps >= 0.0f) || !std::isfinite(eps)) return CONV_ERR_INVALID_ARG;
    if (dtype != CONV_F32 && dtype != CONV_BF16) return CONV_ERR_INVALID_ARG;
    if (C > (1 << 20) || M >= (1 << 30) || static_cast<long long>(M) * C > (1LL << 40)) return CONV_ERR_UNSUPPORTED;
    conv_rms_norm_plan* pl = new (std::nothrow) conv_rms_norm_plan();
    if (pl == nullptr) return CONV_ERR_NO_MEMORY;
    int ndev = 0, num_sms = 152;
    unsigned* status = nullptr;
    if (cudaGetDeviceCount(&ndev) != cudaSuccess || ndev == 0) {
        cudaGetLastError();
        pl->device = -1;
    } else if (cudaGetDevice(&pl->device) != cudaSuccess ||
               cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, pl->device) != cudaSuccess ||
               device_status_word(&status) != cudaSuccess) {
        cudaGetLastError();
        delete pl;
        return CONV_ERR_CUDA;
    }
    RmsParams& p = pl->rp;
    p = RmsParams();
    p.M = M;
    p.C = C;
    p.eps = eps;
    p.bf16 = dtype == CONV_BF16;
    p.status = status;
    rms_plan_backward(p, num_sms);
    *out = pl;
    return CONV_OK;
}

conv_status conv_rms_norm_workspace(const conv_rms_norm_plan* p, unsigned long long* backward) {
    if (p == nullptr) return CONV_ERR_INVALID_ARG;
    if (backward != nullptr) *backward = part_bytes(p);
    return CONV_OK;
}

conv_status conv_rms_norm_forward(conv_rms_norm_plan* p, const void* x, const void* residual, const float* gamma,
                                  void* y, void* h, float* rstd, void* stream) {
    if (y == nullptr) return CONV_ERR_INVALID_ARG;
    return forward(p, x, residual, gamma, y, nullptr, nullptr, h, rstd, stream);
}

conv_status conv_rms_norm_forward_int8(conv_rms_norm_plan* p, const void* x, const void* residual, const float* gamma,
                                       void* q, float* q_scale, void* h, float* rstd, void* stream) {
    if (q == nullptr || q_scale == nullptr) return CONV_ERR_INVALID_ARG;
    return forward(p, x, residual, gamma, nullptr, q, q_scale, h, rstd, stream);
}

conv_status conv_rms_norm_backward(conv_rms_norm_plan* pl, const void* dy, const void* h, const float* rstd,
                                   const float* gamma, const void* dh, void* dx, float* dgamma, void* workspace,
                                   void* stream) {
    if (pl == nullptr || dy == nullptr || h == nullptr || rstd == nullptr || dx == nullptr ||
        (dgamma != nullptr && workspace == nullptr && part_bytes(pl) != 0))
        return CONV_ERR_INVALID_ARG;
    if (!all_aligned16(dy, h, rstd, gamma, dh, dx, dgamma, workspace)) return CONV_ERR_MISALIGNED;
    const conv_status s = check_device(pl);
    if (s != CONV_OK) return s;
    RmsParams p = pl->rp;
    p.x = dy;
    p.r = dh;
    p.h_in = h;
    p.gamma = gamma;
    p.y = dx;
    p.rstd = const_cast<float*>(rstd);
    p.dgamma = dgamma;
    p.part = static_cast<float*>(workspace);
    return launched(launch_rms_backward(p, static_cast<cudaStream_t>(stream)));
}

conv_status conv_rms_norm_plan_destroy(conv_rms_norm_plan* p) {
    delete p;
    return CONV_OK;
}

conv_status conv_dropout(const void* x, const void* residual, conv_dtype dtype, unsigned long long n, double p,
                         const unsigned long long* state, void* y, void* stream) {
    if (x == nullptr || state == nullptr || y == nullptr || n == 0 || !(p >= 0.0 && p <= 1.0)) return CONV_ERR_INVALID_ARG;
    if (dtype != CONV_F32 && dtype != CONV_BF16) return CONV_ERR_INVALID_ARG;
    if (n > (1ULL << 40)) return CONV_ERR_UNSUPPORTED;
    if (!all_aligned16(x, residual, y) || (reinterpret_cast<uintptr_t>(state) & 7u) != 0) return CONV_ERR_MISALIGNED;
    int sms = 0;
    const conv_status s = sm_count(sms);
    if (s != CONV_OK) return s;
    DropoutParams d = {};
    d.x = x;
    d.r = residual;
    d.y = y;
    d.n = n;
    d.state = state;
    const double t = std::nearbyint(p * 4294967296.0);
    d.none_left = t >= 4294967296.0;
    d.threshold = d.none_left ? 0u : static_cast<uint32_t>(t);
    d.scale = d.none_left ? 0.0f : static_cast<float>(1.0 / (1.0 - p));
    d.bf16 = dtype == CONV_BF16;
    return launched(launch_dropout(d, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
