// norm_api.cu -- C ABI of the group norm (conv_group_norm_* in include/conv.h):
// shape checks, launch configuration and the calls.
#include <cmath>
#include <new>

#include "../../include/conv.h"
#include "norm_internal.h"

using namespace convgb;

struct conv_group_norm_plan {
    NormParams np[3];  // by NormMode
    int device;
    int num_sms;
};

namespace {

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

// Workspace: per-channel partials, then (a, b) per group, then statistics nobody asked for.
void carve_workspace(NormParams& p, void* workspace) {
    if (p.chunk != 0 && p.dy == nullptr) return;  // resident forward passes need none
    p.part = static_cast<float2*>(workspace);
    p.ab = p.part + norm_part_entries(p);
    if (p.mean == nullptr && (!p.two_pass || p.joined)) {
        p.mean = reinterpret_cast<float*>(p.ab + norm_ab_entries(p));
        p.rstd = p.mean + static_cast<size_t>(p.N) * p.G;
    }
}

size_t workspace_bytes(const conv_group_norm_plan* pl, int mode) {
    const NormParams& p = pl->np[mode];
    return p.chunk != 0 && mode != kNormBackward ? 0 : norm_workspace_bytes(p);  // resident forward passes need none
}

conv_status check_device(const conv_group_norm_plan* pl) {
    if (pl->device < 0) return CONV_ERR_CUDA;  // host-only plan
    int cur = -1;
    if (cudaGetDevice(&cur) != cudaSuccess) {
        cudaGetLastError();
        return CONV_ERR_CUDA;
    }
    return cur == pl->device ? CONV_OK : CONV_ERR_INVALID_ARG;
}

conv_status forward(conv_group_norm_plan* pl, const void* x, const float* gamma, const float* beta, void* y, void* q,
                    float* q_scale, float* stats, void* workspace, void* stream) {
    for (const void* ptr : {x, static_cast<const void*>(gamma), static_cast<const void*>(beta),
                            static_cast<const void*>(y), static_cast<const void*>(q),
                            static_cast<const void*>(q_scale), static_cast<const void*>(stats),
                            static_cast<const void*>(workspace)})
        if (ptr != nullptr && !aligned16(ptr)) return CONV_ERR_MISALIGNED;
    const conv_status s = check_device(pl);
    if (s != CONV_OK) return s;
    NormParams p = pl->np[q != nullptr ? kNormInt8 : kNormForward];
    p.x = x;
    p.gamma = gamma;
    p.beta = beta;
    p.y = y;
    p.q = static_cast<int8_t*>(q);
    p.scale = q_scale;
    p.mean = stats;
    p.rstd = stats ? stats + static_cast<size_t>(p.N) * p.G : nullptr;
    carve_workspace(p, workspace);
    if (launch_norm_forward(p, pl->num_sms, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return CONV_ERR_CUDA;
    }
    return CONV_OK;
}

}  // namespace

extern "C" {

conv_status conv_group_norm_plan_create(conv_group_norm_plan** out, int N, int C, int H, int W, int groups, float eps,
                                        conv_dtype dtype, conv_act act) {
    if (out == nullptr) return CONV_ERR_INVALID_ARG;
    *out = nullptr;
    if (N <= 0 || C <= 0 || H <= 0 || W <= 0 || groups <= 0 || C % groups != 0) return CONV_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return CONV_ERR_INVALID_ARG;
    if (dtype != CONV_F32 && dtype != CONV_BF16) return CONV_ERR_INVALID_ARG;
    if (act != CONV_ACT_NONE && act != CONV_ACT_RELU && act != CONV_ACT_SILU) return CONV_ERR_INVALID_ARG;
    const long long P = static_cast<long long>(H) * W;
    if (P > (1LL << 30) || static_cast<long long>(N) * groups > (1LL << 24) ||
        static_cast<double>(N) * static_cast<double>(P) * C > static_cast<double>(1LL << 40))
        return CONV_ERR_UNSUPPORTED;

    conv_group_norm_plan* pl = new (std::nothrow) conv_group_norm_plan();
    if (pl == nullptr) return CONV_ERR_NO_MEMORY;
    int ndev = 0, smem_optin = 232448;
    if (cudaGetDeviceCount(&ndev) != cudaSuccess || ndev == 0) {
        cudaGetLastError();
        pl->device = -1;
        pl->num_sms = 152;
    } else if (cudaGetDevice(&pl->device) != cudaSuccess ||
               cudaDeviceGetAttribute(&pl->num_sms, cudaDevAttrMultiProcessorCount, pl->device) != cudaSuccess ||
               cudaDeviceGetAttribute(&smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, pl->device) !=
                   cudaSuccess) {
        cudaGetLastError();
        delete pl;
        return CONV_ERR_CUDA;
    }
    NormParams p = NormParams();
    p.N = N;
    p.P = static_cast<int>(P);
    p.C = C;
    p.G = groups;
    p.cpg = C / groups;
    p.eps = eps;
    p.act = act;
    p.bf16 = dtype == CONV_BF16;
    p.smem_optin = smem_optin;
    p.vec = p.bf16 ? 8 : 4;
    while (C % p.vec != 0) p.vec /= 2;
    // By channel, where no other form fits: about eight CTAs an SM, at least four pixels a thread.
    const int vecs = C / p.vec, cv = vecs < kNormThreads ? vecs : kNormThreads;
    const long long blocks = static_cast<long long>(N) * ((vecs + cv - 1) / cv);
    const long long least = 4LL * (kNormThreads / cv);
    long long splits = (8LL * pl->num_sms + blocks - 1) / blocks;
    if (splits > P / least) splits = P / least;
    p.splits = static_cast<int>(splits < 1 ? 1 : splits);
    p.pix_base = p.P / p.splits;
    p.pix_more = p.P % p.splits;
    for (int mode = 0; mode < 3; ++mode) {
        NormParams& m = pl->np[mode];
        m = p;
        NormParams two = p;
        norm_pick_resident(m, mode, pl->num_sms);
        norm_pick_two_pass(two, mode, pl->num_sms);
        int at_a_time = 0;
        if (m.chunk != 0)
            at_a_time = pl->device >= 0 ? norm_resident_at_a_time(m, mode, pl->num_sms) : 2 * pl->num_sms / m.splits;
        if (at_a_time == 0 || (two.two_pass && !norm_resident_pays(m, mode, at_a_time, pl->num_sms))) m = two;
    }
    *out = pl;
    return CONV_OK;
}

conv_status conv_group_norm_workspace(const conv_group_norm_plan* p, unsigned long long* forward,
                                      unsigned long long* forward_int8, unsigned long long* backward) {
    if (p == nullptr) return CONV_ERR_INVALID_ARG;
    unsigned long long* to[3] = {forward, forward_int8, backward};
    for (int mode = 0; mode < 3; ++mode)
        if (to[mode] != nullptr) *to[mode] = workspace_bytes(p, mode);
    return CONV_OK;
}

conv_status conv_group_norm_forward(conv_group_norm_plan* p, const void* x, const float* gamma, const float* beta,
                                    void* y, float* stats, void* workspace, void* stream) {
    if (p == nullptr || x == nullptr || y == nullptr || (workspace == nullptr && workspace_bytes(p, kNormForward) != 0))
        return CONV_ERR_INVALID_ARG;
    return forward(p, x, gamma, beta, y, nullptr, nullptr, stats, workspace, stream);
}

conv_status conv_group_norm_forward_int8(conv_group_norm_plan* p, const void* x, const float* gamma,
                                         const float* beta, void* q, float* q_scale, float* stats, void* workspace,
                                         void* stream) {
    if (p == nullptr || x == nullptr || q == nullptr || q_scale == nullptr ||
        (workspace == nullptr && workspace_bytes(p, kNormInt8) != 0))
        return CONV_ERR_INVALID_ARG;
    return forward(p, x, gamma, beta, nullptr, q, q_scale, stats, workspace, stream);
}

conv_status conv_group_norm_backward(conv_group_norm_plan* pl, const void* dy, const void* x, const float* stats,
                                     const float* gamma, const float* beta, void* dx, float* dgamma, float* dbeta,
                                     void* workspace, void* stream) {
    if (pl == nullptr || dy == nullptr || x == nullptr || stats == nullptr || dx == nullptr || workspace == nullptr ||
        (dgamma == nullptr) != (dbeta == nullptr))
        return CONV_ERR_INVALID_ARG;
    for (const void* ptr : {dy, x, static_cast<const void*>(stats), static_cast<const void*>(gamma),
                            static_cast<const void*>(beta), static_cast<const void*>(dx),
                            static_cast<const void*>(dgamma), static_cast<const void*>(dbeta),
                            static_cast<const void*>(workspace)})
        if (ptr != nullptr && !aligned16(ptr)) return CONV_ERR_MISALIGNED;
    const conv_status s = check_device(pl);
    if (s != CONV_OK) return s;
    NormParams p = pl->np[kNormBackward];
    p.x = x;
    p.dy = dy;
    p.gamma = gamma;
    p.beta = beta;
    p.y = dx;
    p.dgamma = dgamma;
    p.dbeta = dbeta;
    p.mean = const_cast<float*>(stats);
    p.rstd = p.mean + static_cast<size_t>(p.N) * p.G;
    carve_workspace(p, workspace);
    if (launch_norm_backward(p, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return CONV_ERR_CUDA;
    }
    return CONV_OK;
}

conv_status conv_group_norm_plan_destroy(conv_group_norm_plan* p) {
    delete p;
    return CONV_OK;
}

}  // extern "C"
