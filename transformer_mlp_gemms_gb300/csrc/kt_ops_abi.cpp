// kt_ops_abi.cpp -- the extern "C" boundary of the operators around the MLP: argument checks,
// the mixture-of-experts plans, launches.  No call lets a C++ exception out.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <new>

#include "kt_ops_internal.h"

namespace {

kt_status bad(const char* msg) { return kt::report(KT_ERR_INVALID, msg); }

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool known_dtype(int d) { return d == KT_F16 || d == KT_BF16; }
bool known_act(int a) { return a >= KT_ACT_GELU_ERF && a <= KT_ACT_SILU; }

kt_status cuda_failed(const char* what, cudaError_t e) {
    char msg[192];
    std::snprintf(msg, sizeof(msg), "%s: %s", what, cudaGetErrorString(e));
    return kt::report(e == cudaErrorMemoryAllocation ? KT_ERR_NOMEM : KT_ERR_CUDA, msg);
}

// SM count of the current device, which must be an sm_103 one (asked once per device).
constexpr int kMaxDevices = 64;
std::atomic<int> g_sms[kMaxDevices];

kt_status current_device(int* device, int* sms) {
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_failed("cudaGetDevice", e);
    if (dev < 0 || dev >= kMaxDevices) return kt::report(KT_ERR_UNSUPPORTED, "device ordinal beyond the library's table");
    int n = g_sms[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        int major = 0, minor = 0;
        if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess ||
            (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess ||
            (e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
            return cuda_failed("cudaDeviceGetAttribute", e);
        if (major != 10 || minor != 3) return kt::report(KT_ERR_UNSUPPORTED, "this library is built for sm_103a (GB300)");
        if (n > kt::kMaxSms) n = kt::kMaxSms;
        g_sms[dev].store(n, std::memory_order_relaxed);
    }
    *device = dev;
    *sms = n;
    return KT_OK;
}

constexpr unsigned long long kWaitLimitNs = 4000000000ull;  // 4 s: far beyond any legitimate wait
constexpr int64_t kMostStallUs = 10000000;
std::atomic<int64_t> g_linear_stall_us{0};  // kt_linear_i8_debug_stall's limit; 0: off

kt_status done(kt_status s, const char* why) { return kt::report(s, s == KT_OK ? "" : why); }

// What the row operators have in common: sizes, dtype, pitches.
kt_status check_rows(int64_t M, int64_t D, int dtype) {
    if (M < 0 || D < 1) return bad("the row count must not be negative and the row length at least 1");
    if (!known_dtype(dtype)) return bad("unknown dtype");
    if (M > INT32_MAX) return kt::report(KT_ERR_UNSUPPORTED, "more than 2^31 - 1 rows");
    if (D > KT_LAYERNORM_MAX_D) return kt::report(KT_ERR_UNSUPPORTED, "rows longer than KT_LAYERNORM_MAX_D");
    return KT_OK;
}

}  // namespace

struct kt_moe_plan_s {
    kt_moe_options o;
    int device = -1, sms = 0;
    void* workspace = nullptr;
    kt::MoeParams p;
    bool ran = false;
};

namespace {

// Makes a device current, and the former one again at its end.
struct OnDevice {
    int prev = -1, device;
    explicit OnDevice(int d) : device(d) {
        cudaGetDevice(&prev);
        if (prev != device) cudaSetDevice(device);
    }
    ~OnDevice() {
        if (prev >= 0 && prev != device) cudaSetDevice(prev);
    }
    OnDevice(const OnDevice&) = delete;
};

}  // namespace

extern "C" {

kt_status kt_layernorm_forward(int64_t M, int64_t D, kt_dtype dtype, const void* X, int64_t ldx, const void* gamma,
                               const void* beta, float eps, void* Y, int64_t ldy, float* mean, float* rstd,
                               void* stream) {
    kt_status s = check_rows(M, D, dtype);
    if (s != KT_OK) return s;
    if (!(eps >= 0.0f && eps < 3.0e38f)) return bad("eps must be finite and not negative");
    if (ldx < D || ldy < D) return bad("a row pitch is below the row length");
    if ((gamma == nullptr) != (beta == nullptr)) return bad("gamma and beta: both or neither");
    if (M > 0 && (!X || !Y)) return bad("X and Y must be non-NULL");
    if (!aligned(X, 2) || !aligned(Y, 2) || !aligned(gamma, 2) || !aligned(beta, 2) || !aligned(mean, 4) || !aligned(rstd, 4))
        return bad("a pointer is not aligned to its elements");
    if (X == Y && ldx != ldy) return bad("Y may be X only with the same pitch");
    if (M == 0) return done(KT_OK, "");
    int dev, sms;
    if ((s = current_device(&dev, &sms)) != KT_OK) return s;
    const char* why = "";
    kt::LnForward p = {X, gamma, beta, Y, mean, rstd, ldx, ldy, (int)M, (int)D, eps};
    return done(kt::launch_ln_forward(dtype, p, sms, stream, &why), why);
}

size_t kt_layernorm_backward_workspace(int64_t M, int64_t D) {
    if (M < 0 || M > INT32_MAX || D < 1 || D > KT_LAYERNORM_MAX_D) return 0;
    const size_t rows = (size_t)kt::ln_backward_blocks(M, D);
    return (rows ? rows : 1) * 2 * (size_t)D * sizeof(float);
}

kt_status kt_layernorm_backward(int64_t M, int64_t D, kt_dtype dtype, const void* dY, int64_t lddy, const void* X,
                                int64_t ldx, const void* gamma, const float* mean, const float* rstd, void* dX,
                                int64_t lddx, float* dgamma, float* dbeta, void* workspace, size_t workspace_bytes,
                                void* stream) {
    kt_status s = check_rows(M, D, dtype);
    if (s != KT_OK) return s;
    if (lddy < D || ldx < D || lddx < D) return bad("a row pitch is below the row length");
    if ((dgamma == nullptr) != (dbeta == nullptr)) return bad("dgamma and dbeta: both or neither");
    if (M > 0 && (!dY || !X || !mean || !rstd || !dX)) return bad("dY, X, mean, rstd and dX must be non-NULL");
    if (!aligned(dY, 2) || !aligned(X, 2) || !aligned(gamma, 2) || !aligned(dX, 2) || !aligned(mean, 4) ||
        !aligned(rstd, 4) || !aligned(dgamma, 4) || !aligned(dbeta, 4) || !aligned(workspace, 16))
        return bad("a pointer is not aligned to its elements (the workspace: to 16 bytes)");
    if ((dX == dY && lddx != lddy) || (dX == X && lddx != ldx)) return bad("dX may be dY or X only with the same pitch");
    if (dgamma && (!workspace || workspace_bytes < kt_layernorm_backward_workspace(M, D)))
        return bad("the workspace is smaller than kt_layernorm_backward_workspace says");
    if (M == 0 && !dgamma) return done(KT_OK, "");
    int dev, sms;
    if ((s = current_device(&dev, &sms)) != KT_OK) return s;
    const char* why = "";
    kt::LnBackward p = {dY, X, gamma, mean, rstd, dX, dgamma, dbeta, static_cast<float*>(workspace), lddy, ldx, lddx, (int)M, (int)D};
    return done(kt::launch_ln_backward(dtype, p, sms, dev, stream, &why), why);
}

kt_status kt_quantize_rows(int64_t M, int64_t K, kt_dtype dtype, kt_act act, const void* X, int64_t ldx, int8_t* Q,
                           int64_t ldq, float* scale, void* stream) {
    kt_status s = check_rows(M, K, dtype);
    if (s != KT_OK) return s;
    if (!known_act(act)) return bad("unknown activation");
    if (ldx < (act == KT_ACT_GEGLU ? 2 * K : K) || ldq < K) return bad("a row pitch is below the row length");
    if (M > 0 && (!X || !Q || !scale)) return bad("X, Q and scale must be non-NULL");
    if (!aligned(X, 2) || !aligned(scale, 4)) return bad("a pointer is not aligned to its elements");
    if (M == 0) return done(KT_OK, "");
    int dev, sms;
    if ((s = current_device(&dev, &sms)) != KT_OK) return s;
    const char* why = "";
    kt::QuantRows p = {X, Q, scale, ldx, ldq, (int)M, (int)K, (int)act};
    return done(kt::launch_quantize(dtype, p, sms, stream, &why), why);
}

kt_status kt_linear_i8(int64_t M, int64_t N, int64_t K, kt_dtype dtype, const int8_t* Q, int64_t ldq, const int8_t* W,
                       int64_t ldw, const float* scale_x, const float* scale_w, const void* bias, void* Y, int64_t ldy,
                       void* stream) {
    if (M < 0 || N < 1 || K < 1) return bad("M must not be negative, N and K at least 1");
    if (!known_dtype(dtype)) return bad("unknown dtype");
    if (ldq < K || ldw < K || ldy < N) return bad("a row pitch is below the row length");
    if ((M > 0 && (!Q || !scale_x || !Y)) || !W || !scale_w) return bad("Q, W, scale_x, scale_w and Y must be non-NULL");
    if (!aligned(Y, 2) || !aligned(bias, 2) || !aligned(scale_x, 4) || !aligned(scale_w, 4))
        return bad("a pointer is not aligned to its elements");
    if (!aligned(Q, 16) || !aligned(W, 16)) return bad("Q and W must be 16-byte aligned");
    if (K % 16 || ldq % 16 || ldw % 16) return kt::report(KT_ERR_UNSUPPORTED, "K and the pitches of Q and W must be multiples of 16");
    if (M > (1 << 19) || N > (1 << 24) || K >= (1 << 17))
        return kt::report(KT_ERR_UNSUPPORTED, "M above 2^19, N above 2^24, or K at or above 2^17 (the sums' 32 bits)");
    if (M == 0) return done(KT_OK, "");
    kt_status s;
    int dev, sms;
    if ((s = current_device(&dev, &sms)) != KT_OK) return s;
    const char* why = "";
    const unsigned long long stall_ns = 1000ull * (unsigned long long)g_linear_stall_us.load(std::memory_order_relaxed);
    kt::LinearI8 p = {Q,   W,      scale_x, scale_w, bias,    Y,       ldq, ldw, ldy, (int)M, (int)N, (int)K, stall_ns ? stall_ns : kWaitLimitNs,
                      stall_ns};
    return done(kt::launch_linear_i8(dtype, p, sms, dev, stream, &why), why);
}

kt_status kt_linear_i8_status(void* stream) {
    int dev, sms, word = 0;
    kt_status s;
    if ((s = current_device(&dev, &sms)) != KT_OK) return s;
    const char* why = "";
    if ((s = kt::linear_i8_status(stream, &word, &why)) != KT_OK) return kt::report(s, why);
    if (word == 0) return done(KT_OK, "");
    return kt::report(KT_ERR_TIMEOUT, word == kt::DEV_INJECTED_STALL ? "a bounded device wait ran out (injected stall)"
                                                                     : "a bounded device wait ran out");
}

kt_status kt_linear_i8_debug_stall(int enable, int64_t limit_us) {
    if (enable && (limit_us < 1 || limit_us > kMostStallUs)) return bad("limit_us must be in [1, 10 000 000]");
    g_linear_stall_us.store(enable ? limit_us : 0, std::memory_order_relaxed);
    return done(KT_OK, "");
}

kt_status kt_moe_plan(const kt_moe_options* o, kt_moe_plan_t* out) {
    if (!out) return bad("out is NULL");
    *out = nullptr;
    if (!o) return bad("options is NULL");
    if (o->max_tokens < 1 || o->D < 1 || o->F < 1 || o->experts < 1 || o->top_k < 1)
        return bad("max_tokens, D, F, experts and top_k must be positive");
    if (!known_dtype(o->dtype)) return bad("unknown dtype");
    if (!known_act(o->act)) return bad("unknown activation");
    if ((o->bias != 0 && o->bias != 1) || (o->normalize != 0 && o->normalize != 1))
        return bad("bias and normalize must be 0 or 1");
    if (o->top_k > o->experts) return bad("top_k exceeds the number of experts");
    if (o->max_tokens > KT_MOE_MAX_TOKENS || o->experts > KT_MOE_MAX_EXPERTS || o->top_k > KT_MOE_MAX_TOP_K)
        return kt::report(KT_ERR_UNSUPPORTED, "max_tokens, experts or top_k beyond KT_MOE_MAX_*");
    if (o->D % 8 || o->F % 8) return kt::report(KT_ERR_UNSUPPORTED, "D and F must be multiples of 8");
    if (o->D > 65536 || o->F > 65536) return kt::report(KT_ERR_UNSUPPORTED, "D or F above 65536");
    kt_status s;
    int dev, sms;
    if ((s = current_device(&dev, &sms)) != KT_OK) return s;
    kt_moe_plan_s* plan = new (std::nothrow) kt_moe_plan_s;
    if (!plan) return kt::report(KT_ERR_NOMEM, "host allocation failed");
    plan->o = *o;
    plan->device = dev;
    plan->sms = sms;
    const size_t bytes = kt::moe_workspace(o->max_tokens, o->D, o->F, o->top_k);
    cudaError_t e = cudaMalloc(&plan->workspace, bytes);
    // the counters and the error word start at zero, on the device before this returns
    if (e == cudaSuccess) e = cudaMemset(plan->workspace, 0, kt::kMoeControlBytes);
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
    if (e != cudaSuccess) {
        cudaFree(plan->workspace);
        delete plan;
        return cuda_failed("the plan's workspace", e);
    }
    kt::MoeParams& p = plan->p;
    std::memset(&p, 0, sizeof(p));
    p.D = (int)o->D;
    p.F = (int)o->F;
    p.F_up = (int)(o->act == KT_ACT_GEGLU ? 2 * o->F : o->F);
    p.E = (int)o->experts;
    p.top_k = (int)o->top_k;
    p.normalize = o->normalize;
    p.wait_limit_ns = kWaitLimitNs;
    kt::moe_carve(&p, o->max_tokens, plan->workspace);
    *out = plan;
    return done(KT_OK, "");
}

kt_status kt_moe_run(kt_moe_plan_t plan, const kt_moe_tensors* t, void* stream) {
    if (!plan) return bad("plan is NULL");
    if (!t) return bad("tensors is NULL");
    if (t->tokens < 0 || t->tokens > plan->o.max_tokens) return bad("tokens must be between 0 and the plan's max_tokens");
    if (t->tokens == 0) return done(KT_OK, "");
    if (!t->X || !t->W_router || !t->W_up || !t->W_down || !t->Y)
        return bad("X, W_router, W_up, W_down and Y must be non-NULL");
    if (plan->o.bias != (t->b_up != nullptr) || plan->o.bias != (t->b_down != nullptr))
        return bad("b_up and b_down must be given iff the plan has bias = 1");
    if (t->ldx < plan->o.D || t->ldx % 8) return bad("ldx must be at least D and a multiple of 8");
    if (!aligned(t->X, 16) || !aligned(t->W_router, 16) || !aligned(t->W_up, 16) || !aligned(t->W_down, 16) ||
        !aligned(t->b_up, 16) || !aligned(t->b_down, 16) || !aligned(t->R, 16) || !aligned(t->Y, 16) ||
        !aligned(t->ids, 4) || !aligned(t->weights, 4))
        return bad("device pointers must be 16-byte aligned (ids and weights: 4)");
    if (t->Y == t->X && t->ldx != plan->o.D && t->tokens > 1) return bad("Y may be X only where ldx = D, or for a single token");
    int cur = -1;
    cudaError_t e = cudaGetDevice(&cur);
    if (e != cudaSuccess) return cuda_failed("cudaGetDevice", e);
    if (cur != plan->device) return bad("the current device is not the plan's device");
    kt::MoeParams p = plan->p;
    p.X = t->X;
    p.W_router = t->W_router;
    p.W_up = t->W_up;
    p.W_down = t->W_down;
    p.b_up = t->b_up;
    p.b_down = t->b_down;
    p.R = t->R;
    p.Y = t->Y;
    p.ids = t->ids;
    p.weights = t->weights;
    p.ldx = t->ldx;
    p.T = (int)t->tokens;
    plan->ran = true;
    const char* why = "";
    return done(kt::launch_moe(plan->o.act, plan->o.dtype, p, plan->sms, plan->device, stream, &why), why);
}

kt_status kt_moe_status(kt_moe_plan_t plan) {
    if (!plan) return bad("plan is NULL");
    if (!plan->ran) return done(KT_OK, "");
    // the whole device: a captured run may have been replayed on any stream
    const OnDevice on(plan->device);
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_failed("cudaDeviceSynchronize", e);
    int word = 0;
    e = cudaMemcpy(&word, plan->p.error, sizeof(word), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_failed("cudaMemcpy", e);
    if (word == 0) return done(KT_OK, "");
    e = cudaMemset(plan->workspace, 0, kt::kMoeControlBytes);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_failed("clearing the plan's counters", e);
    return kt::report(KT_ERR_TIMEOUT, word == kt::DEV_INJECTED_STALL ? "a device-side wait ran out (injected stall)"
                                                                     : "a device-side wait ran out");
}

kt_status kt_moe_debug_stall(kt_moe_plan_t plan, int enable, int64_t limit_us) {
    if (!plan) return bad("plan is NULL");
    if (enable && (limit_us < 1 || limit_us > kMostStallUs)) return bad("limit_us must be in [1, 10 000 000]");
    plan->p.stall_ns = enable ? 1000ull * (unsigned long long)limit_us : 0;
    plan->p.wait_limit_ns = enable ? plan->p.stall_ns : kWaitLimitNs;
    return done(KT_OK, "");
}

kt_status kt_moe_destroy(kt_moe_plan_t plan) {
    if (!plan) return bad("plan is NULL");
    {
        const OnDevice on(plan->device);
        cudaDeviceSynchronize();
        cudaFree(plan->workspace);
    }
    delete plan;
    return done(KT_OK, "");
}

}  // extern "C"
