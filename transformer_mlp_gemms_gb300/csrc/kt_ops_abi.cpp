// kt_ops_abi.cpp -- the extern "C" boundary of the operators around the MLP: argument checks,
// the mixture-of-experts plans, launches.  No call lets a C++ exception out.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <new>
#include <vector>

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
std::atomic<int64_t> g_matmul_stall_us{0};  // kt_matmul_debug_stall's

kt_status done(kt_status s, const char* why) { return kt::report(s, s == KT_OK ? "" : why); }

// What the row operators have in common: sizes, dtype, pitches.
kt_status check_rows(int64_t M, int64_t D, int dtype) {
    if (M < 0 || D < 1) return bad("the row count must not be negative and the row length at least 1");
    if (!known_dtype(dtype)) return bad("unknown dtype");
    if (M > INT32_MAX) return kt::report(KT_ERR_UNSUPPORTED, "more than 2^31 - 1 rows");
    if (D > KT_LAYERNORM_MAX_D) return kt::report(KT_ERR_UNSUPPORTED, "rows longer than KT_LAYERNORM_MAX_D");
    return KT_OK;
}

// The products of kt_matmul.cu: sizes, and what a tensor copy needs of a matrix.
kt_status check_product(int64_t M, int64_t D, int64_t F, int dtype) {
    if (M < 0 || D < 1 || F < 1) return bad("the row count must not be negative and the other sizes at least 1");
    if (!known_dtype(dtype)) return bad("unknown dtype");
    if (D % 8 || F % 8) return kt::report(KT_ERR_UNSUPPORTED, "row lengths must be multiples of 8");
    if (M > INT32_MAX / 2 || D > (1 << 24) || F > (1 << 24)) return kt::report(KT_ERR_UNSUPPORTED, "M above 2^30 or a row length above 2^24");
    return KT_OK;
}
kt_status check_matrix(const void* p, int64_t ld, int64_t cols) {
    if (!aligned(p, 16)) return bad("device pointers must be 16-byte aligned");
    if (ld < cols) return bad("a row pitch is below the row length");
    if (ld % 8) return kt::report(KT_ERR_UNSUPPORTED, "row pitches must be multiples of 8");
    if (ld > (int64_t)1 << 38) return kt::report(KT_ERR_UNSUPPORTED, "a row pitch above 2^38");
    return KT_OK;
}
kt::Matmul product(int64_t M, int64_t N, int64_t K) {
    kt::Matmul a = {};
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.stall_ns = 1000ull * (unsigned long long)g_matmul_stall_us.load(std::memory_order_relaxed);
    a.wait_limit_ns = a.stall_ns ? a.stall_ns : kWaitLimitNs;
    return a;
}
// dX = dP . W and dW = dP^T . X, for dP [M][N], W [N][K], X [M][K].  scratch: as launch_gradients has it.
kt_status gradients(int64_t M, int64_t N, int64_t K, int dtype, const void* dP, int64_t lddp, const void* X, int64_t ldx, const void* W,
                    void* dX, int64_t lddx, void* dW, void* scratch, bool zeroed, int sms, int device, void* stream) {
    kt::Matmul a[2];
    int count = 0;
    if (dW) {
        kt::Matmul& w = a[count++] = product(N, K, M);
        w.A = dP;
        w.lda = lddp;
        w.a_mn = true;
        w.B = X;
        w.ldb = ldx;
        w.b_mn = true;
        w.C = dW;
        w.ldc = K;
    }
    if (dX) {
        kt::Matmul& x = a[count++] = product(M, K, N);
        x.A = dP;
        x.lda = lddp;
        x.B = W;
        x.ldb = K;
        x.b_mn = true;
        x.C = dX;
        x.ldc = lddx;
    }
    if (!count) return done(KT_OK, "");
    if (count == 2 && a[1].K > a[0].K) std::swap(a[0], a[1]);
    const char* why = "";
    return done(kt::launch_gradients(dtype, a, count, scratch, zeroed, sms, device, stream, &why), why);
}
kt_status zeros(void* p, size_t bytes, void* stream) {
    if (!p || !bytes) return KT_OK;
    const cudaError_t e = cudaMemsetAsync(p, 0, bytes, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KT_OK : cuda_failed("cudaMemsetAsync", e);
}
// The pitch of dP in the workspace: whole 128-byte lines, as a product's copies of 64 columns take longer
// where rows start between lines (1.7 % of the gradients of 729 x 1152 x 2 4304).
int64_t dp_pitch(int64_t F) { return (2 * F + 63) / 64 * 64; }
size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
const size_t kScratch = kt::kGradientsFlags + kt::gradients_partials();  // of launch_gradients
int epilogue_of(int act) { return kt::up_epilogue(act); }

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

kt_status kt_glu_forward(int64_t M, int64_t D, int64_t F, kt_dtype dtype, kt_act act, const void* X, int64_t ldx,
                         const void* W, const void* bias, void* H, int64_t ldh, void* P, int64_t ldp, void* stream) {
    kt_status s = check_product(M, D, F, dtype);
    if (s != KT_OK) return s;
    if (!known_act(act) || act == KT_ACT_GEGLU) return bad("unknown activation of the gate");
    if ((M > 0 && (!X || !H)) || !W) return bad("X, W and H must be non-NULL");
    if ((s = check_matrix(X, ldx, D)) != KT_OK || (s = check_matrix(W, D, D)) != KT_OK || (s = check_matrix(H, ldh, F)) != KT_OK) return s;
    if (P && (s = check_matrix(P, ldp, 2 * F)) != KT_OK) return s;
    if (!aligned(bias, 16)) return bad("device pointers must be 16-byte aligned");
    if (M == 0) return done(KT_OK, "");
    int dev, sms;
    if ((s = current_device(&dev, &sms)) != KT_OK) return s;
    kt::Matmul a = product(M, F, D);
    a.gated = true;
    a.act = epilogue_of(act);
    a.A = X;
    a.lda = ldx;
    a.B = W;
    a.ldb = D;
    a.bias = bias;
    a.C = H;
    a.ldc = ldh;
    a.P = P;
    a.ldp = ldp;
    const char* why = "";
    return done(kt::launch_matmul(dtype, a, sms, dev, stream, &why), why);
}

size_t kt_glu_backward_workspace(int64_t M, int64_t D, int64_t F) {
    if (M < 0 || M > INT32_MAX / 2 || D < 8 || D % 8 || D > (1 << 24) || F < 8 || F % 8 || F > (1 << 24)) return 0;
    return up256((size_t)(M ? M : 1) * 2 * (size_t)dp_pitch(F)) + up256((size_t)kt::column_sum_rows(M, F) * 2 * (size_t)F * sizeof(float)) + kScratch;
}

kt_status kt_glu_backward(int64_t M, int64_t D, int64_t F, kt_dtype dtype, kt_act act, const void* dH, int64_t lddh,
                          const void* P, int64_t ldp, const void* X, int64_t ldx, const void* W, void* dX, int64_t lddx,
                          void* dW, float* db, void* workspace, size_t workspace_bytes, void* stream) {
    kt_status s = check_product(M, D, F, dtype);
    if (s != KT_OK) return s;
    if (!known_act(act) || act == KT_ACT_GEGLU) return bad("unknown activation of the gate");
    if ((M > 0 && (!dH || !P || !X)) || !W) return bad("dH, P, X and W must be non-NULL");
    if ((s = check_matrix(dH, lddh, F)) != KT_OK || (s = check_matrix(P, ldp, 2 * F)) != KT_OK ||
        (s = check_matrix(X, ldx, D)) != KT_OK || (s = check_matrix(W, D, D)) != KT_OK || (s = check_matrix(dW, D, D)) != KT_OK)
        return s;
    if (dX && (s = check_matrix(dX, lddx, D)) != KT_OK) return s;
    if (!aligned(db, 4) || !aligned(workspace, 16)) return bad("db must be aligned to its elements and the workspace to 16 bytes");
    if (!workspace || workspace_bytes < kt_glu_backward_workspace(M, D, F))
        return bad("the workspace is smaller than kt_glu_backward_workspace says");
    int dev, sms;
    if ((s = current_device(&dev, &sms)) != KT_OK) return s;
    if (M == 0) {
        if ((s = zeros(dW, (size_t)4 * F * D, stream)) != KT_OK || (s = zeros(db, (size_t)8 * F, stream)) != KT_OK) return s;
        return done(KT_OK, "");
    }
    char* const sums = static_cast<char*>(workspace) + up256((size_t)M * 2 * (size_t)dp_pitch(F));
    char* const scratch = sums + up256((size_t)kt::column_sum_rows(M, F) * 2 * (size_t)F * sizeof(float));
    const char* why = "";
    kt::GluBackward g = {};
    g.dH = dH;
    g.lddh = lddh;
    g.P = P;
    g.ldp = ldp;
    g.dP = workspace;
    g.lddp = dp_pitch(F);
    g.partials = db ? reinterpret_cast<float*>(sums) : nullptr;
    g.db = db;
    g.zero = reinterpret_cast<int*>(scratch);
    g.M = (int)M;
    g.F = (int)F;
    g.act = epilogue_of(act);
    if ((s = kt::launch_glu_backward(dtype, g, stream, &why)) != KT_OK) return kt::report(s, why);
    return gradients(M, 2 * F, D, dtype, workspace, g.lddp, X, ldx, W, dX, lddx, dW, scratch, true, sms, dev, stream);
}

kt_status kt_linear_forward(int64_t M, int64_t N, int64_t K, kt_dtype dtype, const void* X, int64_t ldx, const void* W,
                            const void* bias, void* Y, int64_t ldy, void* stream) {
    kt_status s = check_product(M, K, N, dtype);
    if (s != KT_OK) return s;
    if ((M > 0 && (!X || !Y)) || !W) return bad("X, W and Y must be non-NULL");
    if ((s = check_matrix(X, ldx, K)) != KT_OK || (s = check_matrix(W, K, K)) != KT_OK || (s = check_matrix(Y, ldy, N)) != KT_OK) return s;
    if (!aligned(bias, 16)) return bad("device pointers must be 16-byte aligned");
    if (M == 0) return done(KT_OK, "");
    int dev, sms;
    if ((s = current_device(&dev, &sms)) != KT_OK) return s;
    kt::Matmul a = product(M, N, K);
    a.A = X;
    a.lda = ldx;
    a.B = W;
    a.ldb = K;
    a.bias = bias;
    a.C = Y;
    a.ldc = ldy;
    const char* why = "";
    return done(kt::launch_matmul(dtype, a, sms, dev, stream, &why), why);
}

size_t kt_linear_backward_workspace(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || M > INT32_MAX / 2 || N < 8 || N % 8 || N > (1 << 24) || K < 8 || K % 8 || K > (1 << 24)) return 0;
    return up256((size_t)kt::column_sum_rows(M, N) * (size_t)N * sizeof(float)) + kScratch;
}

kt_status kt_linear_backward(int64_t M, int64_t N, int64_t K, kt_dtype dtype, const void* dY, int64_t lddy, const void* X,
                             int64_t ldx, const void* W, void* dX, int64_t lddx, void* dW, float* db, void* workspace,
                             size_t workspace_bytes, void* stream) {
    kt_status s = check_product(M, K, N, dtype);
    if (s != KT_OK) return s;
    if ((M > 0 && (!dY || !X)) || !W) return bad("dY, X and W must be non-NULL");
    if ((s = check_matrix(dY, lddy, N)) != KT_OK || (s = check_matrix(X, ldx, K)) != KT_OK || (s = check_matrix(W, K, K)) != KT_OK ||
        (s = check_matrix(dW, K, K)) != KT_OK)
        return s;
    if (dX && (s = check_matrix(dX, lddx, K)) != KT_OK) return s;
    if (!aligned(db, 4) || !aligned(workspace, 16)) return bad("db must be aligned to its elements and the workspace to 16 bytes");
    if (!workspace || workspace_bytes < kt_linear_backward_workspace(M, N, K))
        return bad("the workspace is smaller than kt_linear_backward_workspace says");
    int dev, sms;
    if ((s = current_device(&dev, &sms)) != KT_OK) return s;
    if (M == 0) {
        if ((s = zeros(dW, (size_t)2 * N * K, stream)) != KT_OK || (s = zeros(db, (size_t)4 * N, stream)) != KT_OK) return s;
        return done(KT_OK, "");
    }
    char* const scratch = static_cast<char*>(workspace) + up256((size_t)kt::column_sum_rows(M, N) * (size_t)N * sizeof(float));
    const char* why = "";
    if (db) {
        kt::GluBackward g = {};
        g.dH = dY;
        g.lddh = lddy;
        g.partials = static_cast<float*>(workspace);
        g.db = db;
        g.zero = reinterpret_cast<int*>(scratch);
        g.M = (int)M;
        g.F = (int)N;
        if ((s = kt::launch_glu_backward(dtype, g, stream, &why)) != KT_OK) return kt::report(s, why);
    }
    return gradients(M, N, K, dtype, dY, lddy, X, ldx, W, dX, lddx, dW, scratch, db != nullptr, sms, dev, stream);
}

kt_status kt_adamw(int64_t count, const kt_adamw_tensor* tensors, const kt_adamw_options* o, void* stream) {
    if (count < 0 || count > INT32_MAX || (count > 0 && !tensors) || !o) return bad("a negative count, or no tensors or options");
    auto known = [](int d) { return known_dtype(d) || d == KT_F32; };
    if (!known(o->param_dtype) || !known(o->grad_dtype)) return bad("unknown dtype");
    if (o->state_bits != 8 && o->state_bits != 32) return bad("state_bits must be 8 or 32");
    auto beta = [](double b) { return b >= 0.0 && b < 1.0; };
    auto size = [](double x) { return x >= 0.0 && x < 3.0e38; };
    if (!beta(o->beta1) || !beta(o->beta2)) return bad("beta1 and beta2 must be in [0, 1)");
    if (!size(o->lr) || !size(o->eps)) return bad("lr and eps must be finite and not negative");
    if (!o->step_device && o->step < 1) return bad("step must be at least 1");
    if (!aligned(o->step_device, 8) || !aligned(o->grad_scale, 4)) return bad("a pointer is not aligned to its elements");
    const size_t pb = o->param_dtype == KT_F32 ? 4 : 2, gb = o->grad_dtype == KT_F32 ? 4 : 2, sb = o->state_bits == 8 ? 1 : 4;
    kt::AdamwEntry few[64];
    // the addresses that the call writes to, each in the first free place from its own on
    const void* few_written[512] = {};
    size_t places = 512;
    std::vector<kt::AdamwEntry> many;
    std::vector<const void*> many_written;
    kt::AdamwEntry* e = few;
    const void** written = few_written;
    if (count > 64) {
        try {
            many.resize((size_t)count);
            while (places < 6 * (size_t)count) places *= 2;
            many_written.resize(places);
        } catch (...) {
            return kt::report(KT_ERR_NOMEM, "host allocation failed");
        }
        e = many.data();
        written = many_written.data();
    }
    int live = 0;
    for (int64_t i = 0; i < count; ++i) {
        const kt_adamw_tensor& t = tensors[i];
        if (t.n < 0 || t.n > (int64_t)1 << 48) return bad("a tensor's length is negative or above 2^48");
        if (!(std::fabs(t.weight_decay) < 3.0e38)) return bad("weight_decay must be finite");
        if (t.copy && (o->param_dtype != KT_F32 || !known_dtype(o->copy_dtype))) return bad("a 16-bit copy goes with fp32 parameters");
        if (t.n == 0) continue;
        if (!t.param || !t.grad || !t.m || !t.v) return bad("param, grad, m and v must be non-NULL");
        if (o->state_bits == 8 && (!t.m_scale || !t.v_scale)) return bad("8-bit moments need their scales");
        if (!aligned(t.param, pb) || !aligned(t.grad, gb) || !aligned(t.m, sb) || !aligned(t.v, sb) || !aligned(t.m_scale, 4) ||
            !aligned(t.v_scale, 4) || !aligned(t.copy, 2))
            return bad("a pointer is not aligned to its elements");
        for (const void* p : {(const void*)t.param, (const void*)t.m, (const void*)t.v}) {
            size_t at = (size_t)(((uint64_t)(uintptr_t)p * 0x9e3779b97f4a7c15ull) >> 32) & (places - 1);
            for (; written[at]; at = (at + 1) & (places - 1))
                if (written[at] == p) return bad("a parameter or moment is listed twice");  // (two blocks would update it)
            written[at] = p;
        }
        kt::AdamwEntry& x = e[live++];
        x.p = t.param;
        x.g = t.grad;
        x.m = t.m;
        x.v = t.v;
        x.ms = t.m_scale;
        x.vs = t.v_scale;
        x.copy = t.copy;
        x.n = t.n;
        x.first = 0;
        x.keep = (float)(1.0 - o->lr * t.weight_decay);
        const size_t state = o->state_bits == 8 ? 8 : 16;
        x.wide = aligned(t.param, 16) && aligned(t.grad, 16) && aligned(t.m, state) && aligned(t.v, state) && aligned(t.copy, 16);
    }
    if (!live) return done(KT_OK, "");
    kt_status s;
    int dev, sms;
    if ((s = current_device(&dev, &sms)) != KT_OK) return s;
    kt::AdamwStep a = {};
    a.param_dtype = o->param_dtype;
    a.grad_dtype = o->grad_dtype;
    a.copy_dtype = o->copy_dtype;
    a.bits = o->state_bits;
    a.b1 = (float)o->beta1;
    a.c1 = (float)(1.0 - o->beta1);
    a.b2 = (float)o->beta2;
    a.c2 = (float)(1.0 - o->beta2);
    a.eps = (float)o->eps;
    a.lr = o->lr;
    a.beta1 = o->beta1;
    a.beta2 = o->beta2;
    if (!o->step_device) {
        a.rate = (float)(o->lr / (1.0 - std::pow(o->beta1, (double)o->step)));
        a.root = (float)(1.0 / std::sqrt(1.0 - std::pow(o->beta2, (double)o->step)));
    }
    a.step = o->step_device;
    // on the device the step is 1 at least, and the correction largest there
    a.one = 1.0f;
    a.plain = 1.0 / std::sqrt(1.0 - o->beta2) <= 0x1p20 && o->eps <= 0x1p20;
    a.grad_scale = o->grad_scale;
    const char* why = "";
    return done(kt::launch_adamw(e, live, a, sms, dev, stream, &why), why);
}

kt_status kt_quantize_fp8(int64_t M, int64_t K, kt_dtype dtype, kt_act act, const void* X, int64_t ldx, void* Q, int64_t ldq,
                          float* scale, void* stream) {
    if (M < 0 || K < 1) return bad("the row count must not be negative and the row length at least 1");
    if (!known_dtype(dtype)) return bad("unknown dtype");
    if (!known_act(act)) return bad("unknown activation");
    if (M > INT32_MAX / 2 || K > (1 << 24)) return kt::report(KT_ERR_UNSUPPORTED, "M above 2^30 or K above 2^24");
    if (ldx < (act == KT_ACT_GEGLU ? 2 * K : K) || ldq < K) return bad("a row pitch is below the row length");
    if (M > 0 && (!X || !Q || !scale)) return bad("X, Q and scale must be non-NULL");
    if (!aligned(X, 2) || !aligned(scale, 4)) return bad("a pointer is not aligned to its elements");
    if (M == 0) return done(KT_OK, "");
    kt_status s;
    int dev, sms;
    if ((s = current_device(&dev, &sms)) != KT_OK) return s;
    const char* why = "";
    kt::QuantFp8 p = {X, static_cast<uint8_t*>(Q), scale, ldx, ldq, (int)M, (int)K, epilogue_of(act)};
    return done(kt::launch_quantize_fp8(dtype, p, sms, stream, &why), why);
}

kt_status kt_linear_fp8(int64_t M, int64_t N, int64_t K, kt_dtype dtype, const void* Q, int64_t ldq, const void* W, int64_t ldw,
                        const float* scale_x, const float* scale_w, const void* bias, void* Y, int64_t ldy, void* stream) {
    if (M < 0 || N < 1 || K < 1) return bad("M must not be negative, N and K at least 1");
    if (!known_dtype(dtype)) return bad("unknown dtype");
    if (ldq < K || ldw < K || ldy < N) return bad("a row pitch is below the row length");
    if ((M > 0 && (!Q || !scale_x || !Y)) || !W || !scale_w) return bad("Q, W, scale_x, scale_w and Y must be non-NULL");
    if (!aligned(Q, 16) || !aligned(W, 16) || !aligned(Y, 16) || !aligned(bias, 16)) return bad("Q, W, Y and bias must be 16-byte aligned");
    if (!aligned(scale_x, 4) || !aligned(scale_w, 4)) return bad("a pointer is not aligned to its elements");
    if (K % 16 || ldq % 16 || ldw % 16 || N % 8 || ldy % 8)
        return kt::report(KT_ERR_UNSUPPORTED, "K and the pitches of Q and W must be multiples of 16, N and Y's pitch of 8");
    if (M > INT32_MAX / 2 || N > (1 << 24) || K > (1 << 24) || ldq > (int64_t)1 << 38 || ldw > (int64_t)1 << 38 || ldy > (int64_t)1 << 38)
        return kt::report(KT_ERR_UNSUPPORTED, "M above 2^30, N or K above 2^24, or a pitch above 2^38");
    if (M == 0) return done(KT_OK, "");
    kt_status s;
    int dev, sms;
    if ((s = current_device(&dev, &sms)) != KT_OK) return s;
    const char* why = "";
    const unsigned long long stall_ns = 1000ull * (unsigned long long)g_matmul_stall_us.load(std::memory_order_relaxed);
    kt::LinearFp8 a = {Q, W, scale_x, scale_w, bias, Y, ldq, ldw, ldy, (int)M, (int)N, (int)K, stall_ns ? stall_ns : kWaitLimitNs, stall_ns};
    return done(kt::launch_linear_fp8(dtype, a, sms, dev, stream, &why), why);
}

kt_status kt_matmul_status(void* stream) {
    int dev, sms, word = 0, word8 = 0;
    kt_status s;
    if ((s = current_device(&dev, &sms)) != KT_OK) return s;
    const char* why = "";
    if ((s = kt::matmul_status(stream, &word, &why)) != KT_OK || (s = kt::linear_fp8_status(stream, &word8, &why)) != KT_OK)
        return kt::report(s, why);
    if (word == 0) word = word8;
    if (word == 0) return done(KT_OK, "");
    return kt::report(KT_ERR_TIMEOUT, word == kt::DEV_INJECTED_STALL ? "a bounded device wait ran out (injected stall)"
                                                                     : "a bounded device wait ran out");
}

kt_status kt_matmul_debug_stall(int enable, int64_t limit_us) {
    if (enable && (limit_us < 1 || limit_us > kMostStallUs)) return bad("limit_us must be in [1, 10 000 000]");
    g_matmul_stall_us.store(enable ? limit_us : 0, std::memory_order_relaxed);
    return done(KT_OK, "");
}

}  // extern "C"
