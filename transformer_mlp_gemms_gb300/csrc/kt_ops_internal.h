// kt_ops_internal.h -- between the ABI of the operators around the MLP (kt_ops_abi.cpp) and
// their kernels.  Not part of the public interface (that is include/kt_ops.h).
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include <cstddef>
#include <cstdint>

#include "kt_internal.h"
#include "kt_ops.h"

namespace kt {

// The calling thread's last error (kt_mlp_abi.cpp): record a message and return the status.
kt_status report(kt_status s, const char* msg);

struct LnForward {
    const void *X, *gamma, *beta;
    void* Y;
    float *mean, *rstd;
    int64_t ldx, ldy;
    int M, D;
    float eps;
};
kt_status launch_ln_forward(int dtype, const LnForward& p, int sms, void* stream, const char** why);

struct LnBackward {
    const void *dY, *X, *gamma;
    const float *mean, *rstd;
    void* dX;
    float *dgamma, *dbeta;
    float* partials;  // [ln_backward_blocks][2][D]
    int64_t lddy, ldx, lddx;
    int M, D;
};
// Blocks (and rows of partial sums) of a backward call on any device of up to kMaxSms SMs.
constexpr int kMaxSms = 160;
int ln_backward_blocks(int64_t M, int64_t D);
kt_status launch_ln_backward(int dtype, const LnBackward& p, int sms, int device, void* stream, const char** why);

struct QuantRows {
    const void* X;
    int8_t* Q;
    float* scale;
    int64_t ldx, ldq;
    int M, K, act;
};
kt_status launch_quantize(int dtype, const QuantRows& p, int sms, void* stream, const char** why);

struct LinearI8 {
    const int8_t *Q, *W;
    const float *sx, *sw;
    const void* bias;
    void* Y;
    int64_t ldq, ldw, ldy;
    int M, N, K;
    unsigned long long wait_limit_ns, stall_ns;  // bound of every device-side wait; the tests' hook (0: off)
};
kt_status launch_linear_i8(int dtype, const LinearI8& p, int sms, int device, void* stream, const char** why);
// The current device's error word once `stream` is done, cleared if it was set.
kt_status linear_i8_status(void* stream, int* word, const char** why);

// The mixture-of-experts layer (kt_moe.cu).
struct MoeParams {
    const void *X, *W_router, *W_up, *W_down, *b_up, *b_down, *R;
    void* Y;
    int32_t* ids;
    float* weights;
    int64_t ldx;
    int T, D, F, F_up, E, top_k, normalize;
    // workspace
    float2* choices;     // [T][top_k]: each token's experts (as integer bits) and their weights
    uint16_t* H;         // [2][T * top_k][F]: the hidden layer's rounding, then the remainder's
    float* Z;            // [splits][T * top_k][D]: each pair's output before its weight
    unsigned* barriers;  // grid barrier counters, zero between runs
    unsigned* ready;     // of each active expert: tiles of its H that are stored; zero between runs
    int* error;          // device error word
    unsigned long long wait_limit_ns, stall_ns;  // bound of every device-side wait; the tests' hook (0: off)
};
// Splits of the down projection along F that there is room for: up to 32 while pairs are few.
KT_HOST_DEVICE inline int moe_splits(int pairs) { return pairs >= 1024 ? 1 : pairs * 32 < 1024 ? 32 : 1024 / pairs; }
inline size_t moe_z_rows(int max_pairs) {  // for any number of pairs up to max_pairs
    return max_pairs >= 1024 ? max_pairs : max_pairs * 32 < 1024 ? max_pairs * 32 : 1024;
}
constexpr size_t kMoeControlBytes = 256 + KT_MOE_MAX_EXPERTS * sizeof(unsigned);  // counters and error word, zero at first
size_t moe_workspace(int64_t T, int64_t D, int64_t F, int64_t top_k);
void moe_carve(MoeParams* p, int64_t max_tokens, void* workspace);
kt_status launch_moe(int act, int dtype, const MoeParams& p, int sms, int device, void* stream, const char** why);

// Opt a kernel in to `bytes` of dynamic shared memory on the current device, once per device: the
// attribute stays.  `done` belongs to the kernel (a static of its launch function).
struct SmemOptIn {
    std::atomic<uint64_t> done{0};  // a bit per device ordinal
    template <typename K>
    cudaError_t operator()(K kern, int bytes, int device) {
        const uint64_t bit = 1ull << (device & 63);
        if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
        return e;
    }
};

// A launch as a programmatic dependent of the previous kernel in the stream.
template <typename... P, typename... A>
inline cudaError_t launch_pdl(void (*kern)(P...), unsigned grid, unsigned block, size_t smem, void* stream, A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(block, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

}  // namespace kt
