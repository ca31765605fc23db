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

// Products of 16-bit matrices (kt_matmul.cu): C[M][N] = round(A . B^T (+ bias)).
struct Matmul {
    const void* A;        // [M][K] or, a_mn, [K][M]; pitch lda
    const void* B;        // [N][K] or, b_mn, [K][N]; pitch ldb.  gated: [2N][K], value rows, then gate rows
    void* C;              // [M][N], pitch ldc.  gated: value * act(gate)
    const void* bias;     // [N] (gated: [2N]) or null
    void* P;              // gated: [M][2N], value and gate, pitch ldp; or null
    int64_t lda, ldb, ldc, ldp;
    int M, N, K, act;     // act: gated, an Epi
    bool a_mn, b_mn, gated;
    unsigned long long wait_limit_ns, stall_ns;
};
// How a product is run: CTAs per tile, accumulator columns per tile, CTAs that share a tile's sums, 64-deep steps per
// stage of the ring.
struct MatmulShape {
    int pair, BN, splits, atoms;  // (atoms: 2 with an MN-major operand)
    double us;  // what it is expected to take
};
MatmulShape matmul_shape(const Matmul& a, int sms, int device);
kt_status launch_matmul_as(int dtype, const Matmul& a, const MatmulShape& s, int sms, int device, void* stream, const char** why);
kt_status launch_matmul(int dtype, const Matmul& a, int sms, int device, void* stream, const char** why);
// One or two products of a backward pass, in one launch (the one with longer sums first) or each in its own.  scratch:
// flags (kGradientsFlags bytes, set to zero here unless zeroed), then gradients_partials() bytes.
constexpr size_t kGradientsFlags = kMaxSms * sizeof(int);  // a flag per CTA
constexpr int kGradientsLeast = 4;  // steps that a pair's share of the last tiles has at least
struct GradientsShape {
    int bn[2], share;  // tile widths (128 or 256); the pairs that the last tiles' steps are shared out to, 0: none are
    double us;         // what it is expected to take
};
size_t gradients_partials();
GradientsShape gradients_shape(const Matmul* a, int count, int sms);
kt_status launch_gradients_as(int dtype, const Matmul* a, int count, const GradientsShape& s, void* scratch, int sms, int device, void* stream, const char** why);
kt_status launch_gradients(int dtype, const Matmul* a, int count, void* scratch, bool zeroed, int sms, int device, void* stream, const char** why);
kt_status matmul_status(void* stream, int* word, const char** why);

// The elementwise part of the backward pass of a gated block, and column sums (kt_glu.cu).
struct GluBackward {
    const void *dH, *P;  // dH: [M][F]; P: [M][2F]; null P: column sums of dH alone
    void* dP;            // [M][2F], pitch lddp
    float* partials;     // [column_sum_rows][2F] (F without P), or null: no sums
    float* db;           // [2F] (F)
    int* zero;           // kGradientsFlags bytes to be zeroed, or null
    int64_t lddh, ldp, lddp;
    int M, F, act;       // act: an Epi
};
int column_sum_rows(int64_t M, int64_t F);
kt_status launch_glu_backward(int dtype, const GluBackward& p, void* stream, const char** why);
kt_status launch_zero(int* at, void* stream, const char** why);  // kGradientsFlags bytes

// AdamW over many tensors (kt_adamw.cu).
struct AdamwEntry {
    void* p;
    const void* g;
    void *m, *v;
    float *ms, *vs;  // 8-bit moments: their scales
    void* copy;      // 16-bit copy of fp32 parameters, or null
    int64_t n;
    int64_t first;   // the launch's: the tensor's first chunk
    float keep;      // 1 - lr * weight decay
    int wide;        // every address allows its vector loads
};
struct AdamwStep {
    int param_dtype, grad_dtype, copy_dtype, bits;
    float b1, c1, b2, c2, eps, rate, root;  // c = 1 - b; rate = lr / (1 - beta1^t), root = 1 / sqrt(1 - beta2^t)
    double lr, beta1, beta2;                // for a step number on the device
    const int64_t* step;                    // it, or null
    const float* grad_scale;                // or null
    float one;                              // 1
    int plain;                              // root and eps up to 2^20: the quick roots and quotients apply
};
kt_status launch_adamw(const AdamwEntry* e, int count, const AdamwStep& s, int sms, int device, void* stream, const char** why);

// The linear layer in 8-bit floating point, and its quantiser (kt_linear_fp8.cu).
struct QuantFp8 {
    const void* X;
    uint8_t* Q;
    float* scale;  // [M][ceil(K / 128)]
    int64_t ldx, ldq;
    int M, K, act;  // act: an Epi
};
kt_status launch_quantize_fp8(int dtype, const QuantFp8& p, int sms, void* stream, const char** why);
struct LinearFp8 {
    const void *Q, *W;
    const float *sx, *sw;
    const void* bias;
    void* Y;
    int64_t ldq, ldw, ldy;
    int M, N, K;
    unsigned long long wait_limit_ns, stall_ns;
};
// CTAs per tile, channels (or, swap, tokens) per tile, whether the weights are the first operand, CTAs that share a tile's runs.
struct Fp8Shape {
    int pair, BN, swap, splits;
};
Fp8Shape linear_fp8_shape(const LinearFp8& a, int sms, int device);
kt_status launch_linear_fp8_as(int dtype, const LinearFp8& a, const Fp8Shape& s, int sms, int device, void* stream, const char** why);
kt_status launch_linear_fp8(int dtype, const LinearFp8& a, int sms, int device, void* stream, const char** why);
kt_status linear_fp8_status(void* stream, int* word, const char** why);

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
