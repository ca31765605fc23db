// kt_linear_i8.cu -- the linear layer on 8-bit integers with a scale for each token and channel:
//   Y[m][n] = round(sx[m] sw[n] sum_k Q[m][k] W[n][k] (+ b[n])).
#include "kt_ops_internal.h"
#include "kt_rows.cuh"

namespace kt {
namespace {

template <int DT>
__device__ __forceinline__ uint16_t to_bits(float v) {
    return (uint16_t)(pack2<DT>(v, 0.0f) & 0xffffu);
}
template <int DT>
__device__ __forceinline__ float from_bits(uint16_t u) {
    float f[8];
    unpack8<DT>(make_uint4(u, 0u, 0u, 0u), f);
    return f[0];
}

// A few tokens.  Bound by the weight's bytes: each is read once (per 8 tokens) and meets 8
// tokens in four-way integer products into 32-bit sums.  Eight lanes share a weight row (128
// consecutive bytes per step), a warp covers 8 rows, and the tokens' rows are in shared
// memory, read as 128-byte broadcasts to the four groups of a warp.
constexpr int kDotWarps = 4, kDotTokens = KT_LINEAR_I8_DOT_ROWS, kDotRows = kDotWarps * 8;
constexpr int kDotChunk = 4096;  // columns of the tokens staged at a time

template <int DT>
__global__ void __launch_bounds__(kDotWarps * 32) kt_linear_i8_dot_kernel(const LinearI8 p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(16) int8_t sq[];  // [8][chunk]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = lane >> 3, k8 = lane & 7;
    const int n0 = (int)blockIdx.x * kDotRows + warp * 8 + group * 2;
    const int m0 = (int)blockIdx.y * kDotTokens;
    const int tokens = min(kDotTokens, p.M - m0);
    const int8_t* w0 = p.W + (int64_t)min(n0, p.N - 1) * p.ldw;
    const int8_t* w1 = p.W + (int64_t)min(n0 + 1, p.N - 1) * p.ldw;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int acc[2][kDotTokens];
#pragma unroll
    for (int t = 0; t < kDotTokens; ++t) acc[0][t] = acc[1][t] = 0;
    for (int k0 = 0; k0 < p.K; k0 += kDotChunk) {
        const int kc = min(kDotChunk, p.K - k0), kp = (kc + 127) & ~127;  // padded to whole steps with zeros
        if (k0) __syncthreads();
        for (int i = threadIdx.x; i < kDotTokens * (kp / 16); i += kDotWarps * 32) {
            const int t = i / (kp / 16), k = (i % (kp / 16)) * 16;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (t < tokens && k < kc) v = *reinterpret_cast<const uint4*>(p.Q + (int64_t)(m0 + t) * p.ldq + k0 + k);
            *reinterpret_cast<uint4*>(sq + t * kp + k) = v;
        }
        __syncthreads();
#pragma unroll 4
        for (int k = k8 * 16; k < kp; k += 128) {
            uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
            if (k < kc) {
                a = __ldg(reinterpret_cast<const uint4*>(w0 + k0 + k));
                b = __ldg(reinterpret_cast<const uint4*>(w1 + k0 + k));
            }
#pragma unroll
            for (int t = 0; t < kDotTokens; ++t) {
                const uint4 q = *reinterpret_cast<const uint4*>(sq + t * kp + k);
                acc[0][t] = __dp4a((int)a.x, (int)q.x, acc[0][t]);
                acc[1][t] = __dp4a((int)b.x, (int)q.x, acc[1][t]);
                acc[0][t] = __dp4a((int)a.y, (int)q.y, acc[0][t]);
                acc[1][t] = __dp4a((int)b.y, (int)q.y, acc[1][t]);
                acc[0][t] = __dp4a((int)a.z, (int)q.z, acc[0][t]);
                acc[1][t] = __dp4a((int)b.z, (int)q.z, acc[1][t]);
                acc[0][t] = __dp4a((int)a.w, (int)q.w, acc[0][t]);
                acc[1][t] = __dp4a((int)b.w, (int)q.w, acc[1][t]);
            }
        }
    }
    // sums over the 8 lanes of a group; lane k8 ends with token k8
    int sum[2] = {0, 0};
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int t = 0; t < kDotTokens; ++t) {
            int v = acc[r][t];
            v += __shfl_xor_sync(0xffffffffu, v, 1);
            v += __shfl_xor_sync(0xffffffffu, v, 2);
            v += __shfl_xor_sync(0xffffffffu, v, 4);
            if (t == k8) sum[r] = v;
        }
    if (k8 >= tokens) return;
    const float sx = p.sx[m0 + k8];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int n = n0 + r;
        if (n >= p.N) break;
        float v = (float)sum[r] * (sx * p.sw[n]);
        if (p.bias) v += from_bits<DT>(static_cast<const uint16_t*>(p.bias)[n]);
        static_cast<uint16_t*>(p.Y)[(int64_t)(m0 + k8) * p.ldy + n] = to_bits<DT>(v);
    }
}

}  // namespace

kt_status launch_linear_i8(int dtype, const LinearI8& p, int sms, void* stream, const char** why) {
    (void)sms;
    const int chunk = std::min(kDotChunk, (p.K + 127) & ~127);
    const dim3 grid((unsigned)((p.N + kDotRows - 1) / kDotRows), (unsigned)((p.M + kDotTokens - 1) / kDotTokens));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kDotWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = (size_t)kDotTokens * chunk;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = dtype == KT_BF16 ? cudaLaunchKernelEx(&cfg, kt_linear_i8_dot_kernel<KT_BF16>, p)
                                     : cudaLaunchKernelEx(&cfg, kt_linear_i8_dot_kernel<KT_F16>, p);
    if (e != cudaSuccess) {
        *why = cudaGetErrorString(e);
        return KT_ERR_CUDA;
    }
    return KT_OK;
}

}  // namespace kt
