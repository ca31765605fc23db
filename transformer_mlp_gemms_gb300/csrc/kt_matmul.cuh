// kt_matmul.cuh -- what the products of kt_matmul.cu and kt_linear_fp8.cu share.
#pragma once
#include "kt_gemm.cuh"

namespace kt {

constexpr int kBand = 8;  // tile rows of a band

// The t-th tile: bands of kBand tile rows, in each column after column.
__device__ __forceinline__ void band_tile(int t, int tiles_m, int tiles_n, int& tm, int& tn) {
    const int per = kBand * tiles_n, band = t / per, in = t - band * per;
    const int rows = min(kBand, tiles_m - band * kBand);
    tn = in / rows;
    tm = band * kBand + in - tn * rows;
}

// As wait_phase, for waits that many warps enter often: the timer is read only after some tries, each of which
// already suspends the thread for a while.
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_turn(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err, int code, unsigned long long limit_ns) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
        if (CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
    return wait_phase<CLUSTER>(bar, parity, abort_flag, err, code, limit_ns);
}

// A value that is the same in all lanes, made known as such to the compiler, which takes what comes from a 64-bit division,
// shared memory or a special register for one that may differ, and all that follows from it: eight products with a
// commit then took 688 clocks of their warp, and 507 (the tensor cores' own time) like this.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// What one thread issues, called by a whole warp with the same arguments and `one` in one lane: the arguments are then in
// uniform registers, where these instructions read them.  From a branch of a single lane each would be moved there
// first, and a step of the ring took 0.28 us however few products it had.
__device__ __forceinline__ void expect_tx_if(uint32_t bar, uint32_t bytes, uint32_t one) {
    asm volatile("{\n\t.reg .pred l;\n\tsetp.ne.b32 l, %2, 0;\n\t@l mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes),
                 "r"(one)
                 : "memory");
}
#define KT_LOAD_IF(dim, group, coords, ...)                                                                                  \
    asm volatile("{\n\t.reg .pred l;\n\tsetp.ne.b32 l, %3, 0;\n\t"                                                              \
                 "@l cp.async.bulk.tensor." dim ".shared::cluster.global.tile.mbarrier::complete_tx::bytes" group " [%0], [%1, " coords "], [%2];\n\t}" ::"r"(dst), \
                 "l"(reinterpret_cast<uint64_t>(tm)), "r"(bar), "r"(one), __VA_ARGS__                                          \
                 : "memory")
template <int PAIR>
__device__ __forceinline__ void load_if(uint32_t dst, const CUtensorMap* tm, uint32_t bar, int x, int y, uint32_t one) {
    if constexpr (PAIR == 2) KT_LOAD_IF("2d", ".cta_group::2", "{%4, %5}", "r"(x), "r"(y));
    else KT_LOAD_IF("2d", "", "{%4, %5}", "r"(x), "r"(y));
}
template <int PAIR>
__device__ __forceinline__ void load3_if(uint32_t dst, const CUtensorMap* tm, uint32_t bar, int x, int y, int z, uint32_t one) {
    if constexpr (PAIR == 2) KT_LOAD_IF("3d", ".cta_group::2", "{%4, %5, %6}", "r"(x), "r"(y), "r"(z));
    else KT_LOAD_IF("3d", "", "{%4, %5, %6}", "r"(x), "r"(y), "r"(z));
}
#undef KT_LOAD_IF
#define KT_MMA_IF(group, kind)                                                                                          \
    asm volatile("{\n\t.reg .pred p, l;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 l, %5, 0;\n\t"                           \
                 "@l tcgen05.mma.cta_group::" group ".kind::" kind " [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(ad), "l"(bd), \
                 "r"(idesc), "r"(accumulate), "r"(one)                                                                \
                 : "memory")
template <int PAIR, bool FP8>
__device__ __forceinline__ void mma_if(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t accumulate, uint32_t one) {
    if constexpr (PAIR == 2 && FP8) KT_MMA_IF("2", "f8f6f4");
    else if constexpr (PAIR == 2) KT_MMA_IF("2", "f16");
    else if constexpr (FP8) KT_MMA_IF("1", "f8f6f4");
    else KT_MMA_IF("1", "f16");
}
#undef KT_MMA_IF
// Arrive on the barrier (at this offset in both CTAs of a pair) once all products so far are done.
template <int PAIR>
__device__ __forceinline__ void commit_if(uint32_t bar, uint32_t one) {
    if constexpr (PAIR == 2)
        asm volatile(
            "{\n\t.reg .pred l;\n\tsetp.ne.b32 l, %2, 0;\n\t"
            "@l tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
            "h"((unsigned short)3), "r"(one)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred l;\n\tsetp.ne.b32 l, %1, 0;\n\t"
            "@l tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(one)
            : "memory");
}

// As mbar_test_wait, acquiring at cluster scope as mbar_try_wait_cluster does.
__device__ __forceinline__ uint32_t mbar_test_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok;
}

// The end of the warp that issues a CTA's (or pair's) products.  It waits for the last of them, whether or not it knows that
// an epilogue warp has given up, which may come later: none may be running when tensor memory is freed.  Those that
// were issued have waited for their copies.  Where some were not (ok false), copies of the stages from `stage` on may be
// on their way into memory that is about to be released, from warps that ended before this CTA gave up: they get 1 ms
// each to land (a copy takes a few microseconds; what nobody counted does not show).
template <int PAIR>
__device__ __forceinline__ void settle(bool ok, uint32_t bar_drain, uint32_t bar_full, uint32_t stage, uint32_t phase, uint32_t stages) {
    const uint32_t one = (threadIdx.x & 31u) == 0;
    commit_if<PAIR>(bar_drain, one);
    if (one) {
        wait_drain(bar_drain, 0u, 100000000ull);
        for (uint32_t s = ok ? stages : 0u; s < stages; ++s) {
            wait_drain(bar_full + 8u * stage, phase, 1000000ull);
            if (++stage == stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
    }
}

// Waits until another CTA's flag is raised, as the wait on a barrier: bounded, and given up where this CTA aborts.
__device__ __forceinline__ bool wait_flag(const int* flag, volatile int* abort_flag, int* err, unsigned long long limit_ns) {
    const unsigned long long t0 = global_ns();
    for (uint32_t i = 1;; ++i) {
        int v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
        if (v) return true;
        if ((i & 15u) == 0) {
            if (*abort_flag) return false;
            if (global_ns() - t0 > limit_ns) {
                *abort_flag = 1;
                atomicCAS(err, 0, DEV_TIMEOUT_EPILOGUE);
                return false;
            }
        }
    }
}

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

// Four fp32 sums of a CTA of this cluster.
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// 32 bias values from column `col` on, zeros in groups of 8 at or past `limit`.  Ordinary loads: the kernel
// before this one may still be writing a bias while this one is already resident.
template <int DT>
__device__ __forceinline__ void bias32(const void* bias, int col, int limit, float* b) {
    const uint16_t* at = static_cast<const uint16_t*>(bias) + col;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (col + 8 * g < limit) w = *reinterpret_cast<const uint4*>(at + 8 * g);
        unpack8<DT>(w, b + 8 * g);
    }
}

// The current device's error word once `stream` is done, cleared if it was set.
template <typename Symbol>
kt_status error_word(const Symbol& symbol, void* stream, int* word, const char** why) {
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemcpyFromSymbolAsync(word, symbol, sizeof(int), 0, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e == cudaSuccess && *word != 0) {
        const int none = 0;
        e = cudaMemcpyToSymbolAsync(symbol, &none, sizeof(int), 0, cudaMemcpyHostToDevice, st);
        if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    }
    if (e == cudaSuccess) return KT_OK;
    *why = cudaGetErrorString(e);
    return KT_ERR_CUDA;
}

}  // namespace kt
