// kt_linear_fp8.cu -- activations in 8-bit floating point with a scale for each token and run of 128 columns, and
// the linear layer on them, its weights with a scale for each block of 128 x 128:
//
//   Y[m][n] = round( sum_j sx[m][j] sw[n / 128][j] sum_{k in run j} Q[m][k] W[n][k]  (+ bias[n]) )
//
// The products are tcgen05.mma kind::f8f6f4 with fp32 accumulators.  A run's sum has scales of its own,
// so each run has an accumulator of its own: while the tensor cores work on the next, the epilogue warps
// take the finished one out of tensor memory and add it, times its scales, to fp32 sums in their registers.
//
// Many tokens: a CTA (or, cta_group::2, a pair) per tile of 128 (256) tokens x BN channels, persistent, in bands
// as kt_matmul.cu; eight epilogue warps share the tile's columns, so that a thread has one token's row and
// BN / 2 sums.  The tokens' scales come through shared memory, eight runs at a time, [run][token]: read from
// where they lie they would cost a line per lane.
// Few tokens (SWAP): the weights are the first operand, 128 channels a tile, and the tokens the second,
// 16 or 32 columns, so that no tensor-core row is idle; a thread has one channel.  Bound by the weights' bytes.
// Bound, with many tokens, by the epilogue warps' way from tensor memory to their sums: a warp's 128 sums leave no registers
// for more than one load of eight columns on its way, and four paired multiply-adds are all that it is hidden behind.
// 8192 x 8192 x 8192: a call alone 369 to 380 us, 2.9 PFLOP/s, the tensor pipe busy 63 % of the time and the schedulers
// 51 %; calls in sequence 408 us, at the 1.75 GHz that the power cap leaves.  4 x 10240 x 1280: 5.4 to 5.9 us, 2.4 TB/s,
// a launch and one round of loads.
// Few tiles with long rows: a cluster per tile, each CTA with its share of the runs; the sums meet in the
// cluster's shared memory, added in the order of the ranks.
#include <cuda_fp8.h>

#include "kt_ops_internal.h"
#include "kt_gemm.cuh"
#include "kt_exact.cuh"
#include "kt_matmul.cuh"

namespace kt {

__device__ int g_fp8_error;

namespace {

constexpr int kRun = 128;
constexpr uint32_t kF8ABytes = 128 * kRun;

// ---------------------------------------------------------------------------
// The quantiser
// ---------------------------------------------------------------------------

constexpr int kQuantThreads = 256, kQuantRows = 4;

__device__ __forceinline__ float activate(float z, int act) {
    f32x2 v = f2(z, 0.0f);
    switch (act) {
        case EPI_GELU_ERF: return act_f2<EPI_GELU_ERF, true>(v).x;
        case EPI_GELU_TANH: return act_f2<EPI_GELU_TANH, true>(v).x;
        case EPI_GELU_SIGMOID: return act_f2<EPI_GELU_SIGMOID, true>(v).x;
        case EPI_SILU: return act_f2<EPI_SILU, true>(v).x;
        default: return z;
    }
}

// Eight elements of a run in 16 bits: consecutive ones (WIDE, a 16-byte load), else every sixteenth; zeros past its end.
template <bool WIDE>
__device__ __forceinline__ uint4 run_slot(const uint16_t* at, int l, int end) {
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (WIDE) {
        if (8 * l < end) w = *reinterpret_cast<const uint4*>(at + 8 * l);
    } else {
        uint32_t u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = l + 16 * e < end ? at[l + 16 * e] : 0u;
        w = make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
    }
    return w;
}

// Sixteen lanes per run of 128 columns, four rows of it at a time, whose loads go out together.  Bound by memory, 3 bytes
// per element: 8192 x 8192 in 41 us, 4.9 TB/s.  ACT: the activation of X is quantised, bound by its instructions (16384 x
// 5120: SiLU 114 us, 2.2 TB/s, GEGLU 122 us, 3.4 TB/s).
template <int DT, bool WIDE, bool ACT>
__global__ void __launch_bounds__(kQuantThreads) kt_quantize_fp8_kernel(const QuantFp8 p, int runs, int64_t total) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int kPer = kQuantThreads / 16;
    const int l = threadIdx.x & 15;
    // the two halves of a warp may end apart: the whole warp goes on while either has a run
    for (int64_t i = (int64_t)blockIdx.x * kPer + (threadIdx.x >> 4); (i & ~(int64_t)1) < total; i += (int64_t)gridDim.x * kPer) {
        const bool live = i < total;
        const int64_t group = !live ? 0 : total <= INT32_MAX ? (int64_t)((uint32_t)i / (uint32_t)runs) : i / runs;
        const int64_t row0 = group * kQuantRows;
        const int run = live ? (int)(i - group * runs) : 0, end = live ? min(kRun, p.K - run * kRun) : 0;
        const int rows = (int)min((int64_t)kQuantRows, p.M - row0);
        const uint16_t* x = static_cast<const uint16_t*>(p.X) + row0 * p.ldx + run * kRun;
        uint4 w[kQuantRows], gate[ACT ? kQuantRows : 1];
#pragma unroll
        for (int a = 0; a < kQuantRows; ++a) {
            w[a] = run_slot<WIDE>(x + a * p.ldx, l, a < rows ? end : 0);
            if constexpr (ACT) gate[a] = p.act == EPI_GEGLU ? run_slot<WIDE>(x + a * p.ldx + p.K, l, a < rows ? end : 0) : w[a];
        }
#pragma unroll
        for (int a = 0; a < kQuantRows; ++a) {
            float f[8];
            unpack8<DT>(w[a], f);
            if constexpr (ACT) {
                float g[8];
                unpack8<DT>(gate[a], g);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = p.act == EPI_GEGLU ? f[e] * activate(g[e], EPI_GELU_ERF) : activate(f[e], p.act);
            }
            float most = fabsf(f[0]);
#pragma unroll
            for (int e = 1; e < 8; ++e) most = max_nan(most, fabsf(f[e]));
#pragma unroll
            for (int o = 8; o; o >>= 1) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
            f32x2 both;  // most / 448, 448 / most
            if (most >= 0x1p-60f && most <= 0x1p60f) both = quotient_rn(f2(most, 448.0f), f2(448.0f, most), f2(-448.0f, -most));
            else both = most < 0x1p-100f ? f2(0.0f) : f2(__fdiv_rn(most, 448.0f), __fdiv_rn(448.0f, most));
            if (a >= rows || !end) continue;
            if (l == 0) p.scale[(row0 + a) * runs + run] = both.x;
            uint32_t q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f32x2 t = f2_mul<true>(f2(f[2 * j], f[2 * j + 1]), f2(both.y));
                q[j] = __nv_cvt_float2_to_fp8x2(make_float2(t.x, t.y), __NV_SATFINITE, __NV_E4M3);
            }
            uint8_t* to = p.Q + (row0 + a) * p.ldq + run * kRun;
            if constexpr (WIDE) {
                if (8 * l < end) *reinterpret_cast<uint2*>(to + 8 * l) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (l + 16 * e < end) to[l + 16 * e] = (uint8_t)(q[e >> 1] >> (8 * (e & 1)));
            }
        }
    }
}

// ---------------------------------------------------------------------------
// The linear layer
// ---------------------------------------------------------------------------

// 8 or 16 columns of a warp's lanes of tensor memory
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld16(taddr, r); }
__device__ __forceinline__ void tmem_wait_cols(uint32_t (&r)[16]) { tmem_wait_ld(r); }
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_cols(uint32_t (&r)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
}

struct F8Params {
    int M, N, runs, tiles_m, tiles_n;
    uint32_t idesc;
    const float *sx, *sw;
    const void* bias;
    void* Y;
    int64_t ldy;
    unsigned long long wait_limit_ns, stall_ns;
};

template <int PAIR, int BN, bool SWAP>
struct F8 {
    static constexpr int kEpi = SWAP ? 4 : 8;               // epilogue warps
    static constexpr int kCols = SWAP ? BN : BN / 2;        // sums per thread
    static constexpr int kBufs = BN > 64 ? 2 : 8;           // accumulators (of kRuns runs each)
    static constexpr int kThreads = (kEpi + 4) * 32;        // warps 0-2: copies of A, products, copies of B; 3: none; then the epilogue
    static constexpr uint32_t kBBytes = (uint32_t)(BN / PAIR) * kRun;
    // Runs of a step (a stage of the ring, a wait and a signal of each role).  A step costs the issuing warp about 500 cycles
    // whatever it holds; a wide tile's run keeps the tensor cores busy that long, narrower ones go by twos
    // (16 x 4096 x 16384 13.0 -> 11.3 us, 1024 x 1024 x 8192 15.9 -> 14.9, or unshared 21.4 -> 19.0).
    static constexpr int kRuns = BN > 128 ? 1 : 2;
    static constexpr uint32_t kStage = kRuns * (kF8ABytes + kBBytes);
    static constexpr int kChunk = 8;                        // runs of scales in shared memory at a time
    static constexpr uint32_t kScales = SWAP ? 0u : 2u * kChunk * (128u + 2u) * 4u;  // [2][kChunk][128], then [2][2][kChunk]
    static constexpr uint32_t kStaging = SWAP ? 0u : (uint32_t)kEpi * 2048u;
    static constexpr int kFit = (int)((kSmemBudget - 1024 - 512 - kScales - kStaging) / kStage);
    static constexpr int kStages = kFit < 10 ? kFit : 10;
};

template <int DT, int PAIR, int BN, bool SWAP>
__global__ void __launch_bounds__(F8<PAIR, BN, SWAP>::kThreads, 1)
    kt_linear_fp8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ CUtensorMap tmY, const __grid_constant__ F8Params p) {
    using C = F8<PAIR, BN, SWAP>;
    constexpr int kEpi = C::kEpi, kCols = C::kCols, kBufs = C::kBufs, kStages = C::kStages, kRuns = C::kRuns;
    extern __shared__ uint8_t raw[];
    uint8_t* const at = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t base = smem_u32(at);
    const uint32_t staging = base + kStages * C::kStage;
    float* const scales = reinterpret_cast<float*>(at + kStages * C::kStage + C::kStaging);  // [2][kChunk][128]
    const uint32_t bars = staging + C::kStaging + C::kScales;
    const uint32_t bar_full = bars, bar_empty = bars + 80u, bar_accf = bars + 160u, bar_acce = bars + 224u, bar_drain = bars + 288u,
                   bar_stall = bars + 296u;
    uint32_t* const words = reinterpret_cast<uint32_t*>(at + (bars - base) + 304u);
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(words + 1);

    const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
    const unsigned long long limit = p.wait_limit_ns;
    const uint32_t rank = PAIR == 2 ? (uint32_t)uniform((int)(cluster_ctarank() & 1u)) : 0u;
    const int splits = PAIR == 1 ? uniform((int)cluster_size()) : 1, part = PAIR == 1 ? uniform((int)cluster_ctarank()) : 0;
    const bool leader = rank == 0;
    const int unit0 = (int)blockIdx.x / (PAIR * splits), units = (int)gridDim.x / (PAIR * splits);
    const int tiles = p.tiles_m * p.tiles_n;
    const int run0 = p.runs * part / splits, runs = p.runs * (part + 1) / splits - run0;  // of a tile, in this CTA

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(bar_full + 8u * s, 1);
            mbar_init(bar_empty + 8u * s, 1);
        }
        for (int b = 0; b < kBufs; ++b) {
            mbar_init(bar_accf + 8u * b, 1);
            mbar_init(bar_acce + 8u * b, kEpi * PAIR);
        }
        mbar_init(bar_drain, 1);
        mbar_init(bar_stall, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
        if (!SWAP) prefetch_tmap(&tmY);
    }
    if (warp == 1) tmem_alloc<PAIR>(smem_u32(words), kTmemCols);
    tc_fence_before();
    __syncthreads();
    if (PAIR == 2) cluster_sync_relaxed();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)words[0]);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // first token and first channel of tile t (of the pair's tile)
    auto origin = [&](int t, int& m, int& n) {
        if constexpr (SWAP) {
            m = 0;
            n = t * 128;
        } else {
            int tm, tn;
            band_tile(t, p.tiles_m, p.tiles_n, tm, tn);
            m = tm * PAIR * 128;
            n = tn * BN;
        }
    };

    if (warp == 0 || warp == 2) {
        // ------------------- copies: one lane issues what the whole warp has in uniform registers -------------------
        const bool a_role = warp == 0;
        const uint32_t one = lane == 0, arm = one && leader;
        uint32_t stage = 0, phase = 0, used = 0, used_phase = 0;
        bool ok = true;
        if (a_role && p.stall_ns && blockIdx.x == 0)  // the tests' hook: nobody signals this barrier
            ok = __all_sync(0xffffffffu, wait_phase(bar_stall, 0, abort_flag, &g_fp8_error, DEV_INJECTED_STALL, p.stall_ns));
        const uint32_t full0 = PAIR == 2 ? (uint32_t)uniform((int)mapa_rank(bar_full, 0)) : bar_full;
        const CUtensorMap* const map = a_role ? &tmA : &tmB;
        for (int t = unit0; t < tiles && ok; t += units) {
            int m, n;
            origin(t, m, n);
            const int row = a_role ? (SWAP ? n : m + (int)rank * 128) : (SWAP ? m : n + (int)rank * (BN / PAIR));
            for (int j = 0; j < runs; j += kRuns) {
                ok = __all_sync(0xffffffffu, wait_turn(bar_empty + 8u * stage, phase ^ 1u, abort_flag, &g_fp8_error, DEV_TIMEOUT_PRODUCER, limit));
                if (!ok) break;
                if (a_role) expect_tx_if(bar_full + 8u * stage, PAIR * C::kStage, arm);
                // the maps count pairs of bytes (a step may reach past the runs, and past K, where zeros are filled in)
#pragma unroll
                for (int i = 0; i < kRuns; ++i)
                    load_if<PAIR>(base + stage * C::kStage + (a_role ? (uint32_t)i * kF8ABytes : kRuns * kF8ABytes + (uint32_t)i * C::kBBytes), map,
                                  full0 + 8u * stage, (run0 + j + i) * (kRun / 2), row, one);
                used |= 1u << stage;
                used_phase = (used_phase & ~(1u << stage)) | (phase << stage);
                if (++stage == (uint32_t)kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (lane == 0) {
            if (*abort_flag) {  // no copy may still be on its way into memory that is about to be released
                if (a_role && leader)
                    for (int s = 0; s < kStages; ++s)
                        if (used & (1u << s)) wait_drain(bar_full + 8u * s, (used_phase >> s) & 1u, 100000000ull);
                const unsigned long long t0 = global_ns();
                while (global_ns() - t0 < 100000ull) __nanosleep(1000);
            }
        }
    } else if (warp == 1) {
        // ------------------- products, likewise -------------------
        if (leader) {
            const uint32_t one = lane == 0;
            uint32_t stage = 0, phase = 0, buf = 0, use = 0;
            const uint64_t ad0 = smem_desc(base, 16u, 1024u), bd0 = smem_desc(base + kRuns * kF8ABytes, 16u, 1024u);
            bool ok = true;
            // Narrow tiles are bound by this warp's instructions: both barriers of the next step are asked for before this
            // one's products, and the answers are there after them (1024 x 1024 x 8192 17.0 -> 16.3 us; wide tiles
            // lose by it, 8192^3 369 -> 378).
            constexpr bool kAhead = BN <= 128;
            // (accumulators come back from both CTAs of a pair: acquired at cluster scope)
            uint32_t full = 0u, free = 0u;
            for (int t = unit0; t < tiles && ok; t += units)
                for (int j = 0; j < runs; j += kRuns) {
                    ok = __all_sync(0xffffffffu,
                                    (full || wait_turn(bar_full + 8u * stage, phase, abort_flag, &g_fp8_error, DEV_TIMEOUT_MMA, limit)) &&
                                        (free || wait_turn<PAIR == 2>(bar_acce + 8u * buf, (use & 1u) ^ 1u, abort_flag, &g_fp8_error, DEV_TIMEOUT_MMA, limit)));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + buf * (uint32_t)(kRuns * BN), now = stage, which = buf;
                    const uint64_t ad = ad0 + stage * (C::kStage >> 4), bd = bd0 + stage * (C::kStage >> 4);
                    if (++stage == (uint32_t)kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (++buf == (uint32_t)kBufs) {
                        buf = 0;
                        ++use;
                    }
                    if constexpr (kAhead) {
                        full = mbar_test_wait(bar_full + 8u * stage, phase);
                        free = PAIR == 2 ? mbar_test_wait_cluster(bar_acce + 8u * buf, (use & 1u) ^ 1u) : mbar_test_wait(bar_acce + 8u * buf, (use & 1u) ^ 1u);
                    }
#pragma unroll
                    for (uint32_t i = 0; i < (uint32_t)kRuns; ++i) {
                        if (i > 0 && j + (int)i >= runs) break;
#pragma unroll
                        for (uint32_t k = 0; k < 4; ++k)  // 32 columns each
                            mma_if<PAIR, true>(d + i * (uint32_t)BN, ad + i * (kF8ABytes >> 4) + 2 * k, bd + i * (C::kBBytes >> 4) + 2 * k, p.idesc, k > 0, one);
                    }
                    commit_if<PAIR>(bar_accf + 8u * which, one);
                    commit_if<PAIR>(bar_empty + 8u * now, one);
                }
            settle<PAIR>(ok, bar_drain, bar_full, stage, phase, (uint32_t)kStages);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ------------------- epilogue -------------------
        const int ew = warp - 4, q = warp & 3, c0 = SWAP ? 0 : (ew >> 2) * kCols;  // lanes of tensor memory, first column
        uint32_t buf = 0, use = 0;
        bool ok = true;
        // The scales, kChunk runs at a time, copied into shared memory a chunk ahead: thread i of the 256 takes four
        // runs of token i / 2, and of the first sixteen each one of a block of 128 channels.
        const int st = (int)threadIdx.x - 128;
        auto copy = [&](float* to, const float* from, bool there) {  // (zero where there is none)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(there ? 4 : 0) : "memory");
        };
        auto fetch = [&](int t, int chunk, uint32_t slot) {
            int m, n;
            origin(t, m, n);
            m += (int)rank * 128 + (st >> 1);
            const int j = chunk * C::kChunk + (st & 1) * 4;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool there = m < p.M && j + i < runs;
                copy(scales + (slot * C::kChunk + (st & 1) * 4 + i) * 128 + (st >> 1), there ? p.sx + (int64_t)m * p.runs + run0 + j + i : p.sx, there);
            }
            if (st < 2 * C::kChunk) {
                const int block = st / C::kChunk, r = chunk * C::kChunk + st % C::kChunk;
                const bool there = block * 128 < BN && n + block * 128 < p.N && r < runs;
                copy(scales + 2 * C::kChunk * 128 + slot * 2 * C::kChunk + st, there ? p.sw + (int64_t)(n / 128 + block) * p.runs + run0 + r : p.sw, there);
            }
        };
        const int chunks = (runs + C::kChunk - 1) / C::kChunk;
        uint32_t slot = 0;  // of the chunk in use
        if (!SWAP && unit0 < tiles) fetch(unit0, 0, 1u);
        for (int t = unit0; t < tiles; t += units) {
            int m, n;
            origin(t, m, n);
            float sum[kCols];
#pragma unroll
            for (int i = 0; i < kCols; ++i) sum[i] = 0.0f;
            const float* sw = p.sw + (int64_t)(n / 128) * p.runs + run0;  // (SWAP: one block of channels)
            float w_next[kRuns], x_next[kRuns];  // SWAP: lane l has token l's
            auto tokens = [&](int j) {
#pragma unroll
                for (int i = 0; i < kRuns; ++i) {
                    const bool there = j + i < runs;
                    w_next[i] = there ? sw[j + i] : 0.0f;
                    x_next[i] = there && lane < p.M ? p.sx[(int64_t)lane * p.runs + run0 + j + i] : 0.0f;
                }
            };
            if constexpr (SWAP) tokens(0);
#pragma unroll 1
            for (int j = 0; j < runs; j += kRuns) {
                float x[kRuns];
                if constexpr (SWAP) {
#pragma unroll
                    for (int i = 0; i < kRuns; ++i) x[i] = x_next[i] * w_next[i];
                    if (j + kRuns < runs) tokens(j + kRuns);
                } else {
                    const int in = j % C::kChunk;
                    if (in == 0) {
                        slot ^= 1u;
                        asm volatile("cp.async.wait_all;" ::: "memory");
                        asm volatile("bar.sync 1, %0;" ::"n"(kEpi * 32) : "memory");
                        if (j / C::kChunk + 1 < chunks) fetch(t, j / C::kChunk + 1, slot ^ 1u);
                        else if (t + units < tiles) fetch(t + units, 0, slot ^ 1u);
                    }
#pragma unroll
                    for (int i = 0; i < kRuns; ++i)  // (chunks are whole steps; past the runs there are zeros)
                        x[i] = scales[2 * C::kChunk * 128 + (slot * 2 + c0 / 128) * C::kChunk + in + i] *
                               scales[(slot * C::kChunk + in + i) * 128 + 32 * q + lane];
                }
                ok = ok && wait_turn(bar_accf + 8u * buf, use & 1u, abort_flag, &g_fp8_error, DEV_TIMEOUT_EPILOGUE, limit);
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();
                const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + buf * (uint32_t)(kRuns * BN) + (uint32_t)c0;
                // 8 columns at a time (16 where there are few sums), the next on their way: a wide tile's 128 sums leave
                // no registers for more.  (After a wait that ran out the sums are of no use, and are NaN below.)
                constexpr int kLd = kCols > 64 ? 8 : 16;
                uint32_t r[2][kLd];
                tmem_ld_cols(acc, r[0]);
#pragma unroll
                for (int a = 0; a < kRuns * kCols; a += kLd) {
                    uint32_t(&now)[kLd] = r[a / kLd & 1];
                    const int c = a % kCols;
                    tmem_wait_cols(now);
                    if (a >= kCols && j + a / kCols >= runs) break;  // (nothing was added up there)
                    if (a + kLd < kRuns * kCols) tmem_ld_cols(acc + (uint32_t)((a + kLd) / kCols * BN + (a + kLd) % kCols), r[a / kLd + 1 & 1]);
#pragma unroll
                    for (int i = 0; i < kLd; i += 2) {
                        f32x2 s;
                        if constexpr (SWAP) s = f2(__shfl_sync(0xffffffffu, x[a / kCols], c + i), __shfl_sync(0xffffffffu, x[a / kCols], c + i + 1));
                        else s = f2(x[a / kCols]);
                        const f32x2 v = f2_fma<true>(f2(__uint_as_float(now[i]), __uint_as_float(now[i + 1])), s, f2(sum[c + i], sum[c + i + 1]));
                        sum[c + i] = v.x;
                        sum[c + i + 1] = v.y;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && ok) {  // (what was not seen is not given back, as in kt_matmul.cu)
                    if constexpr (PAIR == 2) mbar_arrive_cluster_relaxed(mapa_rank(bar_acce + 8u * buf, 0));
                    else mbar_arrive_relaxed(bar_acce + 8u * buf);
                }
                if (++buf == (uint32_t)kBufs) {
                    buf = 0;
                    ++use;
                }
            }
            if (!ok) {
#pragma unroll
                for (int i = 0; i < kCols; ++i) sum[i] = __uint_as_float(0x7fffffffu);
            }
            if (splits > 1) {
                // (one tile per cluster) the sums go where the operands were: 4 columns of 32 rows per 512 bytes
#pragma unroll
                for (int i = 0; i < kCols; i += 4)
                    st_shared_v4(base + (uint32_t)((q * BN + c0 + i) * 128 + lane * 16), __float_as_uint(sum[i]), __float_as_uint(sum[i + 1]),
                                 __float_as_uint(sum[i + 2]), __float_as_uint(sum[i + 3]));
            } else if constexpr (SWAP) {
                const int col = n + 32 * q + lane;
                if (col < p.N) {
                    float b[8] = {};
                    if (p.bias) unpack8<DT>(make_uint4(static_cast<const uint16_t*>(p.bias)[col], 0u, 0u, 0u), b);
                    uint16_t* y = static_cast<uint16_t*>(p.Y) + col;
#pragma unroll
                    for (int i = 0; i < kCols; ++i)
                        if (i < p.M) y[(int64_t)i * p.ldy] = (uint16_t)(pack2<DT>(sum[i] + b[0], 0.0f) & 0xffffu);
                }
            } else {
                const int y = m + (int)rank * 128 + 32 * q;
#pragma unroll
                for (int c = 0; c < kCols; c += 32) {
                    const int col = n + c0 + c;
                    if (col >= p.N || y >= p.M) continue;
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        if (p.bias && col + i < p.N) {
                            float b[8];
                            unpack8<DT>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.bias) + col + i), b);
#pragma unroll
                            for (int e = 0; e < 8; ++e) sum[c + i + e] += b[e];
                        }
#pragma unroll
                        for (int e = 0; e < 8; e += 2) w[(i + e) / 2] = pack2<DT>(sum[c + i + e], sum[c + i + e + 1]);
                    }
                    stage_and_store_packed(&tmY, staging + (uint32_t)ew * 2048u, lane, w, col, y);
                }
            }
        }
        if (!SWAP && lane == 0) bulk_wait0();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR == 1 && splits > 1) {
        if (*abort_flag)  // no sums from this CTA: NaN in their place, and so in the whole tile
            for (int i = threadIdx.x; i < 128 * BN; i += C::kThreads) reinterpret_cast<uint32_t*>(at)[i] = 0x7fffffffu;
        cluster_sync_all();  // every CTA's sums are there
        if (warp >= 4) {
            int m, n;
            origin(unit0, m, n);
            // four columns of 32 rows, over the cluster's CTAs
            auto four = [&](int q, int c) {
                const uint32_t from = base + (uint32_t)((q * BN + c) * 128 + lane * 16);
                float4 x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < splits) x[j] = ld_cluster4(mapa_rank(from, (uint32_t)j));
#pragma unroll
                for (int j = 1; j < 8; ++j)
                    if (j < splits) {
                        x[0].x += x[j].x;
                        x[0].y += x[j].y;
                        x[0].z += x[j].z;
                        x[0].w += x[j].w;
                    }
                return x[0];
            };
            if constexpr (SWAP) {
                for (int u = part + splits * (warp - 4); u < BN; u += splits * kEpi) {  // units of 4 tokens x 32 channels
                    const int q = u & 3, c = u >> 2 << 2, col = n + 32 * q + lane;
                    if (c >= p.M) continue;
                    const float4 s = four(q, c);
                    if (col >= p.N) continue;
                    float b[8] = {};
                    if (p.bias) unpack8<DT>(make_uint4(static_cast<const uint16_t*>(p.bias)[col], 0u, 0u, 0u), b);
                    const float v[4] = {s.x, s.y, s.z, s.w};
                    uint16_t* y = static_cast<uint16_t*>(p.Y) + (int64_t)c * p.ldy + col;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (c + i < p.M) y[(int64_t)i * p.ldy] = (uint16_t)(pack2<DT>(v[i] + b[0], 0.0f) & 0xffffu);
                }
            } else {
                for (int u = part + splits * (warp - 4); u < BN / 8; u += splits * kEpi) {  // units of 32 x 32
                    const int q = u & 3, c = 32 * (u >> 2), col = n + c, y = m + 32 * q;
                    if (col >= p.N || y >= p.M) continue;
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 s = four(q, c + 4 * i);
                        v[4 * i] = s.x, v[4 * i + 1] = s.y, v[4 * i + 2] = s.z, v[4 * i + 3] = s.w;
                    }
                    if (p.bias) {
                        float b[32];
                        bias32<DT>(p.bias, col, p.N, b);
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] += b[i];
                    }
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) w[i] = pack2<DT>(v[2 * i], v[2 * i + 1]);
                    stage_and_store_packed(&tmY, staging + (uint32_t)(warp - 4) * 2048u, lane, w, col, y);
                }
                if (lane == 0) bulk_wait0();
                __syncwarp();
            }
        }
    }
    if (PAIR == 2 || splits > 1) cluster_sync_all();  // neither leaves while another may still signal or read it
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc<PAIR>(tmem, kTmemCols);
    }
}

constexpr int kF8Smem = kSmemBudget;

template <int DT, int PAIR, int BN, bool SWAP>
cudaError_t f8_prepare(int device) {
    static SmemOptIn opt_in;
    return opt_in(kt_linear_fp8_kernel<DT, PAIR, BN, SWAP>, kF8Smem, device);
}

template <int PAIR, int BN, bool SWAP>
cudaLaunchConfig_t f8_config(int grid, int cluster, void* stream, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(F8<PAIR, BN, SWAP>::kThreads, 1, 1);
    cfg.dynamicSmemBytes = kF8Smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cfg;
}

// Clusters of ks CTAs that the device holds at once (one CTA per SM, whatever the tile); 0 if it cannot say.
int f8_clusters(int ks, int device) {
    static std::atomic<int> known[64][9];  // + 1
    int n = known[device & 63][ks].load(std::memory_order_relaxed) - 1;
    if (n >= 0) return n;
    n = 0;
    if (f8_prepare<KT_F16, 1, 128, false>(device) == cudaSuccess) {
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t cfg = f8_config<1, 128, false>(ks, ks, nullptr, attr);
        if (cudaOccupancyMaxActiveClusters(&n, kt_linear_fp8_kernel<KT_F16, 1, 128, false>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
    }
    known[device & 63][ks].store(n + 1, std::memory_order_relaxed);
    return n;
}

template <int PAIR, int BN, bool SWAP>
kt_status f8_launch(int dtype, const LinearFp8& a, int splits, int sms, int device, void* stream, const char** why) {
    F8Params p = {};
    p.M = a.M;
    p.N = a.N;
    p.runs = (a.K + kRun - 1) / kRun;
    p.tiles_m = SWAP ? 1 : (a.M + 128 * PAIR - 1) / (128 * PAIR);
    p.tiles_n = (a.N + (SWAP ? 128 : BN) - 1) / (SWAP ? 128 : BN);
    p.idesc = 1u << 4 | (uint32_t)(BN >> 3) << 17 | (uint32_t)(128 * PAIR >> 4) << 24;  // fp32 sums, e4m3 operands, both K-major
    p.sx = a.sx;
    p.sw = a.sw;
    p.bias = a.bias;
    p.Y = a.Y;
    p.ldy = a.ldy;
    p.wait_limit_ns = a.wait_limit_ns;
    p.stall_ns = a.stall_ns;
    CUtensorMap tm[3];
    // bytes in pairs: rows of K / 2 16-bit elements
    auto encode = [&](CUtensorMap* m, const void* at, int64_t ld, int64_t rows, int box_rows) {
        const uint64_t dims[2] = {(uint64_t)a.K / 2, (uint64_t)rows}, strides[1] = {(uint64_t)ld};
        const uint32_t box[2] = {kRun / 2, (uint32_t)box_rows};
        return encode_tmap_nd(m, at, KT_F16, 2, dims, strides, box, 128, why);
    };
    const uint64_t dims[2] = {(uint64_t)a.N, (uint64_t)a.M}, strides[1] = {(uint64_t)a.ldy * 2};
    const uint32_t box[2] = {kStoreCols, 32};
    if (SWAP) {
        if (!encode(tm, a.W, a.ldw, a.N, 128) || !encode(tm + 1, a.Q, a.ldq, a.M, BN)) return KT_ERR_CUDA;
        tm[2] = tm[0];
    } else if (!encode(tm, a.Q, a.ldq, a.M, 128) || !encode(tm + 1, a.W, a.ldw, a.N, BN / PAIR) ||
               !encode_tmap_nd(tm + 2, a.Y, dtype, 2, dims, strides, box, 64, why)) {
        return KT_ERR_CUDA;
    }
    const int tiles = p.tiles_m * p.tiles_n;
    const int grid = splits > 1 ? tiles * splits : std::min(tiles, sms / PAIR) * PAIR;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = f8_config<PAIR, BN, SWAP>(grid, PAIR * splits, stream, attr);
    cudaError_t e = dtype == KT_BF16 ? f8_prepare<KT_BF16, PAIR, BN, SWAP>(device) : f8_prepare<KT_F16, PAIR, BN, SWAP>(device);
    if (e == cudaSuccess)
        e = dtype == KT_BF16 ? cudaLaunchKernelEx(&cfg, kt_linear_fp8_kernel<KT_BF16, PAIR, BN, SWAP>, tm[0], tm[1], tm[2], p)
                             : cudaLaunchKernelEx(&cfg, kt_linear_fp8_kernel<KT_F16, PAIR, BN, SWAP>, tm[0], tm[1], tm[2], p);
    if (e != cudaSuccess) {
        *why = cudaGetErrorString(e);
        return KT_ERR_CUDA;
    }
    return KT_OK;
}

}  // namespace

kt_status launch_quantize_fp8(int dtype, const QuantFp8& p, int sms, void* stream, const char** why) {
    const int runs = (p.K + kRun - 1) / kRun;
    const bool wide = p.K % 8 == 0 && p.ldx % 8 == 0 && p.ldq % 8 == 0 && (reinterpret_cast<uintptr_t>(p.X) & 15u) == 0 &&
                      (reinterpret_cast<uintptr_t>(p.Q) & 7u) == 0;
    const int64_t total = (int64_t)((p.M + kQuantRows - 1) / kQuantRows) * runs, per = kQuantThreads / 16;
    const unsigned grid = (unsigned)std::min<int64_t>((total + per - 1) / per, (int64_t)sms * 64);
    auto go = [&](auto dt, auto wide_, auto act) {
        return launch_pdl(kt_quantize_fp8_kernel<decltype(dt)::value, decltype(wide_)::value, decltype(act)::value>, grid, (unsigned)kQuantThreads, (size_t)0,
                          stream, p, runs, total);
    };
    auto by_act = [&](auto dt, auto wide_) { return p.act == EPI_NONE ? go(dt, wide_, std::false_type{}) : go(dt, wide_, std::true_type{}); };
    auto by_width = [&](auto dt) { return wide ? by_act(dt, std::true_type{}) : by_act(dt, std::false_type{}); };
    const cudaError_t e = dtype == KT_BF16 ? by_width(std::integral_constant<int, KT_BF16>{}) : by_width(std::integral_constant<int, KT_F16>{});
    if (e != cudaSuccess) {
        *why = cudaGetErrorString(e);
        return KT_ERR_CUDA;
    }
    return KT_OK;
}

Fp8Shape linear_fp8_shape(const LinearFp8& a, int sms, int device) {
    const int runs = (a.K + kRun - 1) / kRun;
    Fp8Shape best = {};
    double least = 1e30;
    // us per run of 128 columns, of a launch, and of sharing a tile's runs; measured from 5 to 128 runs
    auto consider = [&](int pair, int bn, int swap, int64_t tiles, double step, double round, double sharing) {
        const int64_t units = sms / pair, rounds = (tiles + units - 1) / units;
        const double time = rounds * runs * step + (rounds - 1) * 0.7 + round;
        if (time < least) {
            least = time;
            best = {pair, bn, swap, 1};
        }
        if (pair == 2) return;
        for (int ks = 2; ks <= 8; ++ks) {
            if (tiles * ks > sms || runs < 2 * ks || tiles > f8_clusters(ks, device)) continue;
            const double split = (runs + ks - 1) / ks * step + round + sharing;
            if (split < least) {
                least = split;
                best = {1, bn, swap, ks};
            }
        }
    };
    if (a.M <= KT_LINEAR_FP8_FEW) {
        const int64_t tiles = (a.N + 127) / 128;
        if (a.M <= 16) consider(1, 16, 1, tiles, 0.186, 3.5, 1.4);
        else consider(1, 32, 1, tiles, 0.195, 4.0, 1.4);
        return best;
    }
    auto tiles = [&](int rows, int bn) { return (int64_t)((a.M + rows - 1) / rows) * ((a.N + bn - 1) / bn); };
    // (rows that start between 128-byte lines cost the narrow tiles, which read more per product: 769 x 2200 x 2576 takes
    // 13.9 us with 256 channels, 11.3 with pairs' 128 and 12.5 with a single CTA's, 1024 x 1024 x 8192 29.0, 19.1 and 19.0)
    const bool off = (a.ldq | a.ldw) % 128 != 0;
    consider(2, 256, 0, tiles(256, 256), 0.37, 5.9, 0.0);
    consider(2, 128, 0, tiles(256, 128), off ? 0.3 : 0.22, 5.0, 0.0);
    consider(1, 128, 0, tiles(128, 128), off ? 0.36 : 0.22, 4.8, 3.3);
    return best;
}

kt_status launch_linear_fp8_as(int dtype, const LinearFp8& a, const Fp8Shape& s, int sms, int device, void* stream, const char** why) {
    if (s.swap) {
        if (s.BN == 16) return f8_launch<1, 16, true>(dtype, a, s.splits, sms, device, stream, why);
        return f8_launch<1, 32, true>(dtype, a, s.splits, sms, device, stream, why);
    }
    if (s.pair == 1) return f8_launch<1, 128, false>(dtype, a, s.splits, sms, device, stream, why);
    if (s.BN == 128) return f8_launch<2, 128, false>(dtype, a, 1, sms, device, stream, why);
    return f8_launch<2, 256, false>(dtype, a, 1, sms, device, stream, why);
}

kt_status launch_linear_fp8(int dtype, const LinearFp8& a, int sms, int device, void* stream, const char** why) {
    return launch_linear_fp8_as(dtype, a, linear_fp8_shape(a, sms, device), sms, device, stream, why);
}

kt_status linear_fp8_status(void* stream, int* word, const char** why) { return error_word(g_fp8_error, stream, word, why); }

}  // namespace kt
