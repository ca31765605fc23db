// kt_matmul.cu -- products of 16-bit matrices in whichever order their operands lie in memory, for the
// training step of a feed-forward block:
//
//   C[M][N] = round(A . B^T (+ bias)),  A: [M][K] or, a_mn, [K][M];  B: [N][K] or, b_mn, [K][N]
//
// A linear layer is A = X, B = W; its gradient dX = dY W has B = W by its other side (b_mn), and
// dW = dY^T X both operands by theirs.  GATED (kt_glu_forward): B holds F value rows, then F gate rows;
// a tile takes value and gate rows of the same columns, so that its epilogue has both and stores
// h = value * act(gate), and p = [value | gate] where a backward pass will want it.
//
// The structure is kt_gemm.cuh's with both operands free in their order: TMA copies of 64-deep
// steps into a ring in shared memory (K-major boxes of 64 columns, or boxes of 64 rows along K and 64
// columns, both under the 128-byte swizzle), tcgen05.mma into one of two fp32 accumulators, and eight
// epilogue warps.  One CTA per tile of 128 rows or a pair per 256 (cta_group::2); persistent, the
// tiles in bands of kBand tile rows so that what runs at a time shares its operands in L2.
//   warp 0: copies of A, and each step's byte count; warp 10: copies of B; warp 1: products;
//   warps 2-9: epilogue.
// SPLIT: few tiles with long sums: a cluster per tile, each CTA with its share of the steps; the fp32 sums meet
// in the cluster's shared memory, added in the order of the ranks.
// SHARED (the gradients): both products of a backward pass in one launch, dW's tiles and dX's, on pairs.  Whole
// rounds of tiles go one to a pair; the steps of the tiles that are left, of both products, are dealt out
// evenly before them, so that every pair ends at the same time.  A tile whose steps fall to several pairs is
// summed by the last of them to finish, from fp32 partial sums in the workspace, in the order of the steps, while
// the products of the whole tiles are already running.
//
// Every wait is bounded: one that runs out leaves an error word and NaN in the elements that the call
// could not compute.
#include "kt_ops_internal.h"
#include "kt_gemm.cuh"
#include "kt_matmul.cuh"

namespace kt {

__device__ int g_matmul_error;

namespace {

constexpr int kMmThreads = 11 * 32;
constexpr int kMmEpi = 8;
constexpr uint32_t kMmABytes = 128 * 128;  // one step of 128 rows

struct MmProduct {
    int M, N;                 // of the output (GATED: N = F)
    int BN, tiles_m, tiles_n, kblocks;
    int a_mn, b_mn;
    uint32_t idesc, b_bytes;  // b_bytes: one step of a CTA's share of B
    int rounds;               // SHARED: whole rounds of tiles
    int left;                 // SHARED: tiles after them
};
struct MmParams {
    MmProduct of[2];          // SHARED: two, else the first
    int stages, act, has_p;
    uint32_t stage_bytes;
    const void* bias;
    // SHARED: the steps of the tiles left, of both products, and the pairs that they are dealt to
    int steps, sharers;
    float* partials;          // [sharers][2][2 CTAs][128][BN]
    int* counters;            // [tiles left, of both products][2 CTAs], zero before the launch
    unsigned long long wait_limit_ns, stall_ns;
};

// A run of steps of one tile, for a CTA or pair.
struct MmItem {
    int product, tile, kb0, kb1;
    int slot;                 // SHARED: where the partial sums of a part of a tile go (of this pair's two), or -1: a whole tile
};

// The items of unit `unit` of `units`, in order: every role of the CTA (or pair) walks through the same ones.
template <bool SHARED>
struct MmWalk {
    const MmParams& p;
    int unit, units, product = 0, round = 0, at = -1, end = 0, first = 0;
    __device__ __forceinline__ MmWalk(const MmParams& q, int u, int n) : p(q), unit(u), units(n) {}
    __device__ __forceinline__ bool next(MmItem& it) {
        if constexpr (!SHARED) {
            it = {0, unit + round * units, 0, p.of[0].kblocks, -1};
            ++round;
            return it.tile < p.of[0].tiles_m * p.of[0].tiles_n;
        } else {
            if (at < 0) {
                at = first = unit < p.sharers ? (int)((int64_t)p.steps * unit / p.sharers) : 0;
                end = unit < p.sharers ? (int)((int64_t)p.steps * (unit + 1) / p.sharers) : 0;
            }
            if (at >= end) {
                for (; product < 2; ++product, round = 0)
                    if (round < p.of[product].rounds) {
                        it = {product, unit + round * units, 0, p.of[product].kblocks, -1};
                        ++round;
                        return true;
                    }
                return false;
            }
            const int steps0 = p.of[0].left * p.of[0].kblocks;
            const int i = at >= steps0, kb = p.of[i].kblocks, t = (at - (i ? steps0 : 0)) / kb;
            const int start = t * kb + (i ? steps0 : 0);  // of the tile
            it.product = i;
            it.tile = p.of[i].rounds * units + t;
            it.kb0 = at - start;
            it.kb1 = min(kb, end - start);
            it.slot = it.kb1 - it.kb0 == kb ? -1 : at == first ? 0 : 1;
            at = start + it.kb1;
            return true;
        }
    }
};

// GATED: the activation of 32 gates times their values, packed.
template <int DT, int EPI>
__device__ __forceinline__ void gate32(const float* v, const float* g, uint32_t* w) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const f32x2 h = f2_mul<true>(f2(v[2 * i], v[2 * i + 1]), act_f2<EPI, true>(f2(g[2 * i], g[2 * i + 1])));
        w[i] = pack2<DT>(h.x, h.y);
    }
}

template <int DT>
__device__ __forceinline__ void pack32(const float* v, uint32_t* w) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack2<DT>(v[2 * i], v[2 * i + 1]);
}

template <int DT, int PAIR, bool GATED, bool SPLIT, bool SHARED>
__global__ void __launch_bounds__(kMmThreads, 1)
    kt_matmul_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmG, const __grid_constant__ CUtensorMap tmX,
                     const __grid_constant__ MmParams p) {
    static_assert(!(SPLIT && (GATED || PAIR == 2)), "a split tile is one CTA's, not gated");
    static_assert(!SHARED || (PAIR == 2 && !GATED && !SPLIT), "shared steps are pairs', of plain products");
    // SHARED: tmV, tmG and tmX are the second product's maps of A, B and C
    extern __shared__ uint8_t raw[];
    uint8_t* const at = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t base = smem_u32(at);
    const uint32_t stage_bytes = p.stage_bytes;
    const uint32_t staging = base + (uint32_t)p.stages * stage_bytes;  // two 2 KB buffers per epilogue warp
    const uint32_t bars = staging + kMmEpi * 4096u;
    const uint32_t bar_full = bars, bar_empty = bars + 64u, bar_accf = bars + 128u, bar_acce = bars + 144u, bar_drain = bars + 160u,
                   bar_stall = bars + 168u;
    uint32_t* const words = reinterpret_cast<uint32_t*>(at + (bars - base) + 176u);
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(words + 1);

    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (uniform for the compiler)
    const unsigned long long limit = p.wait_limit_ns;
    const uint32_t rank = PAIR == 2 ? (cluster_ctarank() & 1u) : 0u;
    const int splits = SPLIT ? (int)cluster_size() : 1, part = SPLIT ? (int)cluster_ctarank() : 0;
    const bool leader = rank == 0;
    const int unit0 = (int)blockIdx.x / (PAIR * splits), units = (int)gridDim.x / (PAIR * splits);
    auto walk = [&]() { return MmWalk<SHARED>(p, unit0, units); };
    auto share = [&](MmItem& it) {  // SPLIT: this CTA's share of the steps
        if constexpr (SPLIT) {
            it.kb1 = (int)((int64_t)p.of[0].kblocks * (part + 1) / splits);
            it.kb0 = (int)((int64_t)p.of[0].kblocks * part / splits);
        }
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(bar_full + 8u * s, 1);
            mbar_init(bar_empty + 8u * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_accf + 8u * b, 1);
            mbar_init(bar_acce + 8u * b, kMmEpi * PAIR);
        }
        mbar_init(bar_drain, 1);
        mbar_init(bar_stall, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
        prefetch_tmap(&tmC);
    }
    if (warp == 1) tmem_alloc<PAIR>(smem_u32(words), kTmemCols);
    tc_fence_before();
    __syncthreads();
    if (PAIR == 2) cluster_sync_relaxed();  // the other CTA's barriers are initialised before any signal to them
    tc_fence_after();
    const uint32_t tmem = words[0];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // first row of A and first row of B (GATED: value row) of this CTA's part of a tile
    auto origin = [&](const MmItem& it, int& m, int& n) {
        const MmProduct& o = p.of[SHARED ? it.product : 0];
        int tm, tn;
        band_tile(it.tile, o.tiles_m, o.tiles_n, tm, tn);
        m = (tm * PAIR + (int)rank) * 128;
        n = tn * (GATED ? o.BN / 2 : o.BN) + (int)rank * (GATED ? o.BN / 2 / PAIR : o.BN / PAIR);
    };

    if (warp == 0 || warp == 10) {
        // ------------------- copies: one lane issues what the whole warp has in uniform registers -------------------
        const bool a_role = warp == 0;
        const uint32_t one = lane == 0, arm = one && leader;
        uint32_t stage = 0, phase = 0, used = 0, used_phase = 0;
        bool ok = true;
        if (a_role && p.stall_ns && blockIdx.x == 0)  // the tests' hook: nobody signals this barrier
            ok = __all_sync(0xffffffffu, wait_phase(bar_stall, 0, abort_flag, &g_matmul_error, DEV_INJECTED_STALL, p.stall_ns));
        const uint32_t full0 = PAIR == 2 ? mapa_rank(bar_full, 0) : bar_full;
        MmItem it;
        for (auto w = walk(); ok && w.next(it);) {
            share(it);
            const MmProduct& o = p.of[SHARED ? it.product : 0];
            const CUtensorMap *mA = SHARED && it.product ? &tmV : &tmA, *mB = SHARED && it.product ? &tmG : &tmB;
            const bool mn = a_role ? o.a_mn : o.b_mn;
            const uint32_t b_bytes = o.b_bytes, bytes = PAIR * (kMmABytes + b_bytes);
            int m, n;
            origin(it, m, n);
            for (int kb = it.kb0; kb < it.kb1; ++kb) {
                ok = __all_sync(0xffffffffu, wait_turn(bar_empty + 8u * stage, phase ^ 1u, abort_flag, &g_matmul_error, DEV_TIMEOUT_PRODUCER, limit));
                if (!ok) break;
                const uint32_t sA = base + stage * stage_bytes, sB = sA + kMmABytes, fb = full0 + 8u * stage;
                const int k = kb * kAtomK;
                if (a_role) {
                    expect_tx_if(bar_full + 8u * stage, bytes, arm);
                    if (mn) {
                        load_if<PAIR>(sA, mA, fb, m, k, one);
                        load_if<PAIR>(sA + 8192u, mA, fb, m + 64, k, one);
                    } else {
                        load_if<PAIR>(sA, mA, fb, k, m, one);
                    }
                    used |= 1u << stage;
                    used_phase = (used_phase & ~(1u << stage)) | (phase << stage);
                } else if (GATED) {
                    load_if<PAIR>(sB, mB, fb, k, n, one);
                    load_if<PAIR>(sB + b_bytes / 2, mB, fb, k, o.N + n, one);
                } else if (mn) {
                    for (uint32_t j = 0; j < b_bytes; j += 8192u) load_if<PAIR>(sB + j, mB, fb, n + (int)(j / 128u), k, one);
                } else {
                    load_if<PAIR>(sB, mB, fb, k, n, one);
                }
                if (++stage == (uint32_t)p.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (lane == 0) {
            if (*abort_flag) {
                // no copy may still be on its way into memory that is about to be released: the byte
                // counts cover both CTAs' copies, and what was never counted gets 100 us to land
                if (a_role && leader)
                    for (int s = 0; s < p.stages; ++s)
                        if (used & (1u << s)) wait_drain(bar_full + 8u * s, (used_phase >> s) & 1u, 100000000ull);
                const unsigned long long t0 = global_ns();
                while (global_ns() - t0 < 100000ull) __nanosleep(1000);
            }
        }
    } else if (warp == 1) {
        // ------------------- products, likewise -------------------
        if (leader) {
            const uint32_t one = lane == 0, stage16 = stage_bytes >> 4;
            uint32_t stage = 0, phase = 0;
            bool ok = true, any = false;
            int local = 0;
            MmItem it;
            for (auto w = walk(); ok && w.next(it); ++local) {
                share(it);
                const MmProduct& o = p.of[SHARED ? it.product : 0];
                const uint64_t ad0 = smem_desc(base, o.a_mn ? 8192u : 16u, 1024u);
                const uint64_t bd0 = smem_desc(base + kMmABytes, o.b_mn ? 8192u : 16u, 1024u);
                // 16 columns of K further: 32 bytes of a K-major row, 16 rows of an MN-major box
                const uint32_t a_step = o.a_mn ? 128u : 2u, b_step = o.b_mn ? 128u : 2u, idesc = o.idesc;
                const uint32_t buf = local & 1, d = tmem + buf * (uint32_t)kAccSlot;
                ok = __all_sync(0xffffffffu, wait_phase<PAIR == 2>(bar_acce + 8u * buf, ((local >> 1) & 1u) ^ 1u, abort_flag, &g_matmul_error,
                                                                   DEV_TIMEOUT_MMA, limit));
                if (!ok) break;
                tc_fence_after();
                for (int kb = it.kb0; kb < it.kb1; ++kb) {
                    ok = __all_sync(0xffffffffu, wait_turn(bar_full + 8u * stage, phase, abort_flag, &g_matmul_error, DEV_TIMEOUT_MMA, limit));
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t ad = ad0 + stage * stage16, bd = bd0 + stage * stage16;
#pragma unroll
                    for (uint32_t k = 0; k < 4; ++k) mma_if<PAIR, false>(d, ad + k * a_step, bd + k * b_step, idesc, kb > it.kb0 || k > 0, one);
                    any = true;
                    commit_if<PAIR>(bar_empty + 8u * stage, one);
                    if (++stage == (uint32_t)p.stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (ok) commit_if<PAIR>(bar_accf + 8u * buf, one);
            }
            if (!ok && any) {  // no product may still be running when tensor memory is freed
                commit_if<PAIR>(bar_drain, one);
                if (lane == 0) wait_drain(bar_drain, 0u, 100000000ull);
            }
        }
        __syncwarp();
    } else {
        // ------------------- epilogue -------------------
        const int ew = warp - 2, q = warp & 3, half = ew >> 2;  // this warp's lanes of tensor memory, its column groups
        const uint32_t stg = staging + (uint32_t)ew * 4096u;
        uint32_t stores = 0;
        bool ok = true;
        int local = 0;
        MmItem it;
        for (auto walker = walk(); walker.next(it); ++local) {
            const MmProduct& o = p.of[SHARED ? it.product : 0];
            const CUtensorMap* const mC = SHARED && it.product ? &tmX : &tmC;
            const uint32_t buf = local & 1;
            ok = ok && wait_phase(bar_accf + 8u * buf, (local >> 1) & 1u, abort_flag, &g_matmul_error, DEV_TIMEOUT_EPILOGUE, limit);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            int m, n;
            origin(it, m, n);
            if (PAIR == 2) n -= (int)rank * (GATED ? o.BN / 4 : o.BN / 2);  // every column of the tile
            const int y = m + 32 * q;
            const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + buf * (uint32_t)kAccSlot;
            // 32 columns of the accumulator (NaN where there is none), with their bias
            auto columns = [&](uint32_t from, const uint16_t* bias, int col, int limit_col, float* v) {
                uint32_t r[32];
                if (ok) {
                    tmem_ld32(acc + from, r);
                    tmem_wait_ld_only();
                    reg_fence32(r);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) r[i] = 0x7fffffffu;
                }
                if (bias) {
                    bias32<DT>(bias, col, limit_col, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] += __uint_as_float(r[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
                }
            };
            auto store = [&](const CUtensorMap* tm, const uint32_t* w, int col) {
                stage_and_store_packed(tm, stg + (stores++ & 1u) * 2048u, lane, w, col, y, true);
            };
            const uint16_t* bias = static_cast<const uint16_t*>(p.bias);
            if constexpr (SPLIT) {
                // the sums go where the operands were (every product has read them): 32 x 32 units of
                // [4 columns][32 rows], 16 bytes each
                for (int g = half; g < o.BN / 32; g += 2) {
                    uint32_t r[32];
                    if (ok) {
                        tmem_ld32(acc + 32u * g, r);
                        tmem_wait_ld_only();
                        reg_fence32(r);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        st_shared_v4(base + (uint32_t)(4 * g + q) * 4096u + (uint32_t)(i * 512 + lane * 16), ok ? r[4 * i] : 0x7fffffffu,
                                     ok ? r[4 * i + 1] : 0x7fffffffu, ok ? r[4 * i + 2] : 0x7fffffffu, ok ? r[4 * i + 3] : 0x7fffffffu);
                }
            } else if constexpr (GATED) {
                const int share = o.BN / PAIR, hs = share / 2;  // accumulator: per share its value columns, then its gates
                for (int g = half; g < o.BN / 64; g += 2) {
                    const int c = 32 * g, col = n + c;
                    if (col >= o.N || y >= o.M) continue;
                    const uint32_t from = (uint32_t)(c / hs * share + c % hs);
                    float v[32], gt[32];
                    uint32_t w[16];
                    columns(from, bias, col, o.N, v);
                    if (p.has_p) {
                        pack32<DT>(v, w);
                        store(&tmV, w, col);
                    }
                    columns(from + (uint32_t)hs, bias ? bias + o.N : nullptr, col, o.N, gt);
                    if (p.has_p) {
                        pack32<DT>(gt, w);
                        store(&tmG, w, col);
                    }
                    switch (p.act) {
                        case EPI_GELU_ERF: gate32<DT, EPI_GELU_ERF>(v, gt, w); break;
                        case EPI_GELU_TANH: gate32<DT, EPI_GELU_TANH>(v, gt, w); break;
                        case EPI_GELU_SIGMOID: gate32<DT, EPI_GELU_SIGMOID>(v, gt, w); break;
                        case EPI_SILU: gate32<DT, EPI_SILU>(v, gt, w); break;
                        default: gate32<DT, EPI_NONE>(v, gt, w); break;
                    }
                    store(&tmC, w, col);
                }
            } else if (SHARED && it.slot >= 0) {
                // A part of a tile's steps: partial sums into this pair's slot, [16 columns][4 columns][128 rows] of
                // 16 bytes, so that a warp's accesses are 512 consecutive bytes; then the tile's count.
                const size_t half_tile = (size_t)128 * 256;  // floats of a slot of one CTA
                float4* const mine = reinterpret_cast<float4*>(p.partials + ((size_t)(unit0 * 2 + it.slot) * 2 + rank) * half_tile) + 32 * q + lane;
                for (int g = half; g < o.BN / 32; g += 2) {
                    uint32_t r[32];
                    if (ok) {
                        tmem_ld32(acc + 32u * g, r);
                        tmem_wait_ld_only();
                        reg_fence32(r);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) r[i] = 0x7fffffffu;
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        __stcg(mine + (8 * g + i) * 128, make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                                                                     __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3])));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(mapa_rank(bar_acce + 8u * buf, 0));
                // the pairs that have steps of this tile: first .. last
                const int steps0 = p.of[0].left * p.of[0].kblocks, t = it.tile - o.rounds * units;
                const int64_t start = (int64_t)t * o.kblocks + (it.product ? steps0 : 0);
                const int first = (int)(((start + 1) * p.sharers - 1) / p.steps);
                const int last = (int)(((start + o.kblocks) * p.sharers - 1) / p.steps);
                epi_bar_sync<kMmEpi>();  // every warp's sums precede the count
                if (ew == 0 && lane == 0) {
                    __threadfence();
                    const int count = atomicAdd(p.counters + (size_t)(t + (it.product ? p.of[0].left : 0)) * 2 + rank, 1);
                    words[2] = count == last - first;
                    __threadfence();
                }
                epi_bar_sync<kMmEpi>();
                if (words[2]) {
                    const bool starts = (int)((int64_t)p.steps * first / p.sharers) == start;  // the first pair's share begins with this tile
                    const float4* const from = reinterpret_cast<const float4*>(p.partials + rank * half_tile) + 32 * q + lane;
                    for (int g = half; g < o.BN / 32; g += 2) {
                        const int col = n + 32 * g;
                        if (col >= o.N || y >= o.M) continue;
                        float v[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = 0.0f;
                        // three pairs' sums on their way at a time
                        for (int u0 = first; u0 <= last; u0 += 3) {
                            float4 x[3][8];
#pragma unroll
                            for (int j = 0; j < 3; ++j) {
                                const int u = u0 + j;
                                if (u > last) break;
                                const float4* part_of = from + (size_t)(u * 2 + (u == first && !starts)) * 2 * (half_tile / 4) + (size_t)(8 * g) * 128;
#pragma unroll
                                for (int i = 0; i < 8; ++i) x[j][i] = __ldcg(part_of + i * 128);
                            }
#pragma unroll
                            for (int j = 0; j < 3; ++j) {
                                if (u0 + j > last) break;
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    v[4 * i] += x[j][i].x;
                                    v[4 * i + 1] += x[j][i].y;
                                    v[4 * i + 2] += x[j][i].z;
                                    v[4 * i + 3] += x[j][i].w;
                                }
                            }
                        }
                        uint32_t w[16];
                        pack32<DT>(v, w);
                        store(mC, w, col);
                    }
                }
                epi_bar_sync<kMmEpi>();  // words[2] is free for the next tile
            } else {
                for (int g = half; g < o.BN / 32; g += 2) {
                    const int col = n + 32 * g;
                    if (col >= o.N || y >= o.M) continue;
                    float v[32];
                    uint32_t w[16];
                    columns(32u * g, bias, col, o.N, v);
                    pack32<DT>(v, w);
                    store(mC, w, col);
                }
            }
            if constexpr (SHARED) {
                if (it.slot >= 0) continue;  // (handed back above)
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR == 2) mbar_arrive_cluster_relaxed(mapa_rank(bar_acce + 8u * buf, 0));
                else mbar_arrive_relaxed(bar_acce + 8u * buf);
            }
        }
        if constexpr (!SPLIT) {
            if (lane == 0) bulk_wait0();
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (SPLIT) {
        if (*abort_flag)  // no sums from this CTA: NaN in their place, and so in the whole tile
            for (int i = threadIdx.x; i < 128 * p.of[0].BN; i += kMmThreads) reinterpret_cast<uint32_t*>(at)[i] = 0x7fffffffu;
        cluster_sync_all();  // every CTA's sums are there
        if (warp >= 2 && warp < 10) {
            const int ew = warp - 2;
            const uint32_t stg = staging + (uint32_t)ew * 4096u;
            int m, n;
            origin(MmItem{0, unit0, 0, 0, -1}, m, n);
            for (int u = part + splits * ew; u < p.of[0].BN / 8; u += splits * kMmEpi) {  // units of this CTA: every splits-th
                const int q = u & 3, col = n + 32 * (u >> 2), y = m + 32 * q;
                if (col >= p.of[0].N || y >= p.of[0].M) continue;
                float v[32];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t from = base + (uint32_t)u * 4096u + (uint32_t)(i * 512 + lane * 16);
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
                    v[4 * i] = x[0].x;
                    v[4 * i + 1] = x[0].y;
                    v[4 * i + 2] = x[0].z;
                    v[4 * i + 3] = x[0].w;
                }
                if (p.bias) {
                    float b[32];
                    bias32<DT>(p.bias, col, p.of[0].N, b);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] += b[i];
                }
                uint32_t w[16];
                pack32<DT>(v, w);
                stage_and_store_packed(&tmC, stg, lane, w, col, y);
            }
            if (lane == 0) bulk_wait0();
            __syncwarp();
        }
    }
    if (PAIR == 2 || SPLIT) cluster_sync_all();  // neither leaves while another may still signal or read it
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc<PAIR>(tmem, kTmemCols);
    }
}

constexpr int kMmSmem = kSmemBudget;
// what the ring may take: alignment, staging, barriers beside it
constexpr int kMmRing = kMmSmem - 1024 - kMmEpi * 4096 - 256;

template <int DT, int PAIR, bool GATED, bool SPLIT, bool SHARED>
cudaError_t mm_prepare(int device) {
    static SmemOptIn opt_in;
    return opt_in(kt_matmul_kernel<DT, PAIR, GATED, SPLIT, SHARED>, kMmSmem, device);
}

cudaLaunchConfig_t mm_config(int grid, int cluster, void* stream, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(kMmThreads, 1, 1);
    cfg.dynamicSmemBytes = kMmSmem;
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

// Clusters of ks CTAs that the device holds at once; 0 if it cannot say.
int mm_clusters(int ks, int device) {
    static std::atomic<int> known[64][9];  // + 1
    int n = known[device & 63][ks].load(std::memory_order_relaxed) - 1;
    if (n >= 0) return n;
    n = 0;
    if (mm_prepare<KT_F16, 1, false, true, false>(device) == cudaSuccess) {
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t cfg = mm_config(ks, ks, nullptr, attr);
        if (cudaOccupancyMaxActiveClusters(&n, kt_matmul_kernel<KT_F16, 1, false, true, false>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
    }
    known[device & 63][ks].store(n + 1, std::memory_order_relaxed);
    return n;
}

template <int DT, int PAIR, bool GATED, bool SPLIT, bool SHARED>
cudaError_t mm_launch(const CUtensorMap* tm, const MmParams& p, int grid, int cluster, int device, void* stream) {
    cudaError_t e = mm_prepare<DT, PAIR, GATED, SPLIT, SHARED>(device);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = mm_config(grid, cluster, stream, attr);
    return cudaLaunchKernelEx(&cfg, kt_matmul_kernel<DT, PAIR, GATED, SPLIT, SHARED>, tm[0], tm[1], tm[2], tm[3], tm[4], tm[5], p);
}

template <int DT>
cudaError_t mm_dispatch(const CUtensorMap* tm, const MmParams& p, const MatmulShape& s, bool gated, int sms, int device, void* stream) {
    const int tiles = p.of[0].tiles_m * p.of[0].tiles_n;
    if (s.splits > 1) return mm_launch<DT, 1, false, true, false>(tm, p, tiles * s.splits, s.splits, device, stream);
    const int grid = std::min(tiles, sms / s.pair) * s.pair;
    if (gated)
        return s.pair == 2 ? mm_launch<DT, 2, true, false, false>(tm, p, grid, 2, device, stream) : mm_launch<DT, 1, true, false, false>(tm, p, grid, 1, device, stream);
    return s.pair == 2 ? mm_launch<DT, 2, false, false, false>(tm, p, grid, 2, device, stream) : mm_launch<DT, 1, false, false, false>(tm, p, grid, 1, device, stream);
}

int64_t mm_tiles(const Matmul& a, int bn, int pair) {
    const int64_t cols = a.gated ? bn / 2 : bn;
    return (int64_t)((a.M + 128 * pair - 1) / (128 * pair)) * ((a.N + cols - 1) / cols);
}

MmProduct mm_product(int dtype, const Matmul& a, int bn, int pair) {
    MmProduct o = {};
    o.M = a.M;
    o.N = a.N;
    o.BN = bn;
    const int cols = a.gated ? bn / 2 : bn;
    o.tiles_m = (a.M + 128 * pair - 1) / (128 * pair);
    o.tiles_n = (a.N + cols - 1) / cols;
    o.kblocks = (a.K + kAtomK - 1) / kAtomK;
    o.a_mn = a.a_mn;
    o.b_mn = a.b_mn;
    o.idesc = make_idesc(dtype, bn, 128 * pair, !a.b_mn) | (a.a_mn ? 1u << 15 : 0u);
    o.b_bytes = (uint32_t)(bn / pair) * 128u;
    return o;
}

// a [rows][cols] matrix of pitch ld, in boxes of box_rows x box_cols
bool mm_encode(CUtensorMap* m, int dtype, const void* at, int64_t ld, int64_t rows, int64_t columns, int box_rows, int box_cols, int swizzle, const char** why) {
    const uint64_t dims[2] = {(uint64_t)columns, (uint64_t)rows}, strides[1] = {(uint64_t)ld * 2};
    const uint32_t box[2] = {(uint32_t)box_cols, (uint32_t)box_rows};
    return encode_tmap_nd(m, at, dtype, 2, dims, strides, box, swizzle, why);
}
// a product's maps of A, B and C
bool mm_maps(CUtensorMap* a_map, CUtensorMap* b_map, CUtensorMap* c_map, int dtype, const Matmul& a, int bn, int pair, const char** why) {
    const int b_rows = a.gated ? bn / pair / 2 : bn / pair;
    return (a.a_mn ? mm_encode(a_map, dtype, a.A, a.lda, a.K, a.M, 64, 64, 128, why) : mm_encode(a_map, dtype, a.A, a.lda, a.M, a.K, 128, 64, 128, why)) &&
           (a.b_mn ? mm_encode(b_map, dtype, a.B, a.ldb, a.K, a.N, 64, 64, 128, why)
                   : mm_encode(b_map, dtype, a.B, a.ldb, a.gated ? 2 * (int64_t)a.N : a.N, a.K, b_rows, 64, 128, why)) &&
           mm_encode(c_map, dtype, a.C, a.ldc, a.M, a.N, 32, kStoreCols, 64, why);
}

kt_status mm_done(cudaError_t e, const char** why) {
    if (e == cudaSuccess) return KT_OK;
    *why = cudaGetErrorString(e);
    return KT_ERR_CUDA;
}

}  // namespace

MatmulShape matmul_shape(const Matmul& a, int sms, int device) {
    const int steps = (a.K + kAtomK - 1) / kAtomK;
    struct {
        int pair, bn;
        double step, round;
    } const kinds[] = {{2, 256, 0.30, 4.0}, {2, 128, 0.21, 3.5}, {1, 128, 0.25, 3.0}, {1, 64, 0.20, 3.0}};
    MatmulShape best = {};
    double least = 1e30;
    for (const auto& k : kinds) {
        const int64_t t = mm_tiles(a, k.bn, k.pair), units = sms / k.pair, rounds = (t + units - 1) / units;
        const double time = rounds * (steps * k.step + 0.5) + k.round;
        if (time < least) {
            least = time;
            best = {k.pair, k.bn, 1};
        }
        if (a.gated || k.pair == 2) continue;
        for (int ks = 2; ks <= 8; ks *= 2) {
            if (t * ks > sms || steps < 2 * ks || t > mm_clusters(ks, device)) continue;
            const double split = (steps + ks - 1) / ks * k.step + k.round + 2.5;
            if (split < least) {
                least = split;
                best = {1, k.bn, ks};
            }
        }
    }
    return best;
}

kt_status launch_matmul_as(int dtype, const Matmul& a, const MatmulShape& s, int sms, int device, void* stream, const char** why) {
    MmParams p = {};
    p.of[0] = mm_product(dtype, a, s.BN, s.pair);
    p.stage_bytes = kMmABytes + p.of[0].b_bytes;
    p.stages = std::min(8, kMmRing / (int)p.stage_bytes);
    p.act = a.act;
    p.has_p = a.P != nullptr;
    p.bias = a.bias;
    p.wait_limit_ns = a.wait_limit_ns;
    p.stall_ns = a.stall_ns;
    CUtensorMap tm[6];
    if (!mm_maps(tm, tm + 1, tm + 2, dtype, a, s.BN, s.pair, why)) return KT_ERR_CUDA;
    tm[3] = tm[4] = tm[5] = tm[2];
    if (a.P) {
        uint16_t* P = static_cast<uint16_t*>(a.P);
        if (!mm_encode(tm + 3, dtype, P, a.ldp, a.M, a.N, 32, kStoreCols, 64, why) ||
            !mm_encode(tm + 4, dtype, P + a.N, a.ldp, a.M, a.N, 32, kStoreCols, 64, why))
            return KT_ERR_CUDA;
    }
    return mm_done(dtype == KT_BF16 ? mm_dispatch<KT_BF16>(tm, p, s, a.gated, sms, device, stream)
                                    : mm_dispatch<KT_F16>(tm, p, s, a.gated, sms, device, stream),
                   why);
}

kt_status launch_matmul(int dtype, const Matmul& a, int sms, int device, void* stream, const char** why) {
    return launch_matmul_as(dtype, a, matmul_shape(a, sms, device), sms, device, stream, why);
}

size_t gradients_partials() { return (size_t)(kMaxSms / 2) * 2 * 2 * 128 * 256 * sizeof(float); }

kt_status launch_gradients_as(int dtype, const Matmul* a, int count, const int* bn, void* scratch, int sms, int device, void* stream, const char** why) {
    MmParams p = {};
    CUtensorMap tm[6];
    const int units = sms / 2;
    for (int i = 0; i < 2; ++i) {
        if (i >= count) {
            std::memcpy(tm + 3, tm, 3 * sizeof(CUtensorMap));
            continue;
        }
        p.of[i] = mm_product(dtype, a[i], bn[i], 2);
        const int tiles = p.of[i].tiles_m * p.of[i].tiles_n;
        p.of[i].rounds = tiles / units;
        p.of[i].left = tiles % units;
        p.steps += p.of[i].left * p.of[i].kblocks;
        p.stage_bytes = std::max(p.stage_bytes, kMmABytes + p.of[i].b_bytes);
        if (!mm_maps(tm + 3 * i, tm + 3 * i + 1, tm + 3 * i + 2, dtype, a[i], bn[i], 2, why)) return KT_ERR_CUDA;
    }
    if (count == 1) p.of[1].kblocks = 1;
    p.stages = std::min(8, kMmRing / (int)p.stage_bytes);
    p.sharers = std::max(1, std::min(units, p.steps / kGradientsLeast));
    p.counters = static_cast<int*>(scratch);
    p.partials = reinterpret_cast<float*>(static_cast<char*>(scratch) + kGradientsCounters);
    p.wait_limit_ns = a[0].wait_limit_ns;
    p.stall_ns = a[0].stall_ns;
    const int busy = p.of[0].rounds || p.of[1].rounds ? units : p.sharers;
    return mm_done(dtype == KT_BF16 ? mm_launch<KT_BF16, 2, false, false, true>(tm, p, 2 * busy, 2, device, stream)
                                    : mm_launch<KT_F16, 2, false, false, true>(tm, p, 2 * busy, 2, device, stream),
                   why);
}

kt_status launch_gradients(int dtype, const Matmul* a, int count, void* scratch, int sms, int device, void* stream, const char** why) {
    int bn[2];
    for (int i = 0; i < count; ++i) bn[i] = mm_tiles(a[i], 256, 2) < sms / 2 ? 128 : 256;
    return launch_gradients_as(dtype, a, count, bn, scratch, sms, device, stream, why);
}

kt_status matmul_status(void* stream, int* word, const char** why) { return error_word(g_matmul_error, stream, word, why); }

}  // namespace kt
