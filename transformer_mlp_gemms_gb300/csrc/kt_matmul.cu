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
// in the cluster's shared memory, added in an order that the place of the sum alone decides.
// SHARED (gradients): both products of a backward pass in one launch, on pairs, as two lists of tiles, unless each is
// quicker in a launch of its own (few tiles with long sums, which clusters share out more finely).  Either whole tiles are dealt out in turn; or, where that would leave many pairs idle at the end, only whole rounds of
// them are, after the steps of the tiles that are left, which are dealt out evenly.  A tile whose steps fall to several
// pairs is summed by the last of them: the others leave fp32 partial sums in the workspace and raise a flag.
// A pair goes through its share backwards, so that what others wait for comes first and what waits for others comes
// last, and a pair waits for pairs of lower numbers alone, which were launched before it.
//
// Bound by the tensor cores where K is long.  16384 tokens x 1280 x 5120 bf16, a call alone on a cool GPU: linear 118 us,
// 1.82 PFLOP/s; the products of a gated block's gradients 454 us, 1.89 PFLOP/s, the tensor pipe busy 94 % of the time; the
// gated projection 215 us, 2.0 PFLOP/s, and 250 us with p, whose 335 MB pass through the shared memory that the operands
// need too.  Calls in sequence run at the 1.4 to 1.5 GHz that the power cap leaves: 137, 512, 256 and 283 us.  For few
// tokens the weights' bytes and a launch bind (4 x 1280 x 2 5120 in 8 to 9 us, 3 TB/s).
//
// Every wait is bounded: one that runs out leaves an error word and NaN in the elements that the call
// could not compute.
#include "kt_ops_internal.h"
#include "kt_gemm.cuh"
#include "kt_matmul.cuh"

#include <cmath>

namespace kt {

__device__ int g_matmul_error;

namespace {

constexpr int kMmThreads = 11 * 32;
constexpr int kMmEpi = 8;
constexpr uint32_t kMmABytes = 128 * 128;  // one step of 128 rows
constexpr size_t kSlot = 128 * 256;        // partial sums of a CTA

struct MmProduct {
    int M, N;                 // of the output (GATED: N = F)
    int BN, tiles_m, tiles_n, kblocks;
    int a_mn, b_mn;
    uint32_t idesc, b_bytes;  // b_bytes: one step of a CTA's share of B
    int rounds;               // SHARED: whole rounds of tiles (-1: all tiles in turn)
    int left;                 // SHARED: tiles after them
};
struct MmParams {
    MmProduct of[2];          // SHARED: two, else the first
    int stages, atoms, act, has_p;  // atoms: 64-deep steps of K per stage of the ring
    uint32_t stage_bytes;
    uint32_t a_bytes, step_bytes;  // the room of one step of A; the bytes of one step's copies
    const void* bias;
    // SHARED: the steps of the tiles left, of both products, and the pairs that they are dealt to
    int steps, sharers;
    float* partials;          // [sharers][2 CTAs][128][256]
    int* flags;               // [sharers][2 CTAs], zero before the launch
    unsigned long long wait_limit_ns, stall_ns;
};

// A run of steps of one tile, for a CTA or pair.
struct MmItem {
    int product, tile, kb0, kb1;
};

// The items of unit `unit` of `units`, in order: every role of the CTA (or pair) walks through the same ones.
template <bool SHARED>
struct MmWalk {
    const MmParams& p;
    int unit, units, product = 0, round = 0, at, low;
    __device__ __forceinline__ MmWalk(const MmParams& q, int u, int n) : p(q), unit(u), units(n) {
        at = low = 0;
        if (SHARED && u < q.sharers) {
            low = uniform((int)((int64_t)q.steps * u / q.sharers));
            at = uniform((int)((int64_t)q.steps * (u + 1) / q.sharers));
        }
    }
    __device__ __forceinline__ bool next(MmItem& it) {
        if constexpr (!SHARED) {
            it = {0, unit + round * units, 0, p.of[0].kblocks};
            ++round;
            return it.tile < p.of[0].tiles_m * p.of[0].tiles_n;
        } else {
            if (at > low) {  // backwards through this pair's share of steps
                const int steps0 = p.of[0].left * p.of[0].kblocks, i = at > steps0, kb = p.of[i].kblocks;
                const int t = (at - 1 - (i ? steps0 : 0)) / kb, start = t * kb + (i ? steps0 : 0);  // the tile's first step
                it = {i, p.of[i].rounds * units + t, max(low - start, 0), at - start};
                at = max(start, low);
                return true;
            }
            if (p.of[0].rounds < 0) {  // all tiles of both products in turn
                const int tiles0 = p.of[0].tiles_m * p.of[0].tiles_n, t = unit + round * units, i = t >= tiles0;
                ++round;
                it = {i, i ? t - tiles0 : t, 0, p.of[i].kblocks};
                return it.tile < p.of[i].tiles_m * p.of[i].tiles_n;
            }
            for (; product < 2; ++product, round = 0)
                if (round < p.of[product].rounds) {
                    it = {product, unit + round * units, 0, p.of[product].kblocks};
                    ++round;
                    return true;
                }
            return false;
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
__device__ __forceinline__ void gate_any(int act, const float* v, const float* g, uint32_t* w) {
    switch (act) {
        case EPI_GELU_ERF: return gate32<DT, EPI_GELU_ERF>(v, g, w);
        case EPI_GELU_TANH: return gate32<DT, EPI_GELU_TANH>(v, g, w);
        case EPI_GELU_SIGMOID: return gate32<DT, EPI_GELU_SIGMOID>(v, g, w);
        case EPI_SILU: return gate32<DT, EPI_SILU>(v, g, w);
        default: return gate32<DT, EPI_NONE>(v, g, w);
    }
}

template <int DT>
__device__ __forceinline__ void pack32(const float* v, uint32_t* w) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack2<DT>(v[2 * i], v[2 * i + 1]);
}

// A shared tile's columns (of this warp's half of the groups of 32): the other pairs' sums in the order of the steps, then
// this one's from tensor memory.
template <int DT>
__device__ __forceinline__ uint32_t sum_shared(const CUtensorMap* tm, const float4* from, int first, int last, bool ok, uint32_t acc, int half, int cols,
                                            int n, int y, uint32_t stg, uint32_t stores) {
    const int lane = threadIdx.x & 31;
    for (int g = half; 32 * g < cols; g += 2) {
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = ok ? 0.0f : __uint_as_float(0x7fffffffu);
        if (ok) {
            for (int u0 = first; u0 < last; u0 += 3) {  // three pairs' sums on their way at a time
                float4 x[3][8];
#pragma unroll
                for (int j = 0; j < 3; ++j) {
                    if (u0 + j >= last) break;
                    const float4* part_of = from + (size_t)(u0 + j) * 2 * (kSlot / 4) + (size_t)(8 * g) * 128;
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[j][i] = __ldcg(part_of + i * 128);
                }
#pragma unroll
                for (int j = 0; j < 3; ++j) {
                    if (u0 + j >= last) break;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        v[4 * i] += x[j][i].x;
                        v[4 * i + 1] += x[j][i].y;
                        v[4 * i + 2] += x[j][i].z;
                        v[4 * i + 3] += x[j][i].w;
                    }
                }
            }
            uint32_t own[32];
            tmem_ld32(acc + 32u * g, own);
            tmem_wait_ld_only();
            reg_fence32(own);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] += __uint_as_float(own[i]);
        }
        uint32_t w[16];
        pack32<DT>(v, w);
        stage_and_store_packed(tm, stg + (stores++ & 1u) * 2048u, lane, w, n + 32 * g, y, true);
    }
    return stores;
}

template <int DT, int PAIR, bool GATED, bool SPLIT, bool SHARED>
__global__ void __launch_bounds__(kMmThreads, 1)
    kt_matmul_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmG, const __grid_constant__ CUtensorMap tmX,
                     const __grid_constant__ MmParams p) {
    static_assert(!(SPLIT && PAIR == 2), "a split tile is one CTA's");
    static_assert(!SHARED || (PAIR == 2 && !GATED && !SPLIT), "shared steps are pairs', of plain products");
    // SHARED: tmV, tmG and tmX are the second product's maps of A, B and C
    extern __shared__ uint8_t raw[];
    uint8_t* const at = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t base = smem_u32(at);
    const uint32_t stage_bytes = p.stage_bytes, a_bytes = SHARED || PAIR == 2 ? kMmABytes : p.a_bytes;
    const uint32_t staging = base + (uint32_t)p.stages * stage_bytes;  // two 2 KB buffers per epilogue warp
    const uint32_t bars = staging + kMmEpi * 4096u;
    const uint32_t bar_full = bars, bar_empty = bars + 64u, bar_accf = bars + 128u, bar_acce = bars + 144u, bar_drain = bars + 160u,
                   bar_stall = bars + 168u;
    uint32_t* const words = reinterpret_cast<uint32_t*>(at + (bars - base) + 176u);
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(words + 1);

    const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
    const unsigned long long limit = p.wait_limit_ns;
    const uint32_t rank = PAIR == 2 ? (uint32_t)uniform((int)(cluster_ctarank() & 1u)) : 0u;
    const int splits = SPLIT ? uniform((int)cluster_size()) : 1, part = SPLIT ? uniform((int)cluster_ctarank()) : 0;
    const bool leader = rank == 0;
    const int unit0 = (int)blockIdx.x / (PAIR * splits), units = (int)gridDim.x / (PAIR * splits);
    auto walk = [&]() { return MmWalk<SHARED>(p, unit0, units); };
    auto share = [&](MmItem& it) {  // SPLIT: this CTA's share of the steps
        if constexpr (SPLIT) {
            it.kb1 = uniform((int)((int64_t)p.of[0].kblocks * (part + 1) / splits));
            it.kb0 = uniform((int)((int64_t)p.of[0].kblocks * part / splits));
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
    const uint32_t tmem = (uint32_t)uniform((int)words[0]);
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
        const uint32_t full0 = PAIR == 2 ? (uint32_t)uniform((int)mapa_rank(bar_full, 0)) : bar_full;
        MmItem it;
        for (auto w = walk(); ok && w.next(it);) {
            share(it);
            const MmProduct& o = p.of[SHARED ? it.product : 0];
            const CUtensorMap *mA = SHARED && it.product ? &tmV : &tmA, *mB = SHARED && it.product ? &tmG : &tmB;
            const CUtensorMap* const map = a_role ? mA : mB;
            const bool mn = a_role ? o.a_mn : o.b_mn;
            const uint32_t atoms = (uint32_t)p.atoms, operand = a_role ? a_bytes : o.b_bytes, bytes = SHARED ? PAIR * atoms * (kMmABytes + o.b_bytes) : p.step_bytes;
            int m, n;
            origin(it, m, n);
            const int row = a_role ? m : n;
            for (int kb = it.kb0; kb < it.kb1; kb += (int)atoms) {
                ok = __all_sync(0xffffffffu, wait_turn(bar_empty + 8u * stage, phase ^ 1u, abort_flag, &g_matmul_error, DEV_TIMEOUT_PRODUCER, limit));
                if (!ok) break;
                // (a stage may reach past the item's steps, and past K, where zeros are filled in: its products end in time)
                const uint32_t to = base + stage * stage_bytes + (a_role ? 0u : atoms * a_bytes), fb = full0 + 8u * stage;
                const int k = kb * kAtomK;
                if (a_role) expect_tx_if(bar_full + 8u * stage, bytes, arm);
                if (mn) {  // 64 columns each
                    for (uint32_t j = 0; j * 8192u < operand; ++j) load_if<PAIR>(to + j * atoms * 8192u, map, fb, row + 64 * (int)j, k, one);
                } else {
                    for (uint32_t i = 0; i < atoms; ++i) {
                        if (GATED && !a_role) load3_if<PAIR>(to + i * operand, map, fb, k + 64 * (int)i, n, 0, one);
                        else load_if<PAIR>(to + i * operand, map, fb, k + 64 * (int)i, row, one);
                    }
                }
                used |= 1u << stage;
                used_phase = (used_phase & ~(1u << stage)) | (phase << stage);
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
            bool ok = true;
            int local = 0;
            MmItem it;
            for (auto w = walk(); ok && w.next(it); ++local) {
                share(it);
                const MmProduct& o = p.of[SHARED ? it.product : 0];
                const uint32_t buf = local & 1, d = tmem + buf * (uint32_t)kAccSlot;
                ok = __all_sync(0xffffffffu, wait_phase<PAIR == 2>(bar_acce + 8u * buf, ((local >> 1) & 1u) ^ 1u, abort_flag, &g_matmul_error,
                                                                   DEV_TIMEOUT_MMA, limit));
                if (!ok) break;
                tc_fence_after();
                // The steps of one item, for operands of known order.  K-major: [64-deep step][row], 16 columns of K
                // further are 32 bytes.  MN-major: [64 columns][K], 16 columns of K further are 16 rows of 128 bytes.
                auto steps = [&](auto a_mn, auto b_mn, auto atoms_) {
                    constexpr uint32_t kA = decltype(a_mn)::value ? 128u : 2u, kB = decltype(b_mn)::value ? 128u : 2u, kAtoms = decltype(atoms_)::value;
                    const uint64_t ad0 = smem_desc(base, decltype(a_mn)::value ? kAtoms * 8192u : 16u, 1024u);
                    const uint64_t bd0 = smem_desc(base + kAtoms * a_bytes, decltype(b_mn)::value ? kAtoms * 8192u : 16u, 1024u);
                    const uint32_t idesc = o.idesc, a16 = decltype(a_mn)::value ? 512u : a_bytes >> 4, b16 = decltype(b_mn)::value ? 512u : o.b_bytes >> 4;
                    uint32_t acc = 0;
                    for (int kb = it.kb0; kb < it.kb1; kb += (int)kAtoms) {
                        ok = __all_sync(0xffffffffu, wait_turn(bar_full + 8u * stage, phase, abort_flag, &g_matmul_error, DEV_TIMEOUT_MMA, limit));
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t ad = ad0 + stage * stage16, bd = bd0 + stage * stage16;
#pragma unroll
                        for (uint32_t i = 0; i < kAtoms; ++i) {
                            if (i > 0 && kb + (int)i >= it.kb1) break;
#pragma unroll
                            for (uint32_t k = 0; k < 4; ++k) {
                                mma_if<PAIR, false>(d, ad + i * a16 + k * kA, bd + i * b16 + k * kB, idesc, acc, one);
                                acc = 1;
                            }
                        }
                        commit_if<PAIR>(bar_empty + 8u * stage, one);
                        if (++stage == (uint32_t)p.stages) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                };
                constexpr std::false_type kK{};
                constexpr std::true_type kMN{};
                constexpr std::integral_constant<uint32_t, 1> kOne{};
                constexpr std::integral_constant<uint32_t, 2> kTwo{};
                if constexpr (GATED) {
                    if (p.atoms == 1) steps(kK, kK, kOne);
                    else steps(kK, kK, kTwo);
                } else if (o.a_mn) {
                    steps(kMN, kMN, kTwo);
                } else if (o.b_mn) {
                    steps(kK, kMN, kTwo);
                } else if constexpr (!SHARED) {
                    if (p.atoms == 1) steps(kK, kK, kOne);
                    else steps(kK, kK, kTwo);
                }
                if (ok) commit_if<PAIR>(bar_accf + 8u * buf, one);
            }
            settle<PAIR>(ok, bar_drain, bar_full, stage, phase, (uint32_t)p.stages);
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
            int m, n;
            origin(it, m, n);
            if (PAIR == 2) n -= (int)rank * (GATED ? o.BN / 4 : o.BN / 2);  // every column of the tile
            // The bias of this warp's columns, asked for before its sums are there: eight values per lane, in the order of
            // the groups of 32 (GATED: the values' groups, then the gates').
            uint4 ahead = make_uint4(0u, 0u, 0u, 0u);
            if (!SPLIT && !SHARED && p.bias && lane < 16) {
                const int g = half + 2 * (GATED ? lane >> 2 & 1 : lane >> 2), col = n + 32 * g + 8 * (lane & 3);
                if (32 * g < (GATED ? o.BN / 2 : o.BN) && col < o.N)
                    ahead = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.bias) + (GATED && lane >= 8 ? o.N : 0) + col);
            }
            ok = ok && wait_phase(bar_accf + 8u * buf, (local >> 1) & 1u, abort_flag, &g_matmul_error, DEV_TIMEOUT_EPILOGUE, limit);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            // 32 sums (NaN where there are none), with their bias, the warp's `group`-th
            auto finish = [&](const uint32_t* r, int group, float* v) {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(ok ? r[i] : 0x7fffffffu);
                if (p.bias) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        float b[8];
                        const int from = 4 * group + i / 8;
                        unpack8<DT>(make_uint4(__shfl_sync(0xffffffffu, ahead.x, from), __shfl_sync(0xffffffffu, ahead.y, from),
                                               __shfl_sync(0xffffffffu, ahead.z, from), __shfl_sync(0xffffffffu, ahead.w, from)), b);
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[i + e] += b[e];
                    }
                }
            };
            const int y = m + 32 * q;
            const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + buf * (uint32_t)kAccSlot;
            auto store = [&](const CUtensorMap* tm, const uint32_t* w, int col) {
                stage_and_store_packed(tm, stg + (stores++ & 1u) * 2048u, lane, w, col, y, true);
            };
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
#pragma unroll 1
                for (int g = half; g < o.BN / 64; g += 2) {
                    const int c = 32 * g, col = n + c;
                    if (col >= o.N || y >= o.M) continue;
                    uint32_t rv[32], rg[32];
#pragma unroll
                    for (int i = 0; i < 32; i += 16) {  // (a share may have 48 columns of either)
                        const uint32_t from = acc + (uint32_t)((c + i) / hs * share + (c + i) % hs);
                        tmem_ld16(from, *reinterpret_cast<uint32_t(*)[16]>(rv + i));
                        tmem_ld16(from + (uint32_t)hs, *reinterpret_cast<uint32_t(*)[16]>(rg + i));
                    }
                    tmem_wait_ld_only();
                    reg_fence32(rv);
                    reg_fence32(rg);
                    float v[32], gt[32];
                    uint32_t w[16];
                    finish(rv, g >> 1, v);
                    if (p.has_p) {
                        pack32<DT>(v, w);
                        store(&tmV, w, col);
                    }
                    finish(rg, 2 + (g >> 1), gt);
                    if (p.has_p) {
                        pack32<DT>(gt, w);
                        store(&tmG, w, col);
                    }
                    gate_any<DT>(p.act, v, gt, w);
                    store(&tmC, w, col);
                }
            } else if (SHARED && it.kb1 < o.kblocks) {
                // A part of a tile's steps, not the last: partial sums into this pair's slot, [16 columns][4 columns][128
                // rows] of 16 bytes, so that a warp's accesses are 512 consecutive bytes; then the flag.
                float4* const mine = reinterpret_cast<float4*>(p.partials + (size_t)(unit0 * 2 + (int)rank) * kSlot) + 32 * q + lane;
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
                epi_bar_sync<kMmEpi>();  // every warp's sums precede the flag
                if (ew == 0 && lane == 0 && !(p.stall_ns && blockIdx.x == 0)) {  // (the tests' hook: the stalled block raises none)
                    __threadfence();
                    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p.flags + unit0 * 2 + (int)rank), "r"(1) : "memory");
                }
            } else if (SHARED && it.kb0 > 0) {
                // The last part of a tile's steps: the other pairs' sums in the order of the steps, then this one's.
                const int64_t start = (int64_t)(it.tile - o.rounds * units) * o.kblocks + (it.product ? p.of[0].left * p.of[0].kblocks : 0);
                const int first = (int)(((start + 1) * p.sharers - 1) / p.steps);  // the pair that has the tile's first step
                bool there = ok;
                if (ew == 0 && lane < unit0 - first && there)  // (a lane per pair; there are fewer than 32)
                    there = wait_flag(p.flags + (first + lane) * 2 + (int)rank, abort_flag, &g_matmul_error, limit);
                // A flag that does not come spoils this tile alone: `ok` stays as it is, since the barriers still work and this
                // item's sums were seen.
                const bool whole = epi_all<kMmEpi>(there);
                if (y < o.M)
                    stores = sum_shared<DT>(mC, reinterpret_cast<const float4*>(p.partials + (int)rank * kSlot) + 32 * q + lane, first, unit0, whole, acc,
                                            half, min(o.BN, o.N - n), n, y, stg, stores);
            } else {
#pragma unroll 1
                for (int g = half; g < o.BN / 32; g += 2) {
                    const int col = n + 32 * g;
                    if (col >= o.N || y >= o.M) continue;
                    uint32_t r[32], w[16];
                    tmem_ld32(acc + 32u * g, r);
                    tmem_wait_ld_only();
                    reg_fence32(r);
                    float v[32];
                    finish(r, g >> 1, v);
                    pack32<DT>(v, w);
                    store(mC, w, col);
                }
            }
            tc_fence_before();
            __syncwarp();
            // An accumulator whose sums this warp has not seen is not given back: the barrier does not tell whose arrivals it
            // counts, and two items' from one CTA would let the products overwrite what the other CTA still reads.  The products
            // wait for it in vain then, as long as any wait.
            if (lane == 0 && ok) {
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
            const MmProduct& o = p.of[0];
            const uint16_t* bias = static_cast<const uint16_t*>(p.bias);
            int m, n;
            origin(MmItem{0, unit0, 0, 0}, m, n);
            uint32_t stores = 0;
            // 32 x 32 sums, with their bias
            auto sums = [&](int unit, const uint16_t* b, int col, float* v) {
                uint32_t from = base + (uint32_t)unit * 4096u + (uint32_t)lane * 16u;
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0.0f;
                for (int j0 = 0; j0 < splits; j0 += 2) {  // two CTAs' sums on their way at a time, from this one's on
                    float4 x[2][8];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (j0 + j >= splits) break;
                        const int from_rank = part + j0 + j, at_rank = from_rank < splits ? from_rank : from_rank - splits;
                        const uint32_t at_j = mapa_rank(from, (uint32_t)at_rank);
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[j][i] = ld_cluster4(at_j + (uint32_t)i * 512u);
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (j0 + j >= splits) break;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            v[4 * i] += x[j][i].x;
                            v[4 * i + 1] += x[j][i].y;
                            v[4 * i + 2] += x[j][i].z;
                            v[4 * i + 3] += x[j][i].w;
                        }
                    }
                }
                if (b) {
                    float add[32];
                    bias32<DT>(b, col, o.N, add);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] += add[i];
                }
            };
            auto store = [&](const CUtensorMap* tm, const uint32_t* w, int col, int y) {
                stage_and_store_packed(tm, stg + (stores++ & 1u) * 2048u, lane, w, col, y, true);
            };
            const int units_here = (GATED ? o.BN / 2 : o.BN) / 8;
            for (int u = part + splits * ew; u < units_here; u += splits * kMmEpi) {  // units of this CTA: every splits-th
                const int q = u & 3, col = n + 32 * (u >> 2), y = m + 32 * q;
                if (col >= o.N || y >= o.M) continue;
                float v[32];
                uint32_t w[16];
                sums(u, bias, col, v);
                if constexpr (GATED) {
                    float gt[32];
                    if (p.has_p) {
                        pack32<DT>(v, w);
                        store(&tmV, w, col, y);
                    }
                    sums(u + units_here, bias ? bias + o.N : nullptr, col, gt);
                    if (p.has_p) {
                        pack32<DT>(gt, w);
                        store(&tmG, w, col, y);
                    }
                    gate_any<DT>(p.act, v, gt, w);
                } else {
                    pack32<DT>(v, w);
                }
                store(&tmC, w, col, y);
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
    if (s.splits > 1)
        return gated ? mm_launch<DT, 1, true, true, false>(tm, p, tiles * s.splits, s.splits, device, stream)
                     : mm_launch<DT, 1, false, true, false>(tm, p, tiles * s.splits, s.splits, device, stream);
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
// An operand's map; rows: of the tile in one CTA.
bool mm_operand(CUtensorMap* m, int dtype, const void* at, int64_t ld, bool mn, int64_t outer, int64_t K, int rows, int atoms, const char** why) {
    return mn ? mm_encode(m, dtype, at, ld, K, outer, 64 * atoms, 64, 128, why) : mm_encode(m, dtype, at, ld, outer, K, rows, 64, 128, why);
}
// GATED: the weight as [value, gate][F][K], `rows` of each in one copy
bool mm_gated(CUtensorMap* m, int dtype, const Matmul& a, int rows, const char** why) {
    const uint64_t dims[3] = {(uint64_t)a.K, (uint64_t)a.N, 2}, strides[2] = {(uint64_t)a.ldb * 2, (uint64_t)a.N * (uint64_t)a.ldb * 2};
    const uint32_t box[3] = {64, (uint32_t)rows, 2};
    return encode_tmap_nd(m, a.B, dtype, 3, dims, strides, box, 128, why);
}
// a product's maps of A, B and C
bool mm_maps(CUtensorMap* tm, int dtype, const Matmul& a, int bn, int pair, int atoms, int a_rows, const char** why) {
    const int share = bn / pair;
    return mm_operand(tm, dtype, a.A, a.lda, a.a_mn, a.M, a.K, a_rows, atoms, why) &&
           (a.gated ? mm_gated(tm + 1, dtype, a, share / 2, why) : mm_operand(tm + 1, dtype, a.B, a.ldb, a.b_mn, a.N, a.K, share, atoms, why)) &&
           mm_encode(tm + 2, dtype, a.C, a.ldc, a.M, a.N, 32, kStoreCols, 64, why);
}

kt_status mm_done(cudaError_t e, const char** why) {
    if (e == cudaSuccess) return KT_OK;
    *why = cudaGetErrorString(e);
    return KT_ERR_CUDA;
}

}  // namespace

// How much longer a step takes where rows of an operand start between 128-byte lines.
static double off_lines(const Matmul& a) { return (a.lda | a.ldb) % 64 ? 1.5 : 1.0; }

MatmulShape matmul_shape(const Matmul& a, int sms, int device) {
    const int steps = (a.K + kAtomK - 1) / kAtomK;
    // us per 64-deep step and per launch, measured from 10 to 80 steps (2048 x 1280 x 5120: 27.4, 22.9, 31.8, 31.8 and 43.2 us
    // in this order; 331 x 640 x 2560: 16.1, 13.7, 11.7, 11.1 and 10.7)
    struct {
        int pair, bn, atoms;
        double step, round;
    } const kinds[] = {{2, 256, 1, 0.26, 6.0}, {2, 192, 1, 0.198, 5.6}, {2, 128, 2, 0.17, 5.3}, {1, 128, 2, 0.17, 4.9}, {1, 64, 2, 0.155, 4.5}};
    // bytes per us that L2 brings to all SMs: fewer where rows start between 128-byte lines, and half as many where they start
    // between 32-byte sectors (a step of the second kind takes 0.36 us in 5000 x 1000 x 1000)
    const bool lines = (a.lda | a.ldb) % 64 == 0, sectors = (a.lda | a.ldb) % 16 == 0;
    const double rate = lines ? 23.0e6 : sectors ? 17.0e6 : 12.5e6;
    // nor are the operands sooner there than memory brings them: tiles that keep it busy gain nothing by sharing
    const double bytes = ((double)a.M + (double)a.N * (a.gated ? 2.0 : 1.0)) * a.K * 2.0, brought = bytes / 6.8e6;
    MatmulShape best = {};
    best.us = 1e30;
    for (const auto& k : kinds) {
        if (k.bn == 192 && (a.a_mn || a.b_mn)) continue;  // (MN-major operands come in boxes of 64 columns per CTA)
        const int64_t t = mm_tiles(a, k.bn, k.pair), units = sms / k.pair, rounds = (t + units - 1) / units;
        const int atoms = a.a_mn || a.b_mn ? 2 : k.atoms;
        const double step_bytes = 128.0 * ((k.pair == 1 && !a.a_mn ? std::min(128, a.M) : 128) + k.bn / k.pair);
        const double alone = k.step * (!sectors ? 1.35 : !lines && k.pair == 1 ? 1.25 : 1.0);
        auto step = [&](int64_t ctas) { return std::max(alone, (double)ctas * step_bytes / rate); };
        const double time = std::max(rounds * steps * step(std::min(t, units) * k.pair), brought) + (rounds - 1) * 0.5 + k.round;
        if (time < best.us) best = {k.pair, k.bn, 1, atoms, time};
        if (k.pair == 2) continue;
        for (int ks = 2; ks <= 8; ++ks) {
            if (t * ks > sms || steps < 2 * ks || t > mm_clusters(ks, device)) continue;
            // (a tile's sharing by a cluster: 2.3 to 3.2 us, 4.8 of a gated one)
            const double split = std::max((steps + ks - 1) / ks * step(t * ks), brought) + k.round + (a.gated ? 2.4 + 0.3 * ks : 2.0 + 0.15 * ks);
            if (split < best.us) best = {1, k.bn, ks, atoms, split};
        }
    }
    return best;
}

kt_status launch_matmul_as(int dtype, const Matmul& a, const MatmulShape& s, int sms, int device, void* stream, const char** why) {
    MmParams p = {};
    p.of[0] = mm_product(dtype, a, s.BN, s.pair);
    p.atoms = s.atoms;
    // Copies ask for no rows that A does not have, and few rows leave their room in the ring to the weights (4 x 1280 x
    // 2 5120 11.0 to 13.6 -> 7.8 us, weights from memory).  The products read 128 rows all the same: what lies there, whatever
    // it is, reaches rows of the accumulator that nobody reads.
    const int a_rows = s.pair == 1 && !a.a_mn ? std::min(128, a.M) : 128;
    p.a_bytes = (uint32_t)(a_rows + 7) / 8 * 1024u;
    p.step_bytes = (uint32_t)s.pair * s.atoms * ((uint32_t)a_rows * 128u + p.of[0].b_bytes);
    p.stage_bytes = (uint32_t)s.atoms * (p.a_bytes + p.of[0].b_bytes);
    p.stages = std::min(8, kMmRing / (int)p.stage_bytes);
    p.act = a.act;
    p.has_p = a.P != nullptr;
    p.bias = a.bias;
    p.wait_limit_ns = a.wait_limit_ns;
    p.stall_ns = a.stall_ns;
    CUtensorMap tm[6];
    if (!mm_maps(tm, dtype, a, s.BN, s.pair, s.atoms, a_rows, why)) return KT_ERR_CUDA;
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

size_t gradients_partials() { return (size_t)(kMaxSms / 2) * 2 * kSlot * sizeof(float); }

kt_status launch_gradients_as(int dtype, const Matmul* a, int count, const GradientsShape& s, void* scratch, int sms, int device, void* stream, const char** why) {
    constexpr int kAtoms = 2;
    MmParams p = {};
    CUtensorMap tm[6];
    const int units = sms / 2;
    int tiles = 0;
    for (int i = 0; i < 2; ++i) {
        if (i >= count) {
            std::memcpy(tm + 3, tm, 3 * sizeof(CUtensorMap));
            p.of[i].kblocks = 1;
            continue;
        }
        p.of[i] = mm_product(dtype, a[i], s.bn[i], 2);
        const int n = p.of[i].tiles_m * p.of[i].tiles_n;
        tiles += n;
        p.of[i].rounds = s.share ? n / units : -1;
        p.of[i].left = s.share ? n % units : 0;
        p.steps += p.of[i].left * p.of[i].kblocks;
        p.stage_bytes = std::max(p.stage_bytes, kAtoms * (kMmABytes + p.of[i].b_bytes));
        if (!mm_maps(tm + 3 * i, dtype, a[i], s.bn[i], 2, kAtoms, 128, why)) return KT_ERR_CUDA;
    }
    p.atoms = kAtoms;
    p.stages = std::min(8, kMmRing / (int)p.stage_bytes);
    // a tile falls to 32 pairs at most (a lane each)
    p.sharers = p.steps ? std::max(1, std::min(s.share, std::min(units, p.steps))) : 0;
    for (int i = 0; i < count; ++i)
        if (p.of[i].left) p.sharers = (int)std::min<int64_t>(p.sharers, std::max<int64_t>(1, 30ll * p.steps / p.of[i].kblocks));
    p.flags = static_cast<int*>(scratch);
    p.partials = reinterpret_cast<float*>(static_cast<char*>(scratch) + kGradientsFlags);
    p.wait_limit_ns = a[0].wait_limit_ns;
    p.stall_ns = a[0].stall_ns;
    const int busy = !s.share ? std::min(tiles, units) : p.of[0].rounds + p.of[1].rounds > 0 ? units : p.sharers;
    return mm_done(dtype == KT_BF16 ? mm_launch<KT_BF16, 2, false, false, true>(tm, p, 2 * busy, 2, device, stream)
                                    : mm_launch<KT_F16, 2, false, false, true>(tm, p, 2 * busy, 2, device, stream),
                   why);
}

GradientsShape gradients_shape(const Matmul* a, int count, int sms) {
    constexpr double kSharing = 7.0, kLaunch = 6.0;  // us
    const int units = sms / 2;
    GradientsShape best = {};
    best.us = 1e30;
    for (int mask = 0; mask < 1 << count; ++mask) {
        int64_t tiles[2] = {}, steps[2] = {};
        double step[2] = {}, tile[2] = {};
        GradientsShape s = {};
        for (int i = 0; i < count; ++i) {
            s.bn[i] = mask >> i & 1 ? 128 : 256;
            tiles[i] = mm_tiles(a[i], s.bn[i], 2);
            steps[i] = (a[i].K + kAtomK - 1) / kAtomK;
            // us, measured; a tile of few steps takes its epilogue's time
            step[i] = (s.bn[i] == 256 ? 0.27 : 0.165) * off_lines(a[i]);
            tile[i] = std::max(steps[i] * step[i], s.bn[i] == 256 ? 1.9 : 1.2);
        }
        // in turn: the pair with the most
        double most = 0.0;
        for (int u = 0; u < units; ++u) {
            const int64_t n0 = tiles[0] > u ? (tiles[0] - u - 1) / units + 1 : 0, all = tiles[0] + tiles[1] > u ? (tiles[0] + tiles[1] - u - 1) / units + 1 : 0;
            most = std::max(most, n0 * tile[0] + (all - n0) * tile[1]);
        }
        // shared: the whole rounds, an even share of the rest, the adding of a tile's partial sums (of a pair: 0.9 or 0.5
        // us; the two together are least at the root below), and their way through memory
        double share = kSharing, rest = 0.0, adding = 0.0;
        int64_t left_steps = 0;
        for (int i = 0; i < count; ++i) {
            const int64_t n = tiles[i] % units;
            share += (double)(tiles[i] / units) * tile[i];
            rest += (double)n * tile[i];
            if (n) adding = std::max(adding, (double)steps[i] * (s.bn[i] == 256 ? 0.9 : 0.5));
            left_steps += n * steps[i];
        }
        int sharers = 0;
        if (left_steps) {
            adding /= (double)left_steps;  // of each sharer
            sharers = (int)std::max(1.0, std::min({(double)units, (double)(left_steps / kGradientsLeast), std::sqrt(rest / adding)}));
            share += rest / sharers + adding * sharers;
        }
        for (int k = 0; k < 2; ++k) {
            const double time = k ? share : most;
            if (time + kLaunch < best.us && (!k || sharers)) {
                best = s;
                best.share = k ? sharers : 0;
                best.us = time + kLaunch;
            }
        }
    }
    return best;
}

kt_status launch_gradients(int dtype, const Matmul* a, int count, void* scratch, bool zeroed, int sms, int device, void* stream, const char** why) {
    const GradientsShape both = gradients_shape(a, count, sms);
    // each on its own, where that is quicker: clusters on few tiles with long sums
    MatmulShape each[2];
    double us = -1.5 * (count - 1);  // (the second launch's beginning is hidden)
    for (int i = 0; i < count; ++i) {
        each[i] = matmul_shape(a[i], sms, device);
        us += each[i].us;
    }
    if (both.us <= us) {
        if (both.share && !zeroed) {
            const kt_status s = launch_zero(static_cast<int*>(scratch), stream, why);
            if (s != KT_OK) return s;
        }
        return launch_gradients_as(dtype, a, count, both, scratch, sms, device, stream, why);
    }
    for (int i = 0; i < count; ++i) {
        const kt_status s = launch_matmul_as(dtype, a[i], each[i], sms, device, stream, why);
        if (s != KT_OK) return s;
    }
    return KT_OK;
}

kt_status matmul_status(void* stream, int* word, const char** why) { return error_word(g_matmul_error, stream, word, why); }

}  // namespace kt
