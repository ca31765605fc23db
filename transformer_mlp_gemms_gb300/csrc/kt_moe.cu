// kt_moe.cu -- a whole mixture-of-experts feed-forward layer for a few tokens, in one kernel.
//
//   logits = x . W_router^T; each token's top_k experts; weight_j from their softmax;
//   y = sum_j weight_j ( act(x . W_up[e_j]^T + b_up[e_j]) . W_down[e_j]^T + b_down[e_j] ) (+ R)
//
// Bound by HBM: a few tokens touch up to top_k experts each, and every touched expert's
// weights have to be read once, for all of its tokens together; each weight then meets 1 to 64
// tokens.  One persistent grid of co-resident blocks, one per SM:
//
//   logits    one warp per (token, expert), as pairs of fp32 numbers (below);  grid barrier;
//   routing   every block finds all tokens' experts for itself (the same order everywhere) and
//             lists the (token, expert) pairs by expert;
//   up        its share of the up projections: H[pair][f], pairs in the list's order;
//   down      its share of the down projections: Z[split][pair][d], each expert's once its H is there;
//   y         grid barrier; its share of y: the weighted sum over a token's pairs.
//
// The projections are tcgen05 products with the weights as the 128-row operand (GEGLU: 64 value
// rows and the 64 gate rows that belong to them) and the tokens as the columns: all the tokens in
// the up projection (an expert's own are picked when the sums are read), the expert's rows of H in
// the down projection, once for H's 16-bit rounding and once for the remainder's.  The weights
// come by TMA, 16 KB per stage of a ring that takes the rest of shared memory (100 to 180 KB in
// flight per SM), issued by a thread that waits for nothing but free stages: it runs on from
// the up into the down projections, so the memory is busy while the blocks wait for one another's
// H, and a down projection waits for its own expert's alone (with one wait for all of H, 32 tokens, 2
// of 8 x 1280 x 5120, took 74 us, here 66; 64 tokens, 8 of 16 x 2560 x 2560, 121 and 107).  A
// first form with mma.sync, whose warps took weights from global memory straight to
// registers four steps ahead, spent its time on the tokens' operand and on strip ends: it read
// 1.5 to 1.75 TB/s at every size.  Measured, in us, that form and this one: 1 token, 2 of 8 x 1280 x
// 5120 52 and 32; 9 tokens, 2 of 16 x 1152 x 4304 124 and 52; 64 tokens, 4 of 32 x 1280 x 5120 800
// and 217 (5.8 TB/s).  What remains beside the weights is about 20 us: logits, choices and lists
// (4 to 7), the first weights' latency, the waits for H and for all sums.
#include "kt_ops_internal.h"
#include "kt_rows.cuh"

namespace kt {
namespace {

constexpr int kMoeWarps = 16, kMoeThreads = kMoeWarps * 32;
constexpr int kMoePairs = KT_MOE_MAX_TOKENS * KT_MOE_MAX_TOP_K;
constexpr int kMoeWeightBytes = 128 * 128;  // a stage's weights: 128 rows x 64 columns
constexpr int kMoeMaxStages = 12;
constexpr int kMoeWeightThreads = 2;       // threads that issue the weights' copies, in turn
constexpr int kMoeEpiWarps = 4;             // warps 4-7
constexpr uint32_t kMoeAccCols = 128;       // tensor-memory columns of one accumulator buffer

// What every block knows after routing.
struct MoeRoute {
    float weight[kMoePairs];           // of pair t * top_k + j
    short expert[kMoePairs];           // of pair t * top_k + j
    short list[kMoePairs];             // pairs in the order of their experts
    short place[kMoePairs];            // where a pair stands in list
    short active[KT_MOE_MAX_EXPERTS];  // the experts that have pairs
    short start[KT_MOE_MAX_EXPERTS + 1];  // of each active expert's pairs in list
    short count[KT_MOE_MAX_EXPERTS];   // pairs per expert
    float2 logits[KT_MOE_MAX_EXPERTS]; // scratch of the choices
    int n_active;
    int splits, split_kblocks;         // of the down projections along F
};

// One thread waits until `blocks` blocks have arrived on `counter` (zero at the kernel's start).
// Bounded: a wait that runs out, or another block's that did, records an error and returns false.
__device__ __forceinline__ bool wait_blocks(const unsigned* counter, unsigned blocks, const MoeParams& p) {
    const unsigned long long t0 = global_ns();
    for (unsigned i = 1;; ++i) {
        unsigned v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
        if (v >= blocks) return true;
        if ((i & 63u) == 0) {
            if (*reinterpret_cast<volatile int*>(p.error) != 0) return false;
            if (global_ns() - t0 > p.wait_limit_ns) {
                atomicCAS(p.error, 0, DEV_TIMEOUT_PRODUCER);
                return false;
            }
        }
    }
}

// Barrier over the grid, for all threads of every block; false in all of them after a time-out.
__device__ __forceinline__ bool grid_barrier(unsigned* counter, const MoeParams& p, int* ok_slot) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        atomicAdd(counter, 1u);
        *ok_slot = wait_blocks(counter, gridDim.x, p);
        __threadfence();
    }
    __syncthreads();
    return *ok_slot != 0;
}

// A sum as an unevaluated pair hi + lo of fp32 numbers: the terms are exact fp32 products of two
// 16-bit numbers, and each addition's rounding error is computed and kept (Knuth's two-sum).
// About 48 bits, so that the order of two logits is the order of the exact sums unless these
// agree to that many bits, without the double-precision unit, which this GPU hardly has.
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ void pair_add(Pair& s, float hi, float lo) {
    const float t = __fadd_rn(s.hi, hi), b = __fsub_rn(t, s.hi);
    const float e = __fadd_rn(__fsub_rn(s.hi, __fsub_rn(t, b)), __fsub_rn(hi, b));
    s.hi = t;
    s.lo = __fadd_rn(s.lo, __fadd_rn(e, lo));
}

// The order of fp32 numbers as that of unsigned integers; NaN below everything.
__device__ __forceinline__ uint32_t order_key(float f) {
    if (f != f) return 0u;
    const uint32_t u = __float_as_uint(f + 0.0f);  // -0 counts as 0
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// One logit, by a warp; the result in every lane.
template <int DT>
__device__ __forceinline__ float2 moe_logit(const MoeParams& p, int t, int e) {
    const int lane = threadIdx.x & 31;
    const uint16_t* x = static_cast<const uint16_t*>(p.X) + (int64_t)t * p.ldx;
    const uint16_t* w = static_cast<const uint16_t*>(p.W_router) + (int64_t)e * p.D;
    Pair s = {0.0f, 0.0f};
#pragma unroll 4
    for (int k = lane * 8; k < p.D; k += 256) {
        float a[8], b[8];
        unpack8<DT>(*reinterpret_cast<const uint4*>(x + k), a);
        unpack8<DT>(*reinterpret_cast<const uint4*>(w + k), b);
#pragma unroll
        for (int j = 0; j < 8; ++j) pair_add(s, __fmul_rn(a[j], b[j]), 0.0f);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        pair_add(s, __shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o));
    // hi alone where the sum is not finite (lo is then no number)
    const float hi = __fadd_rn(s.hi, s.lo);
    const bool finite = fabsf(s.hi) < __uint_as_float(0x7f800000u);
    return finite ? make_float2(hi, __fadd_rn(s.lo, __fsub_rn(s.hi, hi))) : make_float2(s.hi, 0.0f);
}

// One token's experts and their weights from its logits, by a warp: lane j < top_k returns the
// j-th choice.
__device__ __forceinline__ void moe_choose(const float2* logits, const MoeParams& p, int& expert, float& weight) {
    const int lane = threadIdx.x & 31, E = p.E, n = (E + 31) / 32;
    constexpr int per = KT_MOE_MAX_EXPERTS / 32;
    float2 v[per];
    uint32_t h[per], l[per], used = 0;  // used: this lane's experts e = 32 i + lane that are taken or not there
    bool nan = false;
#pragma unroll
    for (int i = 0; i < per; ++i) {
        const int e = 32 * i + lane;
        v[i] = make_float2(0.0f, 0.0f);
        if (i < n) {
            if (e < E) v[i] = logits[e];
            nan |= v[i].x != v[i].x;
        }
        if (e >= E) used |= 1u << i;
        h[i] = order_key(v[i].x);
        l[i] = order_key(v[i].y);
    }
    nan = __any_sync(0xffffffffu, nan);
    float2 top = make_float2(0.0f, 0.0f);
    float total = 0.0f, mine = 0.0f;
    expert = 0;
    for (int j = 0; j < p.top_k; ++j) {
        uint32_t bh = 0, bl = 0, bi = 0xffffffffu;
        float2 bv = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < per; ++i) {
            if (i < n && !((used >> i) & 1u) && (bi == 0xffffffffu || h[i] > bh || (h[i] == bh && l[i] > bl))) {
                bh = h[i];
                bl = l[i];
                bi = (uint32_t)(32 * i + lane);
                bv = v[i];
            }
        }
        const bool any = bi != 0xffffffffu;
        const uint32_t mh = __reduce_max_sync(0xffffffffu, any ? bh : 0u);
        const uint32_t ml = __reduce_max_sync(0xffffffffu, any && bh == mh ? bl : 0u);
        const uint32_t e = __reduce_min_sync(0xffffffffu, any && bh == mh && bl == ml ? bi : 0xffffffffu);
        if (bi == e) used |= 1u << (e >> 5);
        const float2 chosen = make_float2(__shfl_sync(0xffffffffu, bv.x, e & 31u), __shfl_sync(0xffffffffu, bv.y, e & 31u));
        if (j == 0) top = chosen;
        const float term = expf((chosen.x - top.x) + (chosen.y - top.y));
        total += term;
        if (lane == j) {
            mine = term;
            expert = (int)e;
        }
    }
    if (!p.normalize) {
        total = 0.0f;
#pragma unroll
        for (int i = 0; i < per; ++i)
            if (i < n && 32 * i + lane < E) total += expf((v[i].x - top.x) + (v[i].y - top.y));
        total = warp_add(total);
    }
    weight = nan ? __uint_as_float(0x7fffffffu) : mine / total;
}

// Logits and choices.  Few of them (up to two logits a warp): every block computes them all and
// nobody waits.  Else each token belongs to one block, which writes its choices to the workspace
// and arrives at the first grid barrier, and all blocks read them.  (With the logits spread over
// all warps of the grid and every block choosing for all tokens, 64 tokens of 32 experts took 20
// us to get here, 13 of them for the choices.)
template <int DT>
__device__ bool moe_choices(const MoeParams& p, MoeRoute& r, int* ok_slot) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, k = p.top_k;
    const auto publish = [&](int t, int e, float w) {
        if (lane < k) {
            if (p.weights) p.weights[t * k + lane] = w;
            if (p.ids) p.ids[t * k + lane] = e;
        }
    };
    float2* logits = r.logits;
    int e;
    float w;
    if (p.T * p.E <= 2 * kMoeWarps) {
        for (int i = warp; i < p.T * p.E; i += kMoeWarps) {
            const float2 v = moe_logit<DT>(p, i / p.E, i % p.E);
            if (lane == 0) logits[i] = v;
        }
        __syncthreads();
        for (int t = warp; t < p.T; t += kMoeWarps) {
            moe_choose(logits + t * p.E, p, e, w);
            if (lane < k) {
                r.expert[t * k + lane] = (short)e;
                r.weight[t * k + lane] = w;
            }
            if (blockIdx.x == 0) publish(t, e, w);
        }
        __syncthreads();
        return true;
    }
    bool any = false;
    for (int t = (int)blockIdx.x; t < p.T; t += (int)gridDim.x) {
        any = true;
        for (int i = warp; i < p.E; i += kMoeWarps) {
            const float2 v = moe_logit<DT>(p, t, i);
            if (lane == 0) logits[i] = v;
        }
        __syncthreads();
        if (warp == 0) {
            moe_choose(logits, p, e, w);
            if (lane < k) p.choices[t * k + lane] = make_float2(__int_as_float(e), w);
            publish(t, e, w);
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        if (any) {
            __threadfence();
            atomicAdd(p.barriers + 0, 1u);
        }
        *ok_slot = wait_blocks(p.barriers + 0, (unsigned)min(p.T, (int)gridDim.x), p);
        __threadfence();
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.T * k; i += kMoeThreads) {
        const float2 c = __ldcg(p.choices + i);
        r.expert[i] = (short)__float_as_int(c.x);
        r.weight[i] = c.y;
    }
    __syncthreads();
    return *ok_slot != 0;
}

// The pairs by expert.
__device__ void moe_route(const MoeParams& p, MoeRoute& r) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = p.E, pairs = p.T * p.top_k;
    for (int e = warp; e < E; e += kMoeWarps) {
        int n = 0;
        for (int i = 0; i < pairs; i += 32) n += __popc(__ballot_sync(0xffffffffu, i + lane < pairs && r.expert[i + lane] == e));
        if (lane == 0) r.count[e] = (short)n;
    }
    __syncthreads();
    if (warp == 0) {
        int n_active = 0, at = 0;
        for (int i = 0; i < E; i += 32) {
            const int n = i + lane < E ? r.count[i + lane] : 0;
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += up;
            }
            const uint32_t has = __ballot_sync(0xffffffffu, n > 0);
            if (n > 0) {
                const int a = n_active + __popc(has & ((1u << lane) - 1u));
                r.active[a] = (short)(i + lane);
                r.start[a] = (short)(at + incl - n);
            }
            n_active += __popc(has);
            at += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) {
            r.n_active = n_active;
            r.start[n_active] = (short)at;
        }
    }
    __syncthreads();
    if (warp == kMoeWarps - 1) {
        // splits of the down projections along F, a lane for each count: the fewest k-blocks in a
        // row on one block, two more counted per item for its start and end
        const int kblocks = (p.F + 63) / 64, whole = r.n_active * ((p.D + 127) / 128), grid = (int)gridDim.x;
        const int s = min(lane + 1, min(moe_splits(pairs), kblocks));
        const int per = (kblocks + s - 1) / s, n = (kblocks + per - 1) / per;
        const unsigned cost = (unsigned)(((whole * n + grid - 1) / grid) * (per + 2));
        const unsigned best = __reduce_min_sync(0xffffffffu, cost);
        const uint32_t who = __ballot_sync(0xffffffffu, cost == best);
        if (lane == __ffs(who) - 1) {
            r.splits = n;
            r.split_kblocks = per;
        }
    }
    for (int a = warp; a < r.n_active; a += kMoeWarps) {
        const int e = r.active[a];
        int at = r.start[a];
        for (int i = 0; i < pairs; i += 32) {
            const bool is = i + lane < pairs && r.expert[i + lane] == e;
            const uint32_t b = __ballot_sync(0xffffffffu, is);
            if (is) {
                const int place = at + __popc(b & ((1u << lane) - 1u));
                r.list[place] = (short)(i + lane);
                r.place[i + lane] = (short)place;
            }
            at += __popc(b);
        }
    }
    __syncthreads();
}

// What the roles of a block share about the projections' items.  Up: (active expert, tile of 128
// weight rows: 128 hidden columns, or 64 with their gates); down: (active expert, tile of 128
// outputs, split along F).  Block b takes every gridDim-th up item from b on; the down items
// start with the block after the last up item's, so that nobody gets both remainders.
struct MoeItems {
    int up_tiles, up_items, up_kblocks, down_tiles, down_items, first_down;
    bool gated;
};
struct MoeItem {
    int a, tile, kb0, kb1, split;
};
__device__ __forceinline__ MoeItems moe_items(const MoeParams& p, const MoeRoute& r, int act) {
    MoeItems m;
    m.gated = act == KT_ACT_GEGLU;
    m.up_tiles = m.gated ? (p.F + 63) / 64 : (p.F + 127) / 128;
    m.up_items = r.n_active * m.up_tiles;
    m.up_kblocks = (p.D + 63) / 64;
    m.down_tiles = (p.D + 127) / 128;
    m.down_items = r.n_active * m.down_tiles * r.splits;
    m.first_down = ((int)blockIdx.x + (int)gridDim.x - m.up_items % (int)gridDim.x) % (int)gridDim.x;
    return m;
}
__device__ __forceinline__ MoeItem moe_item(const MoeParams& p, const MoeRoute& r, const MoeItems& m, bool up, int i) {
    MoeItem it;
    if (up) {
        it.a = i / m.up_tiles;
        it.tile = i % m.up_tiles;
        it.split = 0;
        it.kb0 = 0;
        it.kb1 = m.up_kblocks;
    } else {
        it.split = i % r.splits;
        const int t = i / r.splits;
        it.a = t / m.down_tiles;
        it.tile = t % m.down_tiles;
        it.kb0 = it.split * r.split_kblocks;
        it.kb1 = min((p.F + 63) / 64, it.kb0 + r.split_kblocks);
    }
    return it;
}

struct MoeBars {
    uint64_t full[kMoeMaxStages], empty[kMoeMaxStages], acc_full[2], acc_empty[2], drain;
    uint32_t tmem;
    int abort, ok, failed;
    int stored[kMoeEpiWarps];  // up items whose part of H each epilogue warp has stored
};

// Pairs per group of the down products' columns, for T tokens.
KT_HOST_DEVICE inline int moe_group(int T) { return T <= 8 ? 8 : 16; }

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* tm, uint32_t bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* tm, uint32_t bar, int x, int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

__device__ __forceinline__ void st_release_cta(uint32_t addr, int v) {
    asm volatile("st.release.cta.shared.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ int ld_acquire_cta(uint32_t addr) {
    int v;
    asm volatile("ld.acquire.cta.shared.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr) : "memory");
    return r;
}

template <int DT>
__global__ void __launch_bounds__(kMoeThreads, 1)
    kt_moe_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_up,
                  const __grid_constant__ CUtensorMap tm_down, const __grid_constant__ CUtensorMap tm_h, const MoeParams p,
                  const int act, const int stages, const uint32_t stage_bytes, const uint32_t idesc0) {
    extern __shared__ uint8_t raw[];
    __shared__ MoeRoute route;
    __shared__ __align__(8) MoeBars bars;
    const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u;
    float* exchange = reinterpret_cast<float*>(raw + (ring - smem_u32(raw)) + (size_t)stages * stage_bytes);  // [T][64]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort_flag = &bars.abort;
    auto bar = [](uint64_t& b) { return smem_u32(&b); };
    // a run that failed is not added to: kt_moe_status clears the word and the counters
    // by the last two warps: the first ones' logits start at once
    if (warp == kMoeWarps - 1 && lane == 0) bars.failed = *reinterpret_cast<volatile int*>(p.error);
    if (warp == kMoeWarps - 2 && lane == 0) {
        bars.ok = 1;
        bars.abort = 0;
        for (int q = 0; q < kMoeEpiWarps; ++q) bars.stored[q] = 0;
        for (int s = 0; s < stages; ++s) {
            mbar_init(bar(bars.full[s]), 2);
            mbar_init(bar(bars.empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(bars.acc_full[b]), 1);
            mbar_init(bar(bars.acc_empty[b]), kMoeEpiWarps);
        }
        mbar_init(bar(bars.drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
        prefetch_tmap(&tm_x);
        prefetch_tmap(&tm_up);
        prefetch_tmap(&tm_down);
        prefetch_tmap(&tm_h);
    }
    if (warp == 1) tmem_alloc<1>(smem_u32(&bars.tmem), 2 * kMoeAccCols);
    tc_fence_before();
    const bool ready = moe_choices<DT>(p, route, &bars.ok);  // ends with a barrier of the block
    tc_fence_after();
    if (!ready || bars.failed) {  // the same in every thread
        if (warp == 1) tmem_dealloc<1>(bars.tmem, 2 * kMoeAccCols);
        return;
    }
    moe_route(p, route);
    const uint32_t tmem = bars.tmem;
    const MoeItems m = moe_items(p, route, act);
    const int grid = (int)gridDim.x;
    const uint32_t up_cols = (uint32_t)(p.T + 15) / 16 * 16;  // a product has a multiple of 16 columns
    // the down products' columns: groups of pairs, H's rounding, then the remainder's, of each group
    const int group = moe_group(p.T);

    if ((warp == 0 || warp == 2 || warp == 3) && lane == 0) {
        // ------------------ producers: weights (warps 0 and 3), tokens (warp 2) ------------------
        // a copy costs the thread that issues it about 0.1 us whatever its size: one copy per
        // stage and operand, and the weights' stages dealt to two threads
        const bool weights = warp != 2;
        const uint32_t every = weights ? kMoeWeightThreads : 1, mine = warp == 3 ? 1 : 0;
        uint32_t stage = 0, phase = 0, armed = 0, armed_phase = 0, count = 0;
        bool ok = true;
        int ready = -1;  // the last active expert whose H is known to be there
        for (int ph = 0; ph < 2 && ok; ++ph) {
            const bool up = ph == 0;
            const int n_items = up ? m.up_items : m.down_items;
            for (int i = up ? (int)blockIdx.x : m.first_down; i < n_items && ok; i += grid) {
                const MoeItem it = moe_item(p, route, m, up, i);
                const int e = route.active[it.a], start = route.start[it.a], n = route.start[it.a + 1] - start;
                const int groups = (n + group - 1) / group;
                if (!up && !weights && it.a != ready) {
                    ready = it.a;
                    ok = wait_blocks(p.ready + it.a, (unsigned)m.up_tiles, p);
                    if (!ok) {
                        *abort_flag = 1;
                        break;
                    }
                    asm volatile("fence.proxy.async;" ::: "memory");  // H was stored by other threads; TMA reads it
                }
                for (int kb = it.kb0; kb < it.kb1; ++kb, ++count) {
                    if (count % every == mine) {
                        ok = wait_phase(bar(bars.empty[stage]), phase ^ 1u, abort_flag, p.error, DEV_TIMEOUT_PRODUCER, p.wait_limit_ns);
                        if (!ok) break;
                        const uint32_t full = bar(bars.full[stage]), dst = ring + stage * stage_bytes;
                        if (weights) {
                            mbar_arrive_expect_tx(full, kMoeWeightBytes);
                            tma_load_4d(dst, up ? &tm_up : &tm_down, full, kb * 64, it.tile * (up && m.gated ? 64 : 128), 0, e);
                        } else if (up) {
                            mbar_arrive_expect_tx(full, (uint32_t)(p.T + 7) / 8 * 1024u);
                            tma_load_2d(dst + kMoeWeightBytes, &tm_x, full, kb * 64, 0);
                        } else {
                            mbar_arrive_expect_tx(full, (uint32_t)(groups * group) * 256u);
                            for (int b = 0; b < groups; ++b)
                                tma_load_3d(dst + kMoeWeightBytes + (uint32_t)(b * group) * 256u, &tm_h, full, kb * 64, start + group * b, 0);
                        }
                        armed |= 1u << stage;
                        armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
                    }
                    if (++stage == (uint32_t)stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
        if (*abort_flag) {  // no copy may still be landing in shared memory that is about to be released
            for (int s = 0; s < stages; ++s)
                if (armed & (1u << s)) wait_drain(bar(bars.full[s]), (armed_phase >> s) & 1u, 100000000ull);
        }
    } else if (warp == 1 && lane == 0) {
        // ------------------ one thread issues the products ------------------
        uint32_t stage = 0, phase = 0, t = 0;
        bool ok = true;
        if (p.stall_ns && blockIdx.x == 0)  // the tests' hook: nobody signals this barrier yet
            ok = wait_phase(bar(bars.drain), 0u, abort_flag, p.error, DEV_INJECTED_STALL, p.stall_ns);
        for (int ph = 0; ph < 2 && ok; ++ph) {
            const bool up = ph == 0;
            const int n_items = up ? m.up_items : m.down_items;
            for (int i = up ? (int)blockIdx.x : m.first_down; i < n_items && ok; i += grid, ++t) {
                const MoeItem it = moe_item(p, route, m, up, i);
                const uint32_t cols = up ? up_cols : (uint32_t)((route.start[it.a + 1] - route.start[it.a] + group - 1) / group * group * 2);
                const uint32_t idesc = idesc0 | ((cols >> 3) << 17), buf = t & 1u, d = tmem + buf * kMoeAccCols;
                ok = wait_phase(bar(bars.acc_empty[buf]), ((t >> 1) & 1u) ^ 1u, abort_flag, p.error, DEV_TIMEOUT_MMA, p.wait_limit_ns);
                tc_fence_after();
                for (int kb = it.kb0; kb < it.kb1 && ok; ++kb) {
                    ok = wait_phase(bar(bars.full[stage]), phase, abort_flag, p.error, DEV_TIMEOUT_MMA, p.wait_limit_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t base = ring + stage * stage_bytes;
                    const uint64_t ad = smem_desc(base, 16u, 1024u), bd = smem_desc(base + kMoeWeightBytes, 16u, 1024u);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f16(d, ad + (uint64_t)(2 * k), bd + (uint64_t)(2 * k), idesc, kb > it.kb0 || k > 0);
                    mma_commit(bar(bars.empty[stage]));
                    if (++stage == (uint32_t)stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (ok) mma_commit(bar(bars.acc_full[buf]));
            }
        }
        if (!ok) {  // no product may still be running when tensor memory is freed
            mma_commit(bar(bars.drain));
            wait_drain(bar(bars.drain), 0u, 100000000ull);
        }
    } else if (warp >= 4 && warp < 4 + kMoeEpiWarps) {
        // ------------------ epilogue: lane = weight row ------------------
        const int q = warp & 3, pairs = p.T * p.top_k;
        const uint32_t lanes = (uint32_t)(q * 32) << 16;
        uint32_t t = 0;
        bool live = true;
        for (int ph = 0; ph < 2 && live; ++ph) {
            const bool up = ph == 0;
            const int n_items = up ? m.up_items : m.down_items;
            for (int i = up ? (int)blockIdx.x : m.first_down; i < n_items; i += grid, ++t) {
                const MoeItem it = moe_item(p, route, m, up, i);
                const int64_t e = route.active[it.a];
                const int start = route.start[it.a], n = route.start[it.a + 1] - start;
                const uint32_t buf = t & 1u, d = tmem + lanes + buf * kMoeAccCols;
                const bool gate = up && m.gated && q >= 2;  // these rows are gates: value rows' lanes take them over
                const int f = up ? (m.gated ? it.tile * 64 + 32 * (q & 1) : it.tile * 128 + 32 * q) + lane : it.tile * 128 + 32 * q + lane;
                const bool in = f < (up ? p.F : p.D);
                float bias = 0.0f;
                if (up && p.b_up && in) {
                    float b[8];
                    unpack8<DT>(make_uint4(static_cast<const uint16_t*>(p.b_up)[e * p.F_up + (gate ? p.F : 0) + f], 0u, 0u, 0u), b);
                    bias = b[0];
                }
                const bool got = wait_phase(bar(bars.acc_full[buf]), (t >> 1) & 1u, abort_flag, p.error, DEV_TIMEOUT_EPILOGUE, p.wait_limit_ns);
                if (!epi_all<kMoeEpiWarps>(got)) {
                    live = false;
                    break;
                }
                tc_fence_after();
                // rolled loops, one column at a time: this code runs from a cold instruction cache (the
                // weights have swept it out of L2 since the last call), and with 8 columns unrolled
                // the first item's epilogue alone took 11 us
                if (!up) {
#pragma unroll 1
                    for (int c = 0; c < n; ++c) {
                        const uint32_t at = d + (uint32_t)(c / group * group + c);
                        uint32_t z = tmem_ld1(at), rest = tmem_ld1(at + group);
                        tmem_wait_ld_only();
                        asm volatile("" : "+r"(z), "+r"(rest)::"memory");
                        if (in) p.Z[((int64_t)it.split * pairs + start + c) * p.D + f] = __uint_as_float(z) + __uint_as_float(rest);
                    }
                } else {
                    float* gates = exchange + 32 * (q & 1) + lane;
                    if (gate) {
#pragma unroll 1
                        for (int c = 0; c < n; ++c) {
                            uint32_t z = tmem_ld1(d + (uint32_t)(route.list[start + c] / p.top_k));
                            tmem_wait_ld_only();
                            asm volatile("" : "+r"(z)::"memory");
                            gates[c * 64] = __uint_as_float(z) + bias;
                        }
                    }
                    if (m.gated) epi_bar_sync<kMoeEpiWarps>();
                    if (!gate) {
#pragma unroll 1
                        for (int c = 0; c < n; ++c) {
                            uint32_t z = tmem_ld1(d + (uint32_t)(route.list[start + c] / p.top_k));
                            tmem_wait_ld_only();
                            asm volatile("" : "+r"(z)::"memory");
                            const float v = __uint_as_float(z) + bias;
                            f32x2 h = f2(m.gated ? gates[c * 64] : v);
                            if (m.gated || act == KT_ACT_GELU_ERF) h = gelu_erf_f2<true>(h);
                            else if (act == KT_ACT_GELU_TANH) h = gelu_tanh_f2<true>(h);
                            else if (act == KT_ACT_GELU_SIGMOID) h = gelu_sigmoid_f2<true>(h);
                            else if (act == KT_ACT_SILU) h = silu_f2<true>(h);
                            if (m.gated) h.x = __fmul_rn(v, h.x);
                            // H in two 16-bit parts, as the products' operands have 16 bits: its rounding, and
                            // the remainder's (none of an infinity).  f16: 22 bits.  bf16: 16, and the outputs
                            // of 1280 x 5120 are 2.4e-6 of their norm off for that, with one part 1.6e-3; a third
                            // part would take half as many bytes and columns again for what their own
                            // rounding, 2^-9, hides.
                            const uint32_t hi = pack2<DT>(h.x, 0.0f) & 0xffffu;
                            float back[8];
                            unpack8<DT>(make_uint4(hi, 0u, 0u, 0u), back);
                            const float rest = fabsf(back[0]) < __uint_as_float(0x7f800000u) ? h.x - back[0] : 0.0f;
                            if (in) {
                                p.H[(int64_t)(start + c) * p.F + f] = (uint16_t)hi;
                                p.H[(int64_t)(pairs + start + c) * p.F + f] = (uint16_t)(pack2<DT>(rest, 0.0f) & 0xffffu);
                            }
                        }
                    }
                }
                tc_fence_before();
                if (up && m.gated) epi_bar_sync<kMoeEpiWarps>();  // the gates have been read
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(bars.acc_empty[buf]));
                    if (up) st_release_cta(smem_u32(&bars.stored[q]), (int)t + 1);
                }
            }
        }
    } else if (warp == 4 + kMoeEpiWarps) {
        // ------------------ tells all blocks of this one's stored tiles of H ------------------
        // by a warp of its own: the fence waits for the stores, 1 to 2 us while the weights come, and
        // in the epilogue's warps that held up short items (20 tokens, 2 of 16 x 640 x 2560: 46 us, here 41)
        const int mine = m.up_items > (int)blockIdx.x ? (m.up_items - 1 - (int)blockIdx.x) / grid + 1 : 0;
        unsigned long long t0 = global_ns();
        for (int done = 0; done < mine;) {
            const int v = lane < kMoeEpiWarps ? ld_acquire_cta(smem_u32(&bars.stored[lane])) : mine;
            const int upto = __reduce_min_sync(0xffffffffu, v);
            if (upto > done) {
                __syncwarp();  // lanes 0 to 3 have each seen one warp's stores: all of them before lane 0 tells
                __threadfence();
                asm volatile("fence.proxy.async;" ::: "memory");
                if (lane == 0)
                    for (int j = done; j < upto; ++j) atomicAdd(p.ready + ((int)blockIdx.x + j * grid) / m.up_tiles, 1u);
                done = upto;
                t0 = global_ns();
            } else {
                __nanosleep(40);
            }
            const bool late = global_ns() - t0 > 2 * p.wait_limit_ns;
            if (late) {
                atomicCAS(p.error, 0, DEV_TIMEOUT_EPILOGUE);
                *abort_flag = 1;
            }
            if (__any_sync(0xffffffffu, late || *abort_flag != 0)) break;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc<1>(tmem, 2 * kMoeAccCols);
    }
    if (*abort_flag) return;
    if (!grid_barrier(p.barriers + 1, p, &bars.ok)) return;
    // no block waits for an expert's H any more
    if (blockIdx.x == 0 && (int)threadIdx.x < route.n_active) p.ready[threadIdx.x] = 0u;

    // y: 8 lanes per 4 columns of a token, each adding up every eighth (choice, split), so that
    // the loads are in flight together; warps dealt out to the blocks in turn
    const int quads = p.D / 4, pairs = p.T * p.top_k, parts = p.top_k * route.splits, sub = lane >> 2;
    const int last = p.T * quads;
    for (int w = warp * grid + (int)blockIdx.x; w * 4 < last; w += grid * kMoeWarps) {
        const int i = min(w * 4 + (lane & 3), last - 1), t = i / quads, d = 4 * (i % quads);
        float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
        for (int c = sub; c < parts; c += 8) {
            const int j = c / route.splits, s = c % route.splits, pair = t * p.top_k + j;
            const float4 v = __ldcg(reinterpret_cast<const float4*>(p.Z + ((int64_t)s * pairs + route.place[pair]) * p.D + d));
            const float wt = route.weight[pair];
            float b[8] = {};
            if (p.b_down && s == 0) {
                const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.b_down) +
                                                                (int64_t)route.expert[pair] * p.D + d);
                unpack8<DT>(make_uint4(u.x, u.y, 0u, 0u), b);
            }
            y[0] = fmaf(wt, v.x + b[0], y[0]);
            y[1] = fmaf(wt, v.y + b[1], y[1]);
            y[2] = fmaf(wt, v.z + b[2], y[2]);
            y[3] = fmaf(wt, v.w + b[3], y[3]);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) y[c] += __shfl_xor_sync(0xffffffffu, y[c], o);
        }
        if (sub == 0 && w * 4 + (lane & 3) < last) {
            const int64_t at = (int64_t)t * p.D + d;
            if (p.R) {
                const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.R) + at);
                float b[8];
                unpack8<DT>(make_uint4(u.x, u.y, 0u, 0u), b);
#pragma unroll
                for (int c = 0; c < 4; ++c) y[c] += b[c];
            }
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.Y) + at) = make_uint2(pack2<DT>(y[0], y[1]), pack2<DT>(y[2], y[3]));
        }
    }
    // the last block to get here leaves the counters at zero: every block is past every barrier
    __syncthreads();
    if (threadIdx.x == 0 && atomicAdd(p.barriers + 2, 1u) == gridDim.x - 1) {
#pragma unroll
        for (int i = 0; i < 3; ++i) p.barriers[i] = 0u;
    }
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

template <int DT>
kt_status launch_moe_t(int act, const MoeParams& p, int sms, int device, void* stream, const char** why) {
    auto kern = kt_moe_kernel<DT>;
    const int group = moe_group(p.T);
    // a stage: the weights, then the larger of the up product's columns (all tokens) and the down
    // product's (an expert's pairs, two parts each)
    const uint32_t stage = kMoeWeightBytes + (uint32_t)((p.T + group - 1) / group * group) * 256u;
    const int fixed = 1024 + p.T * 64 * (int)sizeof(float);
    const int room = kSmemBudget - (int)sizeof(MoeRoute) - (int)sizeof(MoeBars) - 64;
    const int stages = std::min(kMoeMaxStages, (room - fixed) / (int)stage);
    const int smem = fixed + stages * (int)stage;
    alignas(64) CUtensorMap tx, tu, td, th;
    const bool gated = act == KT_ACT_GEGLU;
    const uint64_t D = p.D, F = p.F, E = p.E, T = p.T, pairs = T * p.top_k;
    const uint64_t dx[2] = {D, T}, sx[1] = {2 * (uint64_t)p.ldx};
    const uint32_t bx[2] = {64, (uint32_t)(T + 7) / 8 * 8};
    const uint64_t du[4] = {D, F, gated ? 2u : 1u, E}, su[3] = {2 * D, 2 * D * F, 2 * D * (uint64_t)p.F_up};
    const uint32_t bu[4] = {64, gated ? 64u : 128u, gated ? 2u : 1u, 1};
    const uint64_t dd[4] = {F, D, 1, E}, sd[3] = {2 * F, 2 * D * F, 2 * D * F};
    const uint32_t bd[4] = {64, 128, 1, 1};
    const uint64_t dh[3] = {F, pairs, 2}, sh[2] = {2 * F, 2 * F * pairs};
    const uint32_t bh[3] = {64, (uint32_t)group, 2};
    if (!encode_tmap_nd(&tx, p.X, DT, 2, dx, sx, bx, 128, why) || !encode_tmap_nd(&tu, p.W_up, DT, 4, du, su, bu, 128, why) ||
        !encode_tmap_nd(&td, p.W_down, DT, 4, dd, sd, bd, 128, why) || !encode_tmap_nd(&th, p.H, DT, 3, dh, sh, bh, 128, why))
        return KT_ERR_CUDA;
    static SmemOptIn opt_in;
    cudaError_t e = opt_in(kern, room, device);
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)sms, 1, 1);
        cfg.blockDim = dim3(kMoeThreads, 1, 1);
        cfg.dynamicSmemBytes = (size_t)smem;
        cfg.stream = static_cast<cudaStream_t>(stream);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeCooperative;  // all blocks resident: they wait for one another
        attr[0].val.cooperative = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, kern, tx, tu, td, th, p, act, stages, stage, make_idesc(DT, 0, 128, 1));
    }
    if (e != cudaSuccess) {
        *why = cudaGetErrorString(e);
        return KT_ERR_CUDA;
    }
    return KT_OK;
}

}  // namespace

// Workspace: [barrier counters, error word: 256 bytes][a counter per active expert][choices][H][Z].
size_t moe_workspace(int64_t T, int64_t D, int64_t F, int64_t top_k) {
    const size_t pairs = (size_t)(T * top_k);
    return kMoeControlBytes + round256(pairs * sizeof(float2)) + round256(2 * pairs * (size_t)F * 2) +
           round256(moe_z_rows((int)pairs) * (size_t)D * sizeof(float));
}

void moe_carve(MoeParams* p, int64_t max_tokens, void* workspace) {
    unsigned char* w = static_cast<unsigned char*>(workspace);
    p->barriers = reinterpret_cast<unsigned*>(w);
    p->error = reinterpret_cast<int*>(w + 128);
    p->ready = reinterpret_cast<unsigned*>(w + 256);
    w += kMoeControlBytes;
    p->choices = reinterpret_cast<float2*>(w);
    w += round256((size_t)(max_tokens * p->top_k) * sizeof(float2));
    p->H = reinterpret_cast<uint16_t*>(w);
    w += round256(2 * (size_t)(max_tokens * p->top_k) * (size_t)p->F * 2);
    p->Z = reinterpret_cast<float*>(w);
}

kt_status launch_moe(int act, int dtype, const MoeParams& p, int sms, int device, void* stream, const char** why) {
    return dtype == KT_BF16 ? launch_moe_t<KT_BF16>(act, p, sms, device, stream, why) : launch_moe_t<KT_F16>(act, p, sms, device, stream, why);
}

}  // namespace kt
