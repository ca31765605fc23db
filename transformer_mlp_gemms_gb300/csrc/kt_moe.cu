// kt_moe.cu -- a whole mixture-of-experts feed-forward layer for a few tokens, in one kernel.
//
//   logits = x . W_router^T; each token's top_k experts; weight_j from their softmax;
//   y = sum_j weight_j ( act(x . W_up[e_j]^T + b_up[e_j]) . W_down[e_j]^T + b_down[e_j] ) (+ R)
//
// Bound by HBM: a few tokens touch up to top_k experts each, and every touched expert's
// weights have to be read once, for all of its tokens together; each weight then meets 1 to 64
// tokens.  One persistent grid of co-resident blocks goes through four phases with a barrier
// over the grid after each of the first three:
//
//   0  logits: one warp per (token, expert), in pairs of fp32 numbers (below);
//   1  every block finds all tokens' experts for itself (the order is the same everywhere) and
//      takes its share of the up projections: H[pair][f] for each (token, expert) pair;
//   2  its share of the down projections: Z[split][pair][d];
//   3  its share of y: the weighted sum over a token's pairs.
//
// The projections are mma.sync products with the weights as the 16-row operand: 16 weight rows
// (GEGLU: 8 value rows and the 8 gate rows that belong to them) against the expert's tokens as
// columns, 8 at a time.  Streaming weights is the whole cost, so they go from global memory
// straight to the registers that the product reads, with no staging in between: lane (g, q) of
// a warp loads 16 consecutive bytes of row g, and because a sum over k may take its terms in
// any order, those 8 elements serve as the lane's k positions of two products as they are; the
// tokens' operand is loaded with the same permutation.  The 8 warps of a block share a strip of
// 16 rows, each taking every eighth 32 columns, four steps ahead in a register ring that runs
// on across strips; their sums meet in shared memory in warp order.
#include "kt_ops_internal.h"
#include "kt_rows.cuh"

namespace kt {
namespace {

constexpr int kMoeWarps = 8, kMoeThreads = kMoeWarps * 32;
constexpr int kMoeRing = 4;             // steps of weights in flight per warp
constexpr int kMoeStepK = kMoeWarps * 32;  // columns that the warps of a block take per step
constexpr int kMoePairs = KT_MOE_MAX_TOKENS * KT_MOE_MAX_TOP_K;
constexpr int kMoeSplits = 8;           // most splits of a down projection along F

// What every block knows after routing.
struct MoeRoute {
    float weight[kMoePairs];           // of pair t * top_k + j
    short expert[kMoePairs];           // of pair t * top_k + j
    short list[kMoePairs];             // pairs in the order of their experts
    short active[KT_MOE_MAX_EXPERTS];  // the experts that have pairs
    short start[KT_MOE_MAX_EXPERTS + 1];  // of each active expert's pairs in list
    short count[KT_MOE_MAX_EXPERTS];   // pairs per expert
    int n_active;
};

__device__ __forceinline__ uint4 ld_weights(const uint16_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

template <int DT>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    if constexpr (DT == KT_BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Barrier over the grid: every block arrives once on `counter` (zero at the kernel's start) and
// waits until all have.  Bounded: a wait that runs out, or another block's that did, records an
// error and returns false in every thread of the block.
__device__ __forceinline__ bool grid_barrier(unsigned* counter, const MoeParams& p, int* ok_slot) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        atomicAdd(counter, 1u);
        bool ok = true;
        const unsigned long long t0 = global_ns();
        for (unsigned i = 1;; ++i) {
            unsigned v;
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
            if (v >= gridDim.x) break;
            if ((i & 63u) == 0) {
                if (*reinterpret_cast<volatile int*>(p.error) != 0) {
                    ok = false;
                    break;
                }
                if (global_ns() - t0 > p.wait_limit_ns) {
                    atomicCAS(p.error, 0, DEV_TIMEOUT_PRODUCER);
                    ok = false;
                    break;
                }
            }
        }
        __threadfence();
        *ok_slot = ok;
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

template <int DT>
__device__ void moe_logits(const MoeParams& p) {
    const int lane = threadIdx.x & 31;
    const int warps = (int)gridDim.x * kMoeWarps;
    float2* logits = reinterpret_cast<float2*>(p.logits);
    for (int i = (int)blockIdx.x * kMoeWarps + (threadIdx.x >> 5); i < p.T * p.E; i += warps) {
        const int t = i / p.E, e = i % p.E;
        const uint16_t* x = static_cast<const uint16_t*>(p.X) + (int64_t)t * p.ldx;
        const uint16_t* w = static_cast<const uint16_t*>(p.W_router) + (int64_t)e * p.D;
        Pair s = {0.0f, 0.0f};
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
        if (lane == 0) {
            // hi alone where the sum is not finite (lo is then no number)
            const float hi = __fadd_rn(s.hi, s.lo);
            const bool finite = fabsf(s.hi) < __uint_as_float(0x7f800000u);
            logits[i] = finite ? make_float2(hi, __fadd_rn(s.lo, __fsub_rn(s.hi, hi))) : make_float2(s.hi, 0.0f);
        }
    }
}

// Every token's experts and weights, then the pairs by expert.
__device__ void moe_route(const MoeParams& p, MoeRoute& r) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float2* logits = reinterpret_cast<const float2*>(p.logits);
    const int k = p.top_k, E = p.E, pairs = p.T * k;
    constexpr int per = KT_MOE_MAX_EXPERTS / 32;
    for (int t = warp; t < p.T; t += kMoeWarps) {
        float2 v[per];
        uint32_t used = 0;  // this lane's experts e = 32 i + lane that are taken or not there
        bool nan = false;
#pragma unroll
        for (int i = 0; i < per; ++i) {
            const int e = 32 * i + lane;
            v[i] = make_float2(0.0f, 0.0f);
            if (e < E)
                v[i] = __ldcg(&logits[t * E + e]);
            else
                used |= 1u << i;
            nan |= v[i].x != v[i].x;
        }
        nan = __any_sync(0xffffffffu, nan);
        float2 top = make_float2(0.0f, 0.0f);
        float total = 0.0f, mine = 0.0f;  // lane j keeps the j-th choice's term
        for (int j = 0; j < k; ++j) {
            uint32_t bh = 0, bl = 0, bi = 0xffffffffu;
#pragma unroll
            for (int i = 0; i < per; ++i) {
                const uint32_t h = order_key(v[i].x), l = order_key(v[i].y);
                const bool better = bi == 0xffffffffu || h > bh || (h == bh && l > bl);
                if (!((used >> i) & 1u) && better) {
                    bh = h;
                    bl = l;
                    bi = (uint32_t)(32 * i + lane);
                }
            }
            const bool any = bi != 0xffffffffu;
            const uint32_t mh = __reduce_max_sync(0xffffffffu, any ? bh : 0u);
            const uint32_t ml = __reduce_max_sync(0xffffffffu, any && bh == mh ? bl : 0u);
            const uint32_t e = __reduce_min_sync(0xffffffffu, any && bh == mh && bl == ml ? bi : 0xffffffffu);
            float2 chosen = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < per; ++i)
                if (32 * i + lane == (int)e) {
                    chosen = v[i];
                    used |= 1u << i;
                }
            chosen.x = __shfl_sync(0xffffffffu, chosen.x, e & 31u);
            chosen.y = __shfl_sync(0xffffffffu, chosen.y, e & 31u);
            if (j == 0) top = chosen;
            const float term = expf((chosen.x - top.x) + (chosen.y - top.y));
            total += term;
            if (lane == j) {
                mine = term;
                r.expert[t * k + j] = (short)e;
            }
        }
        if (!p.normalize) {
            total = 0.0f;
#pragma unroll
            for (int i = 0; i < per; ++i)
                if (32 * i + lane < E) total += expf((v[i].x - top.x) + (v[i].y - top.y));
            total = warp_add(total);
        }
        if (lane < k) {
            const float w = nan ? __uint_as_float(0x7fffffffu) : mine / total;
            r.weight[t * k + lane] = w;
            if (blockIdx.x == 0) {
                if (p.weights) p.weights[t * k + lane] = w;
                if (p.ids) p.ids[t * k + lane] = r.expert[t * k + lane];
            }
        }
    }
    __syncthreads();
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
    for (int a = warp; a < r.n_active; a += kMoeWarps) {
        const int e = r.active[a];
        int at = r.start[a];
        for (int i = 0; i < pairs; i += 32) {
            const bool is = i + lane < pairs && r.expert[i + lane] == e;
            const uint32_t b = __ballot_sync(0xffffffffu, is);
            if (is) r.list[at + __popc(b & ((1u << lane) - 1u))] = (short)(i + lane);
            at += __popc(b);
        }
    }
    __syncthreads();
}

// One projection of all active experts: items (active expert, strip of 16 weight rows, split
// along K), block b taking items b, b + grid, ...
struct Projection {
    const uint16_t* W;  // [E][rows][K]
    int rows, K;        // weight rows per expert (UP with GEGLU: 2 F), columns
    int strips, splits;
    int split_k;        // columns of a split, a multiple of kMoeStepK
};

template <int DT, int NT, bool UP>
__device__ void moe_project(const MoeParams& p, const MoeRoute& r, const Projection& q, int act, float* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
    const bool gated = UP && act == KT_ACT_GEGLU;
    const int items = r.n_active * q.strips * q.splits;
    const int steps = q.split_k / kMoeStepK;
    const int mine = items > (int)blockIdx.x ? (items - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
    const int total = mine * steps;
    const int kofs = warp * 32 + t4 * 8;  // this lane's columns within a step

    // where an item's rows are: the expert, the strip's first output, the split's first column
    auto locate = [&](int item, int& a, int& f0, int& split) {
        split = item % q.splits;
        const int s = item / q.splits;
        a = s / q.strips;
        f0 = (s % q.strips) * (gated ? 8 : 16);
    };
    // load cursor
    int l_item = (int)blockIdx.x, l_step = 0, l_k = 0, l_end = 0;
    const uint16_t *row0 = nullptr, *row1 = nullptr;  // null: no such row
    auto l_open = [&]() {
        int a, f0, split;
        locate(l_item, a, f0, split);
        const int64_t e = r.active[a];
        const int n0 = f0 + g, n1 = gated ? p.F + f0 + g : f0 + 8 + g;
        const bool v0 = gated ? f0 + g < p.F : n0 < q.rows, v1 = gated ? v0 : n1 < q.rows;
        row0 = v0 ? q.W + (e * q.rows + n0) * q.K : nullptr;
        row1 = v1 ? q.W + (e * q.rows + n1) * q.K : nullptr;
        l_k = split * q.split_k + kofs;
        l_end = min(q.K, (split + 1) * q.split_k);
    };
    uint4 ring[kMoeRing][2];
    auto load = [&](uint4 (&w)[2]) {
        if (l_step == 0) l_open();
        w[0] = w[1] = make_uint4(0u, 0u, 0u, 0u);
        if (l_k < l_end) {
            if (row0) w[0] = ld_weights(row0 + l_k);
            if (row1) w[1] = ld_weights(row1 + l_k);
        }
        l_k += kMoeStepK;
        if (++l_step == steps) {
            l_step = 0;
            l_item += (int)gridDim.x;
        }
    };
    // product cursor
    int item = (int)blockIdx.x, step = 0, a = 0, f0 = 0, split = 0, n = 0, nt = 0, k = 0, k_end = 0, buffer = 0;
    const uint16_t* src[NT];  // the tokens' rows of this lane's column in each tile of 8; null: none
    const int64_t lo_part = UP ? 0 : (int64_t)p.T * p.top_k * p.F;  // from H's first part to its second
    float acc[NT][4];
    auto open = [&]() {
        locate(item, a, f0, split);
        n = r.start[a + 1] - r.start[a];
        nt = (n + 7) / 8;
        k = split * q.split_k + kofs;
        k_end = min(q.K, (split + 1) * q.split_k);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            src[j] = nullptr;
            if (8 * j + g < n) {
                const int pair = r.list[r.start[a] + 8 * j + g];
                src[j] = UP ? static_cast<const uint16_t*>(p.X) + (int64_t)(pair / p.top_k) * p.ldx
                            : p.H + (int64_t)pair * p.F;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
        }
    };
    auto multiply = [&](const uint4 (&w)[2]) {
        if (step == 0) open();
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (j < nt) {
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                const bool in = src[j] != nullptr && k < k_end;
                if (in) x = *reinterpret_cast<const uint4*>(src[j] + k);
                mma16816<DT>(acc[j], w[0].x, w[1].x, w[0].y, w[1].y, x.x, x.y);
                mma16816<DT>(acc[j], w[0].z, w[1].z, w[0].w, w[1].w, x.z, x.w);
                if constexpr (!UP) {
                    if (in) x = *reinterpret_cast<const uint4*>(src[j] + lo_part + k);
                    mma16816<DT>(acc[j], w[0].x, w[1].x, w[0].y, w[1].y, x.x, x.y);
                    mma16816<DT>(acc[j], w[0].z, w[1].z, w[0].w, w[1].w, x.z, x.w);
                }
            }
        }
        k += kMoeStepK;
        if (++step < steps) return;
        // the strip is complete: sums over the warps, in warp order, through shared memory (two
        // buffers in turn, so one barrier per strip)
        float* line = red + buffer * (kMoeWarps * NT * 128);
        buffer ^= 1;
#pragma unroll
        for (int j = 0; j < NT; ++j)
            if (j < nt) {
#pragma unroll
                for (int i = 0; i < 4; ++i) line[(warp * NT * 4 + j * 4 + i) * 32 + lane] = acc[j][i];
            }
        __syncthreads();
        auto sum = [&](int slot, int ln) {
            float v = 0.0f;
#pragma unroll
            for (int wi = 0; wi < kMoeWarps; ++wi) v += line[(wi * NT * 4 + slot) * 32 + ln];
            return v;
        };
        // accumulator i of lane (g, t4): weight row g + 8 (i / 2), token column 2 t4 + i % 2
        const int n_out = nt * (gated ? 64 : 128);
        for (int o = threadIdx.x; o < n_out; o += kMoeThreads) {
            const int ln = o & 31, i = gated ? (o >> 5) & 1 : (o >> 5) & 3, j = gated ? o >> 6 : o >> 7;
            const int col = 8 * j + 2 * (ln & 3) + (i & 1), f = f0 + (ln >> 2) + (gated ? 0 : 8 * (i >> 1));
            if (col >= n || f >= (gated ? p.F : q.rows)) continue;
            const int pair = r.list[r.start[a] + col];
            float v = sum(4 * j + i, ln);
            if constexpr (UP) {
                const int64_t e = r.active[a];
                const uint16_t* b = static_cast<const uint16_t*>(p.b_up);
                float bb[8];
                if (b) {
                    unpack8<DT>(make_uint4(b[e * q.rows + f], 0u, 0u, 0u), bb);
                    v += bb[0];
                }
                f32x2 h = f2(v);
                if (gated) {
                    float gate = sum(4 * j + 2 + i, ln);
                    if (b) {
                        unpack8<DT>(make_uint4(b[e * q.rows + p.F + f], 0u, 0u, 0u), bb);
                        gate += bb[0];
                    }
                    h = f2_mul<true>(h, gelu_erf_f2<true>(f2(gate)));
                } else if (act == KT_ACT_GELU_ERF) {
                    h = gelu_erf_f2<true>(h);
                } else if (act == KT_ACT_GELU_TANH) {
                    h = gelu_tanh_f2<true>(h);
                } else if (act == KT_ACT_GELU_SIGMOID) {
                    h = gelu_sigmoid_f2<true>(h);
                } else if (act == KT_ACT_SILU) {
                    h = silu_f2<true>(h);
                }
                // H in two 16-bit parts: its rounding, and the remainder's (none of an infinity)
                const uint32_t hi = pack2<DT>(h.x, 0.0f) & 0xffffu;
                float back[8];
                unpack8<DT>(make_uint4(hi, 0u, 0u, 0u), back);
                const float rest = fabsf(back[0]) < __uint_as_float(0x7f800000u) ? h.x - back[0] : 0.0f;
                p.H[(int64_t)pair * p.F + f] = (uint16_t)hi;
                p.H[(int64_t)(p.T * p.top_k + pair) * p.F + f] = (uint16_t)(pack2<DT>(rest, 0.0f) & 0xffffu);
            } else {
                p.Z[((int64_t)split * p.T * p.top_k + pair) * p.D + f] = v;
            }
        }
        step = 0;
        item += (int)gridDim.x;
    };
#pragma unroll
    for (int u = 0; u < kMoeRing; ++u)
        if (u < total) load(ring[u]);
    for (int s = 0; s < total; s += kMoeRing) {
#pragma unroll
        for (int u = 0; u < kMoeRing; ++u) {
            if (s + u < total) {
                multiply(ring[u]);
                if (s + u + kMoeRing < total) load(ring[u]);
            }
        }
    }
}

template <int DT, int NT>
__global__ void __launch_bounds__(kMoeThreads, 2) kt_moe_kernel(const MoeParams p, const int act) {
    extern __shared__ float red[];  // [2][warps][NT * 4][32]
    __shared__ MoeRoute route;
    __shared__ int ok;
    // a run that failed is not added to: kt_moe_status clears the word and the counters
    if (threadIdx.x == 0) ok = *reinterpret_cast<volatile int*>(p.error) == 0;
    __syncthreads();
    if (!ok) return;

    moe_logits<DT>(p);
    if (!grid_barrier(p.barriers + 0, p, &ok)) return;
    moe_route(p, route);

    Projection up;
    up.W = static_cast<const uint16_t*>(p.W_up);
    up.rows = p.F_up;
    up.K = p.D;
    up.strips = act == KT_ACT_GEGLU ? (p.F + 7) / 8 : (p.F + 15) / 16;
    up.splits = 1;
    up.split_k = (p.D + kMoeStepK - 1) / kMoeStepK * kMoeStepK;
    moe_project<DT, NT, true>(p, route, up, act, red);
    if (!grid_barrier(p.barriers + 1, p, &ok)) return;

    Projection down;
    down.W = static_cast<const uint16_t*>(p.W_down);
    down.rows = p.D;
    down.K = p.F;
    down.strips = (p.D + 15) / 16;
    // splits along F: the fewest step rounds over the grid, one more step counted per strip for
    // its end
    const int steps = (p.F + kMoeStepK - 1) / kMoeStepK, whole = route.n_active * down.strips;
    int best = 0;
    for (int s = 1; s <= moe_splits(p.T * p.top_k); ++s) {
        const int cost = ((whole * s + (int)gridDim.x - 1) / (int)gridDim.x) * ((steps + s - 1) / s + 1);
        if (s == 1 || cost < best) {
            best = cost;
            down.splits = s;
        }
    }
    down.split_k = (steps + down.splits - 1) / down.splits * kMoeStepK;
    down.splits = (steps * kMoeStepK + down.split_k - 1) / down.split_k;
    moe_project<DT, NT, false>(p, route, down, act, red);
    if (!grid_barrier(p.barriers + 2, p, &ok)) return;

    // y: a thread per 4 columns of a token
    const int quads = p.D / 4;
    for (int i = (int)blockIdx.x * kMoeThreads + threadIdx.x; i < p.T * quads; i += (int)gridDim.x * kMoeThreads) {
        const int t = i / quads, d = 4 * (i % quads);
        float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int j = 0; j < p.top_k; ++j) {
            const int pair = t * p.top_k + j;
            float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int s = 0; s < down.splits; ++s) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(p.Z + ((int64_t)s * p.T * p.top_k + pair) * p.D + d));
                z[0] += v.x;
                z[1] += v.y;
                z[2] += v.z;
                z[3] += v.w;
            }
            if (p.b_down) {
                const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.b_down) +
                                                                (int64_t)route.expert[pair] * p.D + d);
                float b[8];
                unpack8<DT>(make_uint4(w.x, w.y, 0u, 0u), b);
#pragma unroll
                for (int c = 0; c < 4; ++c) z[c] += b[c];
            }
            const float w = route.weight[pair];
#pragma unroll
            for (int c = 0; c < 4; ++c) y[c] = fmaf(w, z[c], y[c]);
        }
        const int64_t at = (int64_t)t * p.D + d;
        if (p.R) {
            const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.R) + at);
            float b[8];
            unpack8<DT>(make_uint4(w.x, w.y, 0u, 0u), b);
#pragma unroll
            for (int c = 0; c < 4; ++c) y[c] += b[c];
        }
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.Y) + at) = make_uint2(pack2<DT>(y[0], y[1]), pack2<DT>(y[2], y[3]));
    }
    // the last block to get here leaves the counters at zero: every block is past every barrier
    __syncthreads();
    if (threadIdx.x == 0 && atomicAdd(p.barriers + 3, 1u) == gridDim.x - 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p.barriers[i] = 0u;
    }
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

template <int DT, int NT>
kt_status launch_moe_t(int act, const MoeParams& p, int sms, void* stream, const char** why) {
    auto kern = kt_moe_kernel<DT, NT>;
    constexpr int smem = 2 * kMoeWarps * NT * 128 * (int)sizeof(float);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    int per_sm = 0;
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kMoeThreads, smem);
    if (e == cudaSuccess && per_sm < 1) e = cudaErrorLaunchOutOfResources;
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(sms * std::min(per_sm, 2)), 1, 1);
        cfg.blockDim = dim3(kMoeThreads, 1, 1);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = static_cast<cudaStream_t>(stream);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeCooperative;  // all blocks resident: they wait for one another
        attr[0].val.cooperative = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, kern, p, act);
    }
    if (e != cudaSuccess) {
        *why = cudaGetErrorString(e);
        return KT_ERR_CUDA;
    }
    return KT_OK;
}

}  // namespace

// Workspace: [barrier counters, error word: 256 bytes][logits][H][Z].
size_t moe_workspace(int64_t T, int64_t D, int64_t F, int64_t E, int64_t top_k) {
    const size_t pairs = (size_t)(T * top_k);
    return 256 + round256((size_t)(T * E) * sizeof(float2)) + round256(2 * pairs * (size_t)F * 2) +
           round256(moe_z_rows(pairs) * (size_t)D * sizeof(float));
}

void moe_carve(MoeParams* p, int64_t max_tokens, void* workspace) {
    unsigned char* w = static_cast<unsigned char*>(workspace);
    p->barriers = reinterpret_cast<unsigned*>(w);
    p->error = reinterpret_cast<int*>(w + 128);
    w += 256;
    p->logits = reinterpret_cast<float*>(w);
    w += round256((size_t)(max_tokens * p->E) * sizeof(float2));
    p->H = reinterpret_cast<uint16_t*>(w);
    w += round256(2 * (size_t)(max_tokens * p->top_k) * (size_t)p->F * 2);
    p->Z = reinterpret_cast<float*>(w);
}

kt_status launch_moe(int act, int dtype, const MoeParams& p, int sms, void* stream, const char** why) {
    // as many 8-token tiles as an expert can get
    if (dtype == KT_BF16) {
        if (p.T <= 8) return launch_moe_t<KT_BF16, 1>(act, p, sms, stream, why);
        if (p.T <= 16) return launch_moe_t<KT_BF16, 2>(act, p, sms, stream, why);
        return launch_moe_t<KT_BF16, 8>(act, p, sms, stream, why);
    }
    if (p.T <= 8) return launch_moe_t<KT_F16, 1>(act, p, sms, stream, why);
    if (p.T <= 16) return launch_moe_t<KT_F16, 2>(act, p, sms, stream, why);
    return launch_moe_t<KT_F16, 8>(act, p, sms, stream, why);
}

}  // namespace kt
