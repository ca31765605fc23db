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
// memory, read as 128-byte broadcasts to the four groups of a warp.  4 x 10240 x 1280 takes 6.7 us, 2
// TB/s: one round of loads whose latency nothing hides, after a launch (10.3 us before the weights were
// loaded ahead and sent for during the kernel before, 7.8 before the warps shared long rows).
constexpr int kDotWarps = 4, kDotTokens = 8;
constexpr int kDotAhead = 4;     // steps of 128 columns in registers
constexpr int kDotChunk = 4096;  // columns of the tokens staged at a time, a multiple of kDotAhead * 128

template <int DT, int KS>
__global__ void __launch_bounds__(kDotWarps * 32) kt_linear_i8_dot_kernel(const LinearI8 p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(16) int8_t sq[];  // [8][chunk]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = lane >> 3, k8 = lane & 7;
    constexpr int kDotRows = kDotWarps / KS * 8, kStep = kDotAhead * 128;
    const int split = warp % KS;  // this warp's steps: every KS-th
    const int n0 = (int)blockIdx.x * kDotRows + warp / KS * 8 + group * 2;
    const int m0 = (int)blockIdx.y * kDotTokens;
    const int tokens = min(kDotTokens, p.M - m0);
    const int8_t* w0 = p.W + (int64_t)min(n0, p.N - 1) * p.ldw;
    const int8_t* w1 = p.W + (int64_t)min(n0 + 1, p.N - 1) * p.ldw;
    // the block's weights start on their way to L2 while the kernel before this one still runs
    // (a prefetch reads nothing)
    for (int i = threadIdx.x; i < kDotRows * ((p.K + 127) / 128); i += kDotWarps * 32) {
        const int n = (int)blockIdx.x * kDotRows + i % kDotRows;
        if (n < p.N) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.W + (int64_t)n * p.ldw + i / kDotRows * 128));
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int acc[2][kDotTokens];
#pragma unroll
    for (int t = 0; t < kDotTokens; ++t) acc[0][t] = acc[1][t] = 0;
    // weights of kDotAhead steps of 128 columns in registers, the next ones' loads in flight behind them
    uint4 a[2][kDotAhead], b[2][kDotAhead];
    auto load = [&](int k, uint4 (&x)[kDotAhead], uint4 (&y)[kDotAhead]) {
#pragma unroll
        for (int u = 0; u < kDotAhead; ++u) {
            x[u] = y[u] = make_uint4(0u, 0u, 0u, 0u);
            if (k + 128 * u + k8 * 16 < p.K) {
                x[u] = *reinterpret_cast<const uint4*>(w0 + k + 128 * u + k8 * 16);
                y[u] = *reinterpret_cast<const uint4*>(w1 + k + 128 * u + k8 * 16);
            }
        }
    };
    load(split * kStep, a[0], b[0]);
    for (int k0 = 0; k0 < p.K; k0 += kDotChunk) {
        const int kc = min(kDotChunk, p.K - k0);
        const int kp = (kc + KS * kStep - 1) / (KS * kStep) * (KS * kStep);  // padded with zeros
        if (k0) __syncthreads();
        for (int k = threadIdx.x * 16; k < kp; k += kDotWarps * 32 * 16) {
            uint4 v[kDotTokens];
#pragma unroll
            for (int t = 0; t < kDotTokens; ++t) {
                v[t] = make_uint4(0u, 0u, 0u, 0u);
                if (t < tokens && k < kc) v[t] = *reinterpret_cast<const uint4*>(p.Q + (int64_t)(m0 + t) * p.ldq + k0 + k);
            }
#pragma unroll
            for (int t = 0; t < kDotTokens; ++t) *reinterpret_cast<uint4*>(sq + t * kp + k) = v[t];
        }
        __syncthreads();
        for (int k = split * kStep; k < kp; k += KS * kStep) {
            load(k0 + k + KS * kStep, a[1], b[1]);
#pragma unroll
            for (int u = 0; u < kDotAhead; ++u) {
                const uint4 x = a[0][u], y = b[0][u];
#pragma unroll
                for (int t = 0; t < kDotTokens; ++t) {
                    const uint4 q = *reinterpret_cast<const uint4*>(sq + t * kp + k + 128 * u + k8 * 16);
                    acc[0][t] = __dp4a((int)x.x, (int)q.x, acc[0][t]);
                    acc[1][t] = __dp4a((int)y.x, (int)q.x, acc[1][t]);
                    acc[0][t] = __dp4a((int)x.y, (int)q.y, acc[0][t]);
                    acc[1][t] = __dp4a((int)y.y, (int)q.y, acc[1][t]);
                    acc[0][t] = __dp4a((int)x.z, (int)q.z, acc[0][t]);
                    acc[1][t] = __dp4a((int)y.z, (int)q.z, acc[1][t]);
                    acc[0][t] = __dp4a((int)x.w, (int)q.w, acc[0][t]);
                    acc[1][t] = __dp4a((int)y.w, (int)q.w, acc[1][t]);
                }
            }
#pragma unroll
            for (int u = 0; u < kDotAhead; ++u) {
                a[0][u] = a[1][u];
                b[0][u] = b[1][u];
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
    if constexpr (KS > 1) {
        __shared__ int2 part[kDotWarps][32];
        part[warp][lane] = make_int2(sum[0], sum[1]);
        __syncthreads();
        if (split != 0) return;
#pragma unroll
        for (int s = 1; s < KS; ++s) {
            const int2 v = part[warp + s][lane];
            sum[0] += v.x;
            sum[1] += v.y;
        }
    }
    if (k8 >= tokens) return;
    const float sx = p.sx[m0 + k8];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int n = n0 + r;
        if (n >= p.N) break;
        // the same roundings as for many tokens: a row's result does not hang on how many are with it
        const float v = fmaf((float)sum[r], sx * p.sw[n], p.bias ? from_bits<DT>(static_cast<const uint16_t*>(p.bias)[n]) : 0.0f);
        static_cast<uint16_t*>(p.Y)[(int64_t)(m0 + k8) * p.ldy + n] = to_bits<DT>(v);
    }
}

// Many tokens: on the tensor cores.  This GPU has no 8-bit integer kind of tcgen05.mma and its
// older integer products run at the rate of four-way dot products, but every int8 is a 16-bit
// float, every product of two is below 2^15, and fp32 holds sums of them exactly up to 2^24: so
// the operands become fp16 on their way into the tensor cores, and the bytes that move stay one
// per element.
//
// One persistent CTA per SM: tiles of 128 tokens x BN channels, or, above 128 tokens, a pair of CTAs
// (cta_group::2) with 128 tokens each and half of the channels' weights; steps of 128 columns
// through a ring of four slots:
//   warps 0-7    tokens: rows of 128 bytes (4 lanes x 32) from global memory, stored as fp16 into
//                tensor memory, where the product reads its first operand (64 columns per slot);
//                as fp16 that operand never passes through shared memory, whose bandwidth, written
//                and read, would bound the kernel;
//   warps 8-15   channels: rows of the weight likewise, into shared memory as fp16, K-major with
//                the 128-byte swizzle.  Both kinds are two groups of four warps that take the
//                steps in turn, so that one's loads arrive while the other converts;
//   warps 16-23  epilogue: accumulator x token scale x channel scale (+ bias), one rounding, parts
//                of 64 columns put together in shared memory, then stored as full lines;
//   warp 24      issues tcgen05.mma (fp16, fp32 accumulators: two buffers, so that a tile's
//                epilogue runs beside the next tile's products, or one of 192 or 256 columns);
//   warps 24-27  of a pair's second CTA tell the first of its full slots.
// Few tiles with long rows: a cluster per tile instead, each CTA with its share of the steps (SPLIT).
// A sum over k may take its terms in any order.  So the bytes of a step go where their lanes' places
// in tensor memory are (lane c of a row's four: words 2 c and 2 c + 1 of every eight; the first 16
// of its 32 bytes in the slot's first half, the others in the second), and the channels follow the
// same order.
// Bound by the products for long rows and many tokens: 8192 x 8192 x 8192 takes 640 us, 1.72
// PFLOP/s (90% of the measured bf16 rate); 16384 x 4304 x 1152 takes 115 us, 1.41 PFLOP/s, where
// a tile's 9 steps are followed by the wait for its accumulator.  The steps there, in us: a thread's
// own row per load (32 wavefronts each) 279, rows shared by four lanes 258, row pointers kept 184,
// two groups in turn 153, pairs 139, 256 channels with twice the ring 131, all parts staged before
// the stores 125, one barrier per step and the products issued from uniform registers 114.
// Four bytes become two pairs of fp16 in five instructions: with the sign bit flipped a byte is
// q + 128, and next to the byte 0x64 it is the fp16 number 1024 + (q + 128); 1152 is subtracted.
constexpr int kTcSlots = 4;   // steps of 128 columns in the ring: 64 tensor-memory columns of tokens each
constexpr int kTcGroups = 2;  // producers of even and of odd steps
constexpr int kTcTokenWarps = 4, kTcChannelWarps = 4, kTcEpiWarps = 8;  // tokens, channels: per group
constexpr int kTcChannel0 = kTcGroups * kTcTokenWarps, kTcEpi0 = kTcChannel0 + kTcGroups * kTcChannelWarps;
constexpr int kTcMmaWarp = kTcEpi0 + kTcEpiWarps, kTcThreads = (kTcMmaWarp + kTcSlots) * 32;
static_assert(kTcSlots % kTcGroups == 0 && kTcEpi0 % 4 == 0, "a group has slots of its own; epilogue warp q: lanes 32 q");
constexpr uint32_t kTcACol = 256;  // tensor-memory column of the first operand's slots, after the accumulators
// A bounded wait that ran out (never in normal operation), until kt_linear_i8_status asks.  The
// elements that the call then cannot compute are stored as NaN, so that its own Y shows it too.
__device__ int g_linear_i8_error;

__device__ __forceinline__ void bytes_to_halves(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u, big = 0x64806480u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    asm("sub.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(big));
    asm("sub.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(big));
}

// 16 rows x 32 columns into tensor memory: lane 4 r + c holds, of every eight columns, 2 c and
// 2 c + 1: of row r in the first two of four registers, of row r + 8 in the other two.
__device__ __forceinline__ void tmem_st_16x32(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// 32 bytes at p: one load where every row starts on a 32-byte boundary, else two.  Bytes at or
// past `left` are zeros (left is a multiple of 16).  Ordinary loads, here and for the few tokens, not
// the read-only path's: this kernel is resident while the one before it may still write Q (or W),
// so they are not read-only for its lifetime, which that path requires; griddepcontrol.wait orders
// ordinary loads.  Not kept in L1, as a CTA reads each byte of a step once (16384 x 4304 x 1152 117.3
// -> 115.4 us).
__device__ __forceinline__ void load32(const int8_t* p, int left, bool wide, uint4& a, uint4& b) {
    a = b = make_uint4(0u, 0u, 0u, 0u);
    if (wide) {
        if (left > 0)
            asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                         : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                         : "l"(p));
    } else {
        if (left > 0) a = *reinterpret_cast<const uint4*>(p);
        if (left > 16) b = *reinterpret_cast<const uint4*>(p + 16);
    }
}

// The product with its first operand in tensor memory (PAIR = 2: 128 rows in each CTA's, half of
// the channels in each CTA's shared memory, at the same places).  The whole warp calls it with the
// same arguments and `leader` in one lane, so that they are in uniform registers, where the
// instruction wants them; a lone thread's were moved there each time, 66 cycles per product.
template <int PAIR>
__device__ __forceinline__ void mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate, uint32_t leader) {
    if constexpr (PAIR == 2)
        asm volatile(
            "{\n\t.reg .pred p, l;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 l, %5, 0;\n\t"
            "@l tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
            "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(leader)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, l;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 l, %5, 0;\n\t"
            "@l tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
            "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(leader)
            : "memory");
}
template <int PAIR>
__device__ __forceinline__ void commit_ta(uint32_t bar, uint32_t leader) {
    if constexpr (PAIR == 2)
        asm volatile(
            "{\n\t.reg .pred l;\n\tsetp.ne.b32 l, %2, 0;\n\t"
            "@l tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
            "h"((unsigned short)3), "r"(leader)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred l;\n\tsetp.ne.b32 l, %1, 0;\n\t"
            "@l tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
            "r"(leader)
            : "memory");
}

template <int BN, int PAIR>
struct TcSmem {
    alignas(1024) uint8_t b[kTcSlots][2][BN / PAIR * 128];  // [channel][64 fp16], 128-byte swizzle
    static constexpr int kParts = (BN + 127) / 128;  // 64-column parts per epilogue warp
    alignas(128) uint8_t out[kTcEpiWarps][kParts][32 * 128];  // 32 rows x 64 columns of the output each
    float2 ch[2][BN];                               // channel scale and bias of the tile
    alignas(8) uint64_t full[kTcSlots], empty[kTcSlots], acc_full[2], acc_empty[2], drain;
    uint32_t tmem;
    int abort;
};

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

// Byte of four columns (chunk) of a row of a split tile's sums, [128][BN] fp32: the chunks swizzled by
// the row's number, so that neither rows over lanes nor columns over lanes share banks.
template <int BN>
__device__ __forceinline__ uint32_t split_at(int row, int chunk) {
    return (uint32_t)(row * BN * 4 + ((chunk ^ (row & 7)) << 4));
}

// SPLIT (PAIR = 1): one tile per cluster of up to 8 CTAs, each with its share of the tile's steps.
// Their sums meet through the cluster's shared memory: each CTA adds its share of the tile's rows
// over all of them, in the order of their ranks, and stores it.
template <int DT, int BN, int PAIR, bool SPLIT>
__global__ void __launch_bounds__(kTcThreads, 1) kt_linear_i8_tc_kernel(const LinearI8 p, int tiles_n, int tiles, uint32_t idesc,
                                                                        int wide_y) {
    extern __shared__ uint8_t raw[];
    using Smem = TcSmem<BN, PAIR>;
    constexpr int kShare = BN / PAIR;  // channels whose weights this CTA stages
    constexpr int kBufs = 256 / BN >= 2 ? 2 : 1;  // accumulators
    Smem& sm = *reinterpret_cast<Smem*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort_flag = &sm.abort;
    const unsigned long long limit = p.wait_limit_ns;
    auto bar = [&](uint64_t& b) { return smem_u32(&b); };
    const int rank = PAIR == 2 ? (int)cluster_ctarank() : 0;
    const int splits = SPLIT ? (int)cluster_size() : 1, part = SPLIT ? (int)cluster_ctarank() : 0;
    const int unit = (int)blockIdx.x / (PAIR * splits), units = (int)gridDim.x / (PAIR * splits);  // CTAs, pairs or clusters
    const int all_steps = (p.K + 127) / 128, step0 = all_steps * part / splits;
    const int steps = all_steps * (part + 1) / splits - step0;  // of a tile, in this CTA
    if (threadIdx.x == 0) {
        for (int s = 0; s < kTcSlots; ++s) {
            // the first CTA of a pair also waits for the other's forwarded arrival
            mbar_init(bar(sm.full[s]), kTcTokenWarps + kTcChannelWarps + (PAIR == 2 && rank == 0 ? 1 : 0));
            mbar_init(bar(sm.empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(sm.acc_full[b]), 1);
            mbar_init(bar(sm.acc_empty[b]), kTcEpiWarps * PAIR);
        }
        mbar_init(bar(sm.drain), 1);
        sm.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
    }
    if (warp == kTcMmaWarp) tmem_alloc<PAIR>(smem_u32(&sm.tmem), kTmemCols);
    tc_fence_before();
    __syncthreads();
    if (PAIR == 2) cluster_sync_relaxed();  // the other CTA's barriers are initialised before any signal to them
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // the first tile's weights start on their way to L2 while the kernel before this one still runs
    // (a prefetch reads nothing)
    if (warp >= kTcChannel0 && warp < kTcEpi0 && unit < tiles) {
        const int n0 = (unit % tiles_n) * BN + rank * kShare, lines = min(steps, 64);
        for (int i = (int)threadIdx.x - kTcChannel0 * 32; i < kShare * lines; i += kTcGroups * kTcChannelWarps * 32)
            if (n0 + i % kShare < p.N)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p.W + (int64_t)(n0 + i % kShare) * p.ldw + (step0 + i / kShare) * 128));
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int mine = tiles > unit ? (tiles - 1 - unit) / units + 1 : 0;
    const int total = mine * steps;  // steps of all this CTA's tiles, in order

    // A producer group's loop over its steps of 128 columns, every kTcGroups-th of the CTA's: N
    // pieces of 32 bytes per thread in registers; when their slot is free, the pieces' first halves are
    // converted into its first 64 columns and the second halves into the others, and the next
    // step's loads go out, to arrive while the other group converts.
    auto produce = [&](auto pieces, int group, auto&& open_tile, auto&& load, auto&& convert) {
        constexpr int N = decltype(pieces)::value;
        uint4 reg[2][N];
        int tile = unit, k = group, opened = -1;
        auto fetch = [&]() {
            while (k >= steps) {
                k -= steps;
                tile += units;
            }
            if (tile != opened) {
                open_tile((tile / tiles_n * PAIR + rank) * 128, (tile % tiles_n) * BN + rank * kShare);
                opened = tile;
            }
            load(reg, (step0 + k) * 128);
            k += kTcGroups;
        };
        uint32_t slot = group, phase = 0;
        if (group < total) fetch();
        for (int s = group; s < total; s += kTcGroups) {
            const bool ok = wait_phase(bar(sm.empty[slot]), phase ^ 1u, abort_flag, &g_linear_i8_error, DEV_TIMEOUT_PRODUCER, limit);
            if (!__all_sync(0xffffffffu, ok)) return;
            convert(reg, slot);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(sm.full[slot]));
            if (s + kTcGroups < total) fetch();
            slot += kTcGroups;
            if (slot >= kTcSlots) {
                slot -= kTcSlots;
                phase ^= 1u;
            }
        }
    };
    const bool wide_q = ((reinterpret_cast<uintptr_t>(p.Q) | (uintptr_t)p.ldq | (uintptr_t)p.K) & 31u) == 0;
    const bool wide_w = ((reinterpret_cast<uintptr_t>(p.W) | (uintptr_t)p.ldw | (uintptr_t)p.K) & 31u) == 0;
    if (warp < kTcChannel0) {
        // ------------------- tokens: bytes from global memory, fp16 to tensor memory -------------------
        const int8_t* row = nullptr;  // row lane / 4 of the warp's 32, at this lane's 32 bytes of a step
        int rows = 0;                 // rows from there on
        const int q = warp & 3;  // rows and tensor-memory lanes 32 q .. + 31
        const int64_t pitch8 = 8 * p.ldq;
        const int k_end = p.K - 32 * (lane & 3);
        produce(
            std::integral_constant<int, 4>{}, warp / kTcTokenWarps,
            [&](int m0, int) {
                const int m = m0 + q * 32 + (lane >> 2);
                rows = p.M - m;
                row = p.Q + (int64_t)m * p.ldq + 32 * (lane & 3);
            },
            [&](uint4 (&r)[2][4], int k) {
#pragma unroll
                for (int j = 0; j < 4; ++j) load32(row + j * pitch8 + k, 8 * j < rows ? k_end - k : 0, wide_q, r[0][j], r[1][j]);
            },
            [&](const uint4 (&r)[2][4], uint32_t slot) {
                tc_fence_after();
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int j = 0; j < 4; j += 2) {  // rows lane / 4 + 8 j and + 8 j + 8 of the warp's 32
                        uint32_t h[16];
#pragma unroll
                        for (int o = 0; o < 2; ++o) {
                            bytes_to_halves(r[half][j + o].x, h[2 * o], h[2 * o + 1]);
                            bytes_to_halves(r[half][j + o].y, h[2 * o + 4], h[2 * o + 5]);
                            bytes_to_halves(r[half][j + o].z, h[2 * o + 8], h[2 * o + 9]);
                            bytes_to_halves(r[half][j + o].w, h[2 * o + 12], h[2 * o + 13]);
                        }
                        tmem_st_16x32(tmem + ((uint32_t)(q * 32 + 8 * j) << 16) + kTcACol + slot * 64u + 32u * half, h);
                    }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
            });
    } else if (warp < kTcEpi0) {
        // ------------------- channels: bytes from global memory, fp16 to shared memory -------------------
        // a warp's 8 rows in the order 0 2 4 6 1 3 5 7, so that the 16 lanes of a store's half
        // touch all banks; this thread's rows are 32 apart
        constexpr int kPieces = kShare / 32;
        const int c = lane & 3, r8 = lane >> 2, n_in = (warp & 3) * 8 + ((r8 & 3) << 1 | r8 >> 2);
        const int8_t* row = nullptr;
        int rows = 0;
        const int64_t pitch32 = 32 * p.ldw;
        const int k_end = p.K - 32 * c;
        // words 2 c and 2 c + 1 of every eight: chunk 2 i + c / 2 of the row, swizzled by its number
        const uint32_t dst = smem_u32(sm.b[0][0]) + (uint32_t)n_in * 128u + 8u * (c & 1);
        const uint32_t first = (uint32_t)((c >> 1) ^ (n_in & 7)) << 4;
        produce(
            std::integral_constant<int, kPieces>{}, (warp - kTcChannel0) / kTcChannelWarps,
            [&](int, int n0) {
                rows = p.N - (n0 + n_in);
                row = p.W + (int64_t)(n0 + n_in) * p.ldw + 32 * c;
            },
            [&](uint4 (&r)[2][kPieces], int k) {
#pragma unroll
                for (int j = 0; j < kPieces; ++j)
                    load32(row + j * pitch32 + k, 32 * j < rows ? k_end - k : 0, wide_w, r[0][j], r[1][j]);
            },
            [&](const uint4 (&r)[2][kPieces], uint32_t slot) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t at = dst + (2u * slot + half) * (uint32_t)(kShare * 128);
#pragma unroll
                    for (int j = 0; j < kPieces; ++j) {
                        const uint32_t w[4] = {r[half][j].x, r[half][j].y, r[half][j].z, r[half][j].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {  // four bytes: two words
                            uint32_t lo, hi;
                            bytes_to_halves(w[i], lo, hi);
                            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at + j * 32u * 128u + (first ^ (uint32_t)(2 * i) << 4)),
                                         "r"(lo), "r"(hi)
                                         : "memory");
                        }
                    }
                }
                fence_async_smem();  // the tensor cores read it through the async proxy
            });
    } else if (warp >= kTcMmaWarp) {
        if (PAIR == 2 && rank == 1) {
            // ------------------- the pair's second CTA: its full slots are told to the first -------------------
            // (an arrival that orders what came before it at cluster scope costs its thread about
            // 0.35 us: one thread per slot)
            if (lane == 0) {
                const int slot = warp - kTcMmaWarp;
                const uint32_t to = mapa_rank(bar(sm.full[slot]), 0u);
                uint32_t phase = 0;
                for (int s = slot; s < total; s += kTcSlots, phase ^= 1u) {
                    if (!wait_phase(bar(sm.full[slot]), phase, abort_flag, &g_linear_i8_error, DEV_TIMEOUT_MMA, limit)) break;
                    tc_fence_after();
                    tc_fence_before();
                    mbar_arrive_cluster(to);
                }
            }
        } else if (warp == kTcMmaWarp) {
            // ------------------- one warp, of which one lane issues the products -------------------
            uint32_t slot = 0, phase = 0;
            const uint32_t leader = lane == 0;
            bool ok = true;
            if (p.stall_ns && unit == 0 && part == 0)  // the tests' hook: nobody signals this barrier yet
                ok = __all_sync(0xffffffffu, wait_phase(bar(sm.drain), 0u, abort_flag, &g_linear_i8_error, DEV_INJECTED_STALL, p.stall_ns));
            const uint64_t bd0 = smem_desc(smem_u32(sm.b[0][0]), 16u, 1024u);
            for (int t = 0; t < mine && ok; ++t) {
                const uint32_t buf = t % kBufs, use = (uint32_t)t / kBufs, d = tmem + buf * (uint32_t)BN;
                ok = __all_sync(0xffffffffu, wait_phase<PAIR == 2>(bar(sm.acc_empty[buf]), (use & 1u) ^ 1u, abort_flag, &g_linear_i8_error,
                                                                   DEV_TIMEOUT_MMA, limit));
                for (int s = 0; s < steps && ok; ++s) {
                    ok = __all_sync(0xffffffffu, wait_phase<PAIR == 2>(bar(sm.full[slot]), phase, abort_flag, &g_linear_i8_error,
                                                                       DEV_TIMEOUT_MMA, limit));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_f16_ta<PAIR>(d, tmem + kTcACol + slot * 64u + 8u * k,
                                         bd0 + (uint64_t)((2u * slot + k / 4) * (uint32_t)(kShare * 128 / 16) + 2u * (k % 4)), idesc,
                                         s > 0 || k > 0, leader);
                    commit_ta<PAIR>(bar(sm.empty[slot]), leader);
                    if (++slot == kTcSlots) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
                if (ok) commit_ta<PAIR>(bar(sm.acc_full[buf]), leader);
            }
            if (!ok) {  // no product may still be running when tensor memory is freed
                commit_ta<PAIR>(bar(sm.drain), leader);
                if (lane == 0) wait_drain(bar(sm.drain), 0u, 100000000ull);
            }
            __syncwarp();
        }
    } else {
        // ------------------- epilogue -------------------
        const int q = warp & 3, ew = warp - kTcEpi0;
        uint16_t* Y = static_cast<uint16_t*>(p.Y);
        int t = 0;
        for (; t < mine; ++t) {
            const int tile = unit + t * units;
            const int m0 = (tile / tiles_n * PAIR + rank) * 128 + q * 32, n0 = (tile % tiles_n) * BN;
            const uint32_t buf = t % kBufs, use = (uint32_t)t / kBufs, cs = t & 1u;
            for (int i = ew * 32 + lane; i < BN; i += kTcEpiWarps * 32) {
                float2 c = make_float2(0.0f, 0.0f);
                if (n0 + i < p.N) {
                    c.x = p.sw[n0 + i];
                    if (p.bias) c.y = from_bits<DT>(static_cast<const uint16_t*>(p.bias)[n0 + i]);
                }
                sm.ch[cs][i] = c;
            }
            const float sx = m0 + lane < p.M ? p.sx[m0 + lane] : 0.0f;
            const bool got = wait_phase(bar(sm.acc_full[buf]), use & 1u, abort_flag, &g_linear_i8_error, DEV_TIMEOUT_EPILOGUE, limit);
            if (!epi_all<kTcEpiWarps>(got)) break;  // also: every warp's part of ch is in place
            tc_fence_after();
            // first all of this warp's columns into shared memory, so that the next tile gets the
            // accumulator soon; then the stores
            const int first = 64 * (ew >> 2);
            if constexpr (SPLIT) {  // fp32, where the weights were: every product has read them
#pragma unroll 1
                for (int c0 = first; c0 < min(first + 64, BN); c0 += 32) {
                    uint32_t r[32];
                    tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + c0, r);
                    tmem_wait_ld_only();
                    reg_fence32(r);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint4*>(sm.b[0][0] + split_at<BN>(q * 32 + lane, c0 / 4 + i)) =
                            make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
                }
                break;
            }
            __syncwarp();  // the previous tile's stores have read the buffers
#pragma unroll 1
            for (int c0 = first; c0 < BN; c0 += 128) {
                uint8_t* out = sm.out[ew][(c0 - first) / 128];
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    uint32_t r[32];
                    tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + buf * (uint32_t)BN + c0 + 32 * half, r);
                    tmem_wait_ld_only();
                    reg_fence32(r);
                    // 16-byte chunk i of row r at chunk i ^ (r & 7): no bank conflicts either way
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 c = *reinterpret_cast<const float4*>(&sm.ch[cs][c0 + 32 * half + 8 * i + 2 * e]);
                            w[e] = pack2<DT>(fmaf(__uint_as_float(r[8 * i + 2 * e]), sx * c.x, c.y),
                                             fmaf(__uint_as_float(r[8 * i + 2 * e + 1]), sx * c.z, c.w));
                        }
                        *reinterpret_cast<uint4*>(out + lane * 128 + (((4 * half + i) ^ (lane & 7)) << 4)) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (rank == 0) mbar_arrive(bar(sm.acc_empty[buf]));
                else mbar_arrive_cluster_relaxed(mapa_rank(bar(sm.acc_empty[buf]), 0u));
            }
            if (m0 >= p.M) continue;
#pragma unroll 1
            for (int c0 = first; c0 < BN; c0 += 128) {
                const uint8_t* out = sm.out[ew][(c0 - first) / 128];
                const int n = n0 + c0;
                if (wide_y) {
                    // eight lanes store a row's 128 bytes
#pragma unroll
                    for (int r0 = 0; r0 < 32; r0 += 4) {
                        const int r = r0 + (lane >> 3), i = lane & 7;
                        const uint4 v = *reinterpret_cast<const uint4*>(out + r * 128 + ((i ^ (r & 7)) << 4));
                        if (m0 + r < p.M && n + 8 * i < p.N)
                            *reinterpret_cast<uint4*>(Y + (int64_t)(m0 + r) * p.ldy + n + 8 * i) = v;
                    }
                } else {
                    for (int r = 0; r < 32 && m0 + r < p.M; ++r)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int c = 32 * h + lane;
                            const uint16_t v = *reinterpret_cast<const uint16_t*>(out + r * 128 + (((c >> 3) ^ (r & 7)) << 4) + 2 * (c & 7));
                            if (n + c < p.N) Y[(int64_t)(m0 + r) * p.ldy + n + c] = v;
                        }
                }
            }
        }
        if constexpr (!SPLIT) {  // tiles left by a wait that ran out
#pragma unroll 1
            for (; t < mine; ++t) {
                const int tile = unit + t * units;
                const int m0 = (tile / tiles_n * PAIR + rank) * 128 + q * 32, n0 = (tile % tiles_n) * BN;
#pragma unroll 1
                for (int r = 0; r < 32 && m0 + r < p.M; ++r)
#pragma unroll 1
                    for (int c = 32 * (ew >> 2) + lane; c < BN && n0 + c < p.N; c += 64) Y[(int64_t)(m0 + r) * p.ldy + n0 + c] = 0x7fffu;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (SPLIT) {  // no sums from this CTA: NaN in their place, and so in the whole tile
        if (*abort_flag)
            for (int i = threadIdx.x; i < 128 * BN; i += kTcThreads) reinterpret_cast<float*>(sm.b[0][0])[i] = __uint_as_float(0x7fffffffu);
    }
    if (PAIR == 2 || SPLIT) cluster_sync_all();  // neither CTA leaves while the other may still signal it; SPLIT: the sums are there
    if constexpr (SPLIT) {
        uint16_t* Y = static_cast<uint16_t*>(p.Y);
        const int m0 = unit / tiles_n * 128, n0 = (unit % tiles_n) * BN;
        const int row0 = 128 * part / splits, rows = min(128 * (part + 1) / splits, p.M - m0) - row0;
        const uint32_t base = smem_u32(sm.b[0][0]);
        for (int i = threadIdx.x; i < rows * (BN / 4); i += kTcThreads) {
            const int r = row0 + i / (BN / 4), c = i % (BN / 4), n = n0 + 4 * c;
            if (n >= p.N) continue;
            const float sx = p.sx[m0 + r];
            float4 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < splits) v[j] = ld_cluster4(mapa_rank(base + split_at<BN>(r, c), (uint32_t)j));
#pragma unroll
            for (int j = 1; j < 8; ++j)
                if (j < splits) {
                    v[0].x += v[j].x;
                    v[0].y += v[j].y;
                    v[0].z += v[j].z;
                    v[0].w += v[j].w;
                }
            const float4 a = *reinterpret_cast<const float4*>(&sm.ch[0][4 * c]), b = *reinterpret_cast<const float4*>(&sm.ch[0][4 * c + 2]);
            const uint32_t lo = pack2<DT>(fmaf(v[0].x, sx * a.x, a.y), fmaf(v[0].y, sx * a.z, a.w));
            const uint32_t hi = pack2<DT>(fmaf(v[0].z, sx * b.x, b.y), fmaf(v[0].w, sx * b.z, b.w));
            uint16_t* y = Y + (int64_t)(m0 + r) * p.ldy + n;
            if (wide_y) {
                *reinterpret_cast<uint2*>(y) = make_uint2(lo, hi);
            } else {
                y[0] = (uint16_t)lo;
                if (n + 1 < p.N) y[1] = (uint16_t)(lo >> 16);
                if (n + 2 < p.N) y[2] = (uint16_t)hi;
                if (n + 3 < p.N) y[3] = (uint16_t)(hi >> 16);
            }
        }
        cluster_sync_all();  // the others have read this CTA's sums
    }
    if (warp == kTcMmaWarp) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc<PAIR>(tmem, kTmemCols);
    }
}

template <int KS>
kt_status launch_dot(int dtype, const LinearI8& p, void* stream, const char** why) {
    constexpr int rows = kDotWarps / KS * 8, step = KS * kDotAhead * 128;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.N + rows - 1) / rows), (unsigned)((p.M + kDotTokens - 1) / kDotTokens));
    cfg.blockDim = dim3(kDotWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = (size_t)kDotTokens * std::min(kDotChunk, (p.K + step - 1) / step * step);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = dtype == KT_BF16 ? cudaLaunchKernelEx(&cfg, kt_linear_i8_dot_kernel<KT_BF16, KS>, p)
                                           : cudaLaunchKernelEx(&cfg, kt_linear_i8_dot_kernel<KT_F16, KS>, p);
    if (e != cudaSuccess) {
        *why = cudaGetErrorString(e);
        return KT_ERR_CUDA;
    }
    return KT_OK;
}

inline int64_t tc_tiles(const LinearI8& p, int bn, int pair) {
    return (int64_t)((p.M + 128 * pair - 1) / (128 * pair)) * ((p.N + bn - 1) / bn);
}

// The tensor-core kernel of a type, opted in to its shared memory.
template <int BN, int PAIR, bool SPLIT>
cudaError_t tc_kernel(int dtype, int device, decltype(&kt_linear_i8_tc_kernel<KT_F16, BN, PAIR, SPLIT>)* kern, int* smem) {
    static SmemOptIn opt_in[2];  // by dtype
    *kern = dtype == KT_BF16 ? kt_linear_i8_tc_kernel<KT_BF16, BN, PAIR, SPLIT> : kt_linear_i8_tc_kernel<KT_F16, BN, PAIR, SPLIT>;
    *smem = (int)sizeof(TcSmem<BN, PAIR>) + 1024;
    return opt_in[dtype == KT_BF16](*kern, *smem, device);
}

// attr: room for two.  `ctas` per cluster.
inline cudaLaunchConfig_t tc_config(int grid, int ctas, int smem, void* stream, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(kTcThreads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cfg;
}

// Clusters of ks (2, 4 or 8) CTAs that the device holds at once; 0 if it cannot say.
template <int BN>
int tc_clusters(int dtype, int ks, int device) {
    static std::atomic<int> known[64][3];  // + 1, by device and ks: both types need the same
    const int slot = ks == 2 ? 0 : ks == 4 ? 1 : 2;
    int n = known[device & 63][slot].load(std::memory_order_relaxed) - 1;
    if (n >= 0) return n;
    decltype(&kt_linear_i8_tc_kernel<KT_F16, BN, 1, true>) kern;
    int smem;
    cudaLaunchAttribute attr[2];
    n = 0;
    if (tc_kernel<BN, 1, true>(dtype, device, &kern, &smem) == cudaSuccess) {
        const cudaLaunchConfig_t cfg = tc_config(ks, ks, smem, nullptr, attr);
        if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
    }
    known[device & 63][slot].store(n + 1, std::memory_order_relaxed);
    return n;
}

// splits > 1 (SPLIT): clusters of so many CTAs, one tile each.
template <int BN, int PAIR, bool SPLIT = false>
kt_status launch_tc(int dtype, const LinearI8& p, int sms, int device, void* stream, const char** why, int splits = 1) {
    const int tiles_n = (p.N + BN - 1) / BN, tiles = (int)tc_tiles(p, BN, PAIR);
    // whole 16-byte pieces of Y's rows: the last one too, as N is a multiple of 8
    const int wide = p.N % 8 == 0 && p.ldy % 8 == 0 && (reinterpret_cast<uintptr_t>(p.Y) & 15u) == 0;
    decltype(&kt_linear_i8_tc_kernel<KT_F16, BN, PAIR, SPLIT>) kern;
    int smem;
    cudaError_t e = tc_kernel<BN, PAIR, SPLIT>(dtype, device, &kern, &smem);
    if (e == cudaSuccess) {
        cudaLaunchAttribute attr[2];
        const int grid = SPLIT ? tiles * splits : std::min(tiles, sms / PAIR) * PAIR;
        const cudaLaunchConfig_t cfg = tc_config(grid, PAIR * splits, smem, stream, attr);
        e = cudaLaunchKernelEx(&cfg, kern, p, tiles_n, tiles, make_idesc(KT_F16, BN, 128 * PAIR, 1), wide);
    }
    if (e != cudaSuccess) {
        *why = cudaGetErrorString(e);
        return KT_ERR_CUDA;
    }
    return KT_OK;
}

}  // namespace

kt_status linear_i8_status(void* stream, int* word, const char** why) {
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemcpyFromSymbolAsync(word, g_linear_i8_error, sizeof(int), 0, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e == cudaSuccess && *word != 0) {
        const int none = 0;
        e = cudaMemcpyToSymbolAsync(g_linear_i8_error, &none, sizeof(int), 0, cudaMemcpyHostToDevice, st);
        if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    }
    if (e == cudaSuccess) return KT_OK;
    *why = cudaGetErrorString(e);
    return KT_ERR_CUDA;
}

kt_status launch_linear_i8(int dtype, const LinearI8& p, int sms, int device, void* stream, const char** why) {
    // Up to 16 tokens the integer products: 10240 channels of 1280, 8 tokens 6.8 us (tensor cores 9.3),
    // 16 8.9 (9.4), 24 11.2 (9.6).
    if (p.M > KT_LINEAR_I8_DOT_ROWS) {
        // tile width: rounds over the CTAs (or pairs) times a round's time.  Measured per round of
        // 76 pairs (9 steps, K = 1152): 8.6, 6.5, 5.2 and 4.6 us for 256, 192, 128 and 64 channels;
        // 30.1, 21.7, 18.5 and 17.0 us for 36 steps.
        constexpr int kWidths = 4;
        constexpr int bn[kWidths] = {256, 192, 128, 64}, per[kWidths] = {86, 65, 52, 46};
        // One CTA per tile, not a pair, where all tiles fit at once: a pair's start and end cost 1 us
        // (1000 x 1152 x 1152 9.4 -> 8.2 us, 1000 x 1152 x 320 6.3 -> 4.9).
        const int pair = p.M > 128 && tc_tiles(p, 128, 1) > sms ? 2 : 1, steps = (p.K + 127) / 128;
        int best = -1;
        int64_t best_cost = 0, best_rounds = 0;
        for (int i = pair == 2 ? 0 : 2; i < kWidths; ++i) {
            const int64_t t = tc_tiles(p, bn[i], pair), units = sms / pair, rounds = (t + units - 1) / units;
            if (best >= 0 && rounds * per[i] >= best_cost) continue;
            best = i;
            best_cost = rounds * per[i];
            best_rounds = rounds;
        }
        // A single round of long rows waits for one step's loads after another's: clusters that share
        // a tile's steps, where all of them fit at once.  A round's time in us with s steps per CTA,
        // measured from 2 to 64 steps (within 1.5 us): 2.6 + 0.55 s and 3.0 + 0.60 s for 64 and 128
        // channels (pairs: the same), and split 4.6 + 0.57 s and 4.7 + 0.70 s.  64 x 1280 x 5120
        // 24.0 -> 10.3 us, 729 x 1152 x 4304 22.9 -> 18.1 us; no gain below about 8 steps.
        if (best_rounds == 1) {
            double least = 0.9 * (bn[best] <= 64 ? 2.6 + 0.55 * steps : 3.0 + 0.60 * steps);
            int width = 0, ways = 1;
            for (const int w : {64, 128})
                for (int ks = 2; ks <= 8 && ks <= steps; ks *= 2) {
                    const int s = (steps + ks - 1) / ks;
                    const double time = w == 64 ? 4.6 + 0.57 * s : 4.7 + 0.70 * s;
                    if (time >= least || tc_tiles(p, w, 1) * ks > sms) continue;
                    if (tc_tiles(p, w, 1) > (w == 64 ? tc_clusters<64>(dtype, ks, device) : tc_clusters<128>(dtype, ks, device))) continue;
                    least = time;
                    width = w;
                    ways = ks;
                }
            if (width == 64) return launch_tc<64, 1, true>(dtype, p, sms, device, stream, why, ways);
            if (width == 128) return launch_tc<128, 1, true>(dtype, p, sms, device, stream, why, ways);
        }
        if (pair == 2) {
            if (best == 0) return launch_tc<256, 2>(dtype, p, sms, device, stream, why);
            if (best == 1) return launch_tc<192, 2>(dtype, p, sms, device, stream, why);
            if (best == 2) return launch_tc<128, 2>(dtype, p, sms, device, stream, why);
            return launch_tc<64, 2>(dtype, p, sms, device, stream, why);
        }
        if (best == 2) return launch_tc<128, 1>(dtype, p, sms, device, stream, why);
        return launch_tc<64, 1>(dtype, p, sms, device, stream, why);
    }
    // warps of a block that share a weight row's columns: as many as leave a step of 512 to each and
    // the SMs with no more than four blocks each
    auto blocks = [&](int ks) { return (int64_t)((p.N * ks + kDotWarps * 8 - 1) / (kDotWarps * 8)) * ((p.M + kDotTokens - 1) / kDotTokens); };
    if (p.K > 3 * kDotAhead * 128 && blocks(4) <= 4 * sms) return launch_dot<4>(dtype, p, stream, why);
    if (p.K > kDotAhead * 128 && blocks(2) <= 4 * sms) return launch_dot<2>(dtype, p, stream, why);
    return launch_dot<1>(dtype, p, stream, why);
}

}  // namespace kt
