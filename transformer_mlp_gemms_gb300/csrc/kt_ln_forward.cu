// kt_ln_forward.cu -- layer norm of the rows of X[M][D], with the statistics that the backward
// pass reads:  mean = avg(x),  rstd = 1 / sqrt(avg((x - mean)^2) + eps),
// y = (x - mean) rstd gamma + beta, rounded once.
//
// Bound by HBM: 2 D bytes read and 2 D written per row, against 8 operations per element.  A
// team of warps (kt_rows.cuh) keeps its row in registers, so the row is read once although the
// variance is a second pass over it; gamma and beta are in shared memory as fp32 (rows up to 2048
// columns; registers beyond), and the next row's loads are issued before this row's reductions.
// What else the time goes to is instructions: the deviations are unpacked once and kept as fp32,
// two at a time (10 instructions per element before, 5 now).  65536 x 640 takes 29.0 us, 5.8 TB/s;
// 32768 x 1280 27.6 us, 6.1 TB/s; 65536 x 642 42 us; a few rows 2.3 us, a launch's latency.  A ring of rows ahead in
// shared memory, as the backward pass has, is slower here: 36 us for the first.
#include "kt_ops_internal.h"
#include "kt_rows.cuh"

namespace kt {
namespace {

constexpr int kLnStagedWarps = 2;

// Resident blocks per SM: as many rows in flight as the registers allow.
constexpr int ln_per_sm(int W, int V) { return W == 16 ? (V <= 2 ? 2 : 1) : V <= 1 ? 5 : V == 2 ? 4 : V == 3 && W <= kLnStagedWarps ? 3 : 2; }

template <int DT, int W, int V, bool VEC>
__global__ void __launch_bounds__(row_block(W), ln_per_sm(W, V)) kt_ln_forward_kernel(const LnForward p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int TL = 32 * W, teams = row_block(W) / TL;
    constexpr bool kStaged = W <= kLnStagedWarps;  // gamma and beta in shared memory
    __shared__ TeamLines<W> lines;
    const int team = threadIdx.x / TL, l = threadIdx.x % TL;
    const uint16_t* X = static_cast<const uint16_t*>(p.X);
    uint16_t* Y = static_cast<uint16_t*>(p.Y);
    const int D = p.D, step = (int)gridDim.x * teams;
    const float inv = 1.0f / (float)D;
    extern __shared__ __align__(16) uint8_t smem[];  // gamma and beta
    const bool affine = p.gamma != nullptr;
    float4* gs = reinterpret_cast<float4*>(smem);
    float4* bs = reinterpret_cast<float4*>(smem + staged_bytes(W, V));
    if (kStaged && affine) {
        stage_vector<DT, VEC, W, V>(static_cast<const uint16_t*>(p.gamma), gs, D);
        stage_vector<DT, VEC, W, V>(static_cast<const uint16_t*>(p.beta), bs, D);
    }
    int row = (int)blockIdx.x * teams + team;
    int turn = 0;

    uint4 c[V], gw[kStaged ? 1 : V], bw[kStaged ? 1 : V];
#pragma unroll
    for (int s = 0; s < V; ++s) c[s] = load_slot<VEC>(X + (int64_t)row * p.ldx, s, l, TL, row < p.M ? D : 0);
    if (!kStaged && affine) {
#pragma unroll
        for (int s = 0; s < (kStaged ? 0 : V); ++s) {
            gw[s] = load_slot<VEC>(static_cast<const uint16_t*>(p.gamma), s, l, TL, D);
            bw[s] = load_slot<VEC>(static_cast<const uint16_t*>(p.beta), s, l, TL, D);
        }
    }
    if (kStaged && affine) __syncthreads();
    if (row >= p.M) return;  // the whole team: the barriers from here on are its own
    for (;;) {
        const int next = p.M - row > step ? row + step : p.M;
        SlotAhead<VEC> n[V];
        if (next < p.M) {
#pragma unroll
            for (int s = 0; s < V; ++s) n[s].load(X + (int64_t)next * p.ldx, s, l, TL, D);
        }
        // a first mean, of terms x / D: no sum overflows that the mean does not
        const f32x2 share = f2(inv);
        f32x2 d[4 * V], acc = f2(0.0f);  // the row, then its deviations
#pragma unroll
        for (int s = 0; s < V; ++s) {
            f32x2 f[4];
            unpack_pairs<DT>(c[s], f);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                d[4 * s + e] = f[e];
                acc = f2_fma<true>(f[e], share, acc);  // past the row's end: zeros
            }
        }
        float about = acc.x + acc.y, none = 0.0f;
        team_add2<W>(about, none, lines, turn, team);
        // The deviations are those from the 16-bit number nearest to it: a difference of two such
        // numbers is off by one fp32 rounding of itself, so neither a row far from zero nor a value
        // far from the others costs the rest its digits, and a row of equal values has none at all.
        // Their average corrects the mean, and its square the variance; it is below the spread of
        // any row that is not all equal (the values stand on the same 16-bit grid), so that
        // the difference keeps its digits.
        float near[8];
        unpack8<DT>(make_uint4(pack2<DT>(about, 0.0f) & 0xffffu, 0u, 0u, 0u), near);
        const f32x2 origin = f2(near[0]);
        f32x2 squares = f2(0.0f);
        acc = f2(0.0f);
#pragma unroll
        for (int s = 0; s < V; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                d[4 * s + e] = f2_sub<true>(d[4 * s + e], origin);
                clear_past_end<VEC, W, V>(d[4 * s + e], s, e, l, D);
                acc = f2_add<true>(acc, d[4 * s + e]);
                squares = f2_fma<true>(d[4 * s + e], d[4 * s + e], squares);
            }
        float sum = acc.x + acc.y, sq = squares.x + squares.y;
        team_add2<W>(sum, sq, lines, turn, team);
        const float dmean = sum * inv;  // mean - origin
        float var = sq * inv;
        if (var < __uint_as_float(0x7f800000u)) var = fmaxf(fmaf(-dmean, dmean, var), 0.0f);
        const float rstd = 1.0f / sqrtf(var + p.eps);
        if (l == 0) {
            const float mean = near[0] + dmean;  // `about`: a row with an infinity, or differences beyond fp32
            if (p.mean) p.mean[row] = fabsf(mean) < __uint_as_float(0x7f800000u) ? mean : about;
            if (p.rstd) p.rstd[row] = rstd;
        }
        const f32x2 scale = f2(rstd), shift = f2(-dmean * rstd);
        uint16_t* yr = Y + (int64_t)row * p.ldy;
#pragma unroll
        for (int s = 0; s < V; ++s) {
            f32x2 f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = f2_fma<true>(d[4 * s + e], scale, shift);
            if (affine) {
                f32x2 g[4], b[4];
                if constexpr (kStaged) {
                    staged_pairs<W>(gs, s, l, g);
                    staged_pairs<W>(bs, s, l, b);
                } else {
                    unpack_pairs<DT>(gw[s], g);
                    unpack_pairs<DT>(bw[s], b);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = f2_fma<true>(f[e], g[e], b[e]);
            }
            store_slot<VEC>(yr, s, l, TL, D, pack_pairs<DT>(f));
        }
        if (!kStaged && affine) {
            forget_unpacked(gw);
            forget_unpacked(bw);
        }
        if (next >= p.M) break;
        row = next;
#pragma unroll
        for (int s = 0; s < V; ++s) c[s] = n[s].slot();
    }
}

}  // namespace

kt_status launch_ln_forward(int dtype, const LnForward& p, int sms, void* stream, const char** why) {
    const auto al = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; };
    const bool vec = p.D % 8 == 0 && p.ldx % 8 == 0 && p.ldy % 8 == 0 && al(p.X) && al(p.Y) && al(p.gamma) && al(p.beta);
    RowShape shape;
    if (!(vec ? row_shape(p.D, &shape) : scalar_row_shape(p.D, &shape))) {
        *why = "rows of this length are not supported";
        return KT_ERR_UNSUPPORTED;
    }
    auto go = [&](auto dt, auto v16) {
        return with_shape<decltype(v16)::value, !decltype(v16)::value>(shape, [&](auto W, auto V) -> kt_status {
            constexpr int w = decltype(W)::value, t = decltype(dt)::value, v = decltype(V)::value;
            constexpr bool al16 = decltype(v16)::value;
            constexpr int teams = row_block(w) / (32 * w), per_sm = ln_per_sm(w, v);
            constexpr int staged = w <= kLnStagedWarps ? 2 * staged_bytes(w, v) : 0;
            const int64_t blocks = ((int64_t)p.M + teams - 1) / teams;
            const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)sms * per_sm);
            const cudaError_t e = launch_pdl(kt_ln_forward_kernel<t, w, v, al16>, grid, row_block(w), staged, stream, p);
            if (e != cudaSuccess) {
                *why = cudaGetErrorString(e);
                return KT_ERR_CUDA;
            }
            return KT_OK;
        });
    };
    using F16 = std::integral_constant<int, KT_F16>;
    using BF16 = std::integral_constant<int, KT_BF16>;
    if (dtype == KT_F16) return vec ? go(F16{}, std::true_type{}) : go(F16{}, std::false_type{});
    return vec ? go(BF16{}, std::true_type{}) : go(BF16{}, std::false_type{});
}

}  // namespace kt
