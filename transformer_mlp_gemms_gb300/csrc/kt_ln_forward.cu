// kt_ln_forward.cu -- layer norm of the rows of X[M][D], with the statistics that the backward
// pass reads:  mean = avg(x),  rstd = 1 / sqrt(avg((x - mean)^2) + eps),
// y = (x - mean) rstd gamma + beta, rounded once.
//
// Bound by HBM: 2 D bytes read and 2 D written per row, against 8 operations per element.  A
// team of warps (kt_rows.cuh) keeps its row in registers, so the row is read once although the
// variance is a second pass over it; gamma and beta stay in registers as well, from row to row
// of a persistent grid, and the next row's loads are issued before this row's reductions, so
// that the memory has something to do while the team waits for its sums.
#include "kt_ops_internal.h"
#include "kt_rows.cuh"

namespace kt {
namespace {

template <int DT, int W, int V, bool VEC>
__global__ void __launch_bounds__(row_block(W), W == 16 ? 1 : 2) kt_ln_forward_kernel(const LnForward p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int TL = 32 * W, teams = row_block(W) / TL;
    __shared__ TeamLines<W> lines;
    const int team = threadIdx.x / TL, l = threadIdx.x % TL;
    const uint16_t* X = static_cast<const uint16_t*>(p.X);
    uint16_t* Y = static_cast<uint16_t*>(p.Y);
    const int D = p.D, step = (int)gridDim.x * teams;
    const float inv = 1.0f / (float)D;
    int row = (int)blockIdx.x * teams + team;
    if (row >= p.M) return;  // the whole team: its barriers are its own
    int turn = 0;

    uint4 c[V], gw[V], bw[V];
#pragma unroll
    for (int s = 0; s < V; ++s) c[s] = load_slot<VEC>(X + (int64_t)row * p.ldx, s, l, TL, D);
    uint16_t first = X[(int64_t)row * p.ldx], next_first = 0;
    const bool affine = p.gamma != nullptr;
    if (affine) {
#pragma unroll
        for (int s = 0; s < V; ++s) {
            gw[s] = load_slot<VEC>(static_cast<const uint16_t*>(p.gamma), s, l, TL, D);
            bw[s] = load_slot<VEC>(static_cast<const uint16_t*>(p.beta), s, l, TL, D);
        }
    }
    for (;;) {
        // the deviations are taken from the row's first element, exactly: a row far from zero
        // keeps its low bits in the sums
        float f0[8];
        unpack8<DT>(make_uint4(first, 0u, 0u, 0u), f0);
        const float x0 = f0[0];
        const int next = p.M - row > step ? row + step : p.M;
        uint4 n[V];
        if (next < p.M) {
            next_first = X[(int64_t)next * p.ldx];
#pragma unroll
            for (int s = 0; s < V; ++s) n[s] = load_slot<VEC>(X + (int64_t)next * p.ldx, s, l, TL, D);
        }
        const f32x2 origin = f2(x0);
        f32x2 acc = f2(0.0f);
#pragma unroll
        for (int s = 0; s < V; ++s) {
            f32x2 f[4];
            unpack_pairs<DT>(c[s], f);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f32x2 d = f2_sub<true>(f[e], origin);
                clear_past_end<VEC, W, V>(d, s, e, l, D);
                acc = f2_add<true>(acc, d);
            }
        }
        float sum = acc.x + acc.y, none = 0.0f;
        team_add2<W>(sum, none, lines, turn, team);
        const float dmean = sum * inv;  // mean - x0
        const f32x2 shift = f2(dmean);
        forget_unpacked(c);
        acc = f2(0.0f);
#pragma unroll
        for (int s = 0; s < V; ++s) {
            f32x2 f[4];
            unpack_pairs<DT>(c[s], f);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f32x2 d = f2_sub<true>(f2_sub<true>(f[e], origin), shift);
                clear_past_end<VEC, W, V>(d, s, e, l, D);
                acc = f2_fma<true>(d, d, acc);
            }
        }
        float sq = acc.x + acc.y;
        none = 0.0f;
        team_add2<W>(sq, none, lines, turn, team);
        const float rstd = 1.0f / sqrtf(sq * inv + p.eps);
        if (l == 0) {
            if (p.mean) p.mean[row] = x0 + dmean;
            if (p.rstd) p.rstd[row] = rstd;
        }
        const f32x2 scale = f2(rstd);
        forget_unpacked(c);
        uint16_t* yr = Y + (int64_t)row * p.ldy;
#pragma unroll
        for (int s = 0; s < V; ++s) {
            f32x2 f[4];
            unpack_pairs<DT>(c[s], f);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = f2_mul<true>(f2_sub<true>(f2_sub<true>(f[e], origin), shift), scale);
            if (affine) {
                f32x2 g[4], b[4];
                unpack_pairs<DT>(gw[s], g);
                unpack_pairs<DT>(bw[s], b);
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = f2_fma<true>(f[e], g[e], b[e]);
            }
            store_slot<VEC>(yr, s, l, TL, D, pack_pairs<DT>(f));
        }
        if (affine) {
            forget_unpacked(gw);
            forget_unpacked(bw);
        }
        if (next >= p.M) break;
        row = next;
        first = next_first;
#pragma unroll
        for (int s = 0; s < V; ++s) c[s] = n[s];
    }
}

}  // namespace

kt_status launch_ln_forward(int dtype, const LnForward& p, int sms, void* stream, const char** why) {
    RowShape shape;
    if (!row_shape(p.D, &shape)) {
        *why = "rows of this length are not supported";
        return KT_ERR_UNSUPPORTED;
    }
    const auto al = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; };
    const bool vec = p.D % 8 == 0 && p.ldx % 8 == 0 && p.ldy % 8 == 0 && al(p.X) && al(p.Y) && al(p.gamma) && al(p.beta);
    auto go = [&](auto dt, auto v16) {
        return with_shape<decltype(v16)::value>(shape, [&](auto W, auto V) -> kt_status {
            constexpr int w = decltype(W)::value;
            const int teams = row_block(w) / (32 * w);
            const int64_t blocks = ((int64_t)p.M + teams - 1) / teams;
            const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)sms * (w == 16 ? 1 : 2));
            cudaError_t e = launch_pdl(kt_ln_forward_kernel<decltype(dt)::value, w, decltype(V)::value, decltype(v16)::value>,
                                       grid, row_block(w), 0, stream, p);
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
