// kt_ln_backward.cu -- the gradients of layer norm.  With xhat = (x - mean) rstd, g = dy gamma:
//   dx = rstd (g - avg(g) - xhat avg(g xhat)),  dgamma = sum_rows dy xhat,  dbeta = sum_rows dy.
//
// Bound by HBM: 4 D bytes read and 2 D written per row.  One pass: a team of warps
// (kt_rows.cuh) keeps its rows of x and dy in registers between the two averages and dx, and
// adds each row's terms of dgamma and dbeta to fp32 sums of its own columns, in registers (in
// shared memory for teams of 16 warps, whose threads have too few).  At the end a block adds
// its teams' sums in team order and writes one row of partial sums; a second kernel adds the
// rows of all blocks in order.  No atomics: the same bits from run to run.
// The sums take most of the registers, so an SM holds 8 warps; long batches therefore copy the
// next rows into shared memory asynchronously while a row is at work (48 -> 45 us for 32768 x
// 1280, 5.6 TB/s; without the paired arithmetic 58).  729 x 1152 takes 5.8 us: two dependent kernels.
#include "kt_ops_internal.h"
#include "kt_rows.cuh"

namespace kt {
namespace {

__device__ __forceinline__ float of_pair(const f32x2& v, int e) { return e & 1 ? v.y : v.x; }

// Resident blocks per SM, and whether a row's xhat and g stay in registers between the averages
// and dx (else they are computed twice): what the registers allow beside the sums of dgamma and dbeta
// (and, without 16-byte loads, the next row's elements one by one).
constexpr int ln_back_per_sm(int W, int V) { return W == 16 ? 1 : V <= 1 ? 3 : V == 2 ? 2 : 1; }
constexpr bool ln_back_keeps(int W, int V, bool VEC) { return VEC && W < 16 && V >= 3; }
constexpr int kLnBackStagedWarps = 2;  // gamma in shared memory up to so many warps per row

template <int DT, int W, int V, bool VEC, bool RING>
__global__ void __launch_bounds__(row_block(W), ln_back_per_sm(W, V)) kt_ln_backward_kernel(const LnBackward p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int TL = 32 * W, teams = row_block(W) / TL;
    constexpr bool kSmemSums = W == 16;
    constexpr bool kAhead = !RING && W != 16;  // the next row's loads in flight during this row's sums
    constexpr bool kKeep = ln_back_keeps(W, V, VEC), kStaged = W <= kLnBackStagedWarps;
    __shared__ TeamLines<W> lines;
    // gamma, then the ring; the final addition's [teams][TL * V * 8] where they were; or [2][..] (kSmemSums)
    extern __shared__ __align__(16) uint8_t smem[];
    float* sums = reinterpret_cast<float*>(smem);
    float4* gs = reinterpret_cast<float4*>(smem);
    const int team = threadIdx.x / TL, l = threadIdx.x % TL;
    const uint16_t* X = static_cast<const uint16_t*>(p.X);
    const uint16_t* dY = static_cast<const uint16_t*>(p.dY);
    uint16_t* dX = static_cast<uint16_t*>(p.dX);
    const int D = p.D, step = (int)gridDim.x * teams;
    const float inv = 1.0f / (float)D;
    const bool affine = p.gamma != nullptr, want = p.dgamma != nullptr;
    int row = (int)blockIdx.x * teams + team;
    int turn = 0;

    f32x2 dg[kSmemSums ? 1 : 4 * V], db[kSmemSums ? 1 : 4 * V];
    if constexpr (kSmemSums) {
        for (int i = threadIdx.x; i < 2 * TL * V * 8; i += row_block(W)) sums[i] = 0.0f;
        __syncthreads();
    } else {
#pragma unroll
        for (int i = 0; i < 4 * V; ++i) dg[i] = db[i] = f2(0.0f);
    }
    RowRing<W, V, 2> ring;  // x, then dy
    int slot = 0;
    const auto copy = [&](int at, int64_t r) {
        ring.copy(at, 0, X + r * p.ldx, l, D);
        ring.copy(at, 1, dY + r * p.lddy, l, D);
    };
    uint4 cx[V], cy[V], gw[kStaged ? 1 : V];
    float mean = 0.0f, rstd = 0.0f, next_mean = 0.0f, next_rstd = 0.0f;
    if (row < p.M) {
        mean = p.mean[row];
        rstd = p.rstd[row];
        if constexpr (RING) {
            ring.open(smem + (kStaged ? staged_bytes(W, V) : 0), team, l);
#pragma unroll
            for (int i = 0; i < ring.rows; ++i) {
                if (p.M - row > (int64_t)i * step) copy(i, row + (int64_t)i * step);
                ring.commit();
            }
        } else
#pragma unroll
        for (int s = 0; s < V; ++s) {
            cx[s] = load_slot<VEC>(X + (int64_t)row * p.ldx, s, l, TL, D);
            cy[s] = load_slot<VEC>(dY + (int64_t)row * p.lddy, s, l, TL, D);
        }
    }
    if (kStaged && affine) {
        stage_vector<DT, VEC, W, V>(static_cast<const uint16_t*>(p.gamma), gs, D);
        __syncthreads();
    }
    if (!kStaged && affine) {
#pragma unroll
        for (int s = 0; s < (kStaged ? 0 : V); ++s) gw[s] = load_slot<VEC>(static_cast<const uint16_t*>(p.gamma), s, l, TL, D);
    }
    while (row < p.M) {
        if constexpr (RING) {
            ring.wait_oldest();
            ring.read(slot, 0, cx);
            ring.read(slot, 1, cy);
        }
        const int next = p.M - row > step ? row + step : p.M;
        SlotAhead<VEC> nx[V], ny[V];
        if (next < p.M) {
            next_mean = p.mean[next];
            next_rstd = p.rstd[next];
        }
        if (kAhead && next < p.M) {
#pragma unroll
            for (int s = 0; s < V; ++s) {
                nx[s].load(X + (int64_t)next * p.ldx, s, l, TL, D);
                ny[s].load(dY + (int64_t)next * p.lddy, s, l, TL, D);
            }
        }
        const f32x2 mu = f2(mean), scale = f2(rstd);
        f32x2 a1 = f2(0.0f), a2 = f2(0.0f);
        f32x2 keep_xh[kKeep ? 4 * V : 1], keep_g[kKeep ? 4 * V : 1];
        // x - mean, xhat, dy and g of slot s
        auto terms = [&](int s, f32x2 (&dev)[4], f32x2 (&xh)[4], f32x2 (&y)[4], f32x2 (&ge)[4]) {
            f32x2 x[4], g[4];
            unpack_pairs<DT>(cx[s], x);
            unpack_pairs<DT>(cy[s], y);
            if (affine) {
                if constexpr (kStaged) staged_pairs<W>(gs, s, l, g);
                else unpack_pairs<DT>(gw[s], g);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                dev[e] = f2_sub<true>(x[e], mu);
                xh[e] = f2_mul<true>(dev[e], scale);
                ge[e] = affine ? f2_mul<true>(y[e], g[e]) : y[e];
            }
        };
#pragma unroll
        for (int s = 0; s < V; ++s) {
            f32x2 dev[4], xh[4], y[4], ge[4];
            terms(s, dev, xh, y, ge);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // Columns past the row's end add nothing to either average: dy is 0 there.  But with x = 0
                // their xhat may be beyond fp32 where the row's own are not, and 0 * inf is no number.
                // With 16-byte slots, of which only the last ones are concerned, it is set to 0; without,
                // where a test of each element would cost registers that are not there, the sum is of
                // g (x - mean), which is finite, and rstd comes after it.
                if constexpr (VEC) clear_past_end<VEC, W, V>(xh[e], s, e, l, D);
                a1 = f2_add<true>(a1, ge[e]);
                a2 = f2_fma<true>(ge[e], VEC ? xh[e] : dev[e], a2);
                if constexpr (kKeep) {
                    keep_xh[4 * s + e] = xh[e];
                    keep_g[4 * s + e] = ge[e];
                }
                if constexpr (kSmemSums) {
                    if (want) {
                        float* at = sums + (size_t)(s * 8 + 2 * e) * TL + l;
                        at[0] = fmaf(y[e].x, xh[e].x, at[0]);
                        at[TL] = fmaf(y[e].y, xh[e].y, at[TL]);
                        at[TL * V * 8] += y[e].x;
                        at[TL * V * 8 + TL] += y[e].y;
                    }
                } else {
                    dg[4 * s + e] = f2_fma<true>(y[e], xh[e], dg[4 * s + e]);
                    db[4 * s + e] = f2_add<true>(db[4 * s + e], y[e]);
                }
            }
        }
        float s1 = a1.x + a1.y, s2 = a2.x + a2.y;
        if constexpr (!VEC) s2 = rstd == 0.0f ? 0.0f : s2 * rstd;  // 0: a row whose variance is beyond fp32
        team_add2<W>(s1, s2, lines, turn, team);
        if constexpr (RING) {  // this lane has its part of the row: its slots take the row `rows` ahead
            if (p.M - row > (int64_t)ring.rows * step) copy(slot, (int64_t)row + (int64_t)ring.rows * step);
            ring.commit();
            slot = slot + 1 < ring.rows ? slot + 1 : 0;
        }
        const f32x2 c1 = f2(s1 * inv), c2 = f2(s2 * inv);
        if constexpr (!kKeep) {
            forget_unpacked(cx);
            forget_unpacked(cy);
        }
        if (!kStaged && affine) forget_unpacked(gw);
        uint16_t* xr = dX + (int64_t)row * p.lddx;
#pragma unroll
        for (int s = 0; s < V; ++s) {
            f32x2 dev[4], xh[4], y[4], ge[4];
            if constexpr (kKeep) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    xh[e] = keep_xh[4 * s + e];
                    ge[e] = keep_g[4 * s + e];
                }
            } else {
                terms(s, dev, xh, y, ge);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = f2_mul<true>(scale, f2_sub<true>(ge[e], f2_fma<true>(xh[e], c2, c1)));
            store_slot<VEC>(xr, s, l, TL, D, pack_pairs<DT>(y));
        }
        if (!kStaged && affine) forget_unpacked(gw);
        row = next;
        mean = next_mean;
        rstd = next_rstd;
        if (kAhead) {
#pragma unroll
            for (int s = 0; s < V; ++s) {
                cx[s] = nx[s].slot();
                cy[s] = ny[s].slot();
            }
        } else if (!RING && row < p.M) {
#pragma unroll
            for (int s = 0; s < V; ++s) {
                cx[s] = load_slot<VEC>(X + (int64_t)row * p.ldx, s, l, TL, D);
                cy[s] = load_slot<VEC>(dY + (int64_t)row * p.lddy, s, l, TL, D);
            }
        }
    }
    if (!want) return;
    float* out = p.partials + (size_t)blockIdx.x * 2 * D;
#pragma unroll
    for (int which = 0; which < 2; ++which, out += D) {
        if constexpr (teams == 1) {
#pragma unroll
            for (int s = 0; s < V; ++s)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int c = slot_col<VEC>(s, e, l, TL);
                    if (c < D) {
                        if constexpr (kSmemSums)
                            out[c] = sums[(size_t)which * TL * V * 8 + (size_t)(s * 8 + e) * TL + l];
                        else
                            out[c] = which ? of_pair(db[4 * s + e / 2], e) : of_pair(dg[4 * s + e / 2], e);
                    }
                }
        } else {
            constexpr int width = TL * V * 8;
            __syncthreads();  // every team is done with gamma and its ring; the first sums have been read
#pragma unroll
            for (int s = 0; s < V; ++s)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sums[team * width + (8 * s + e) * TL + l] =
                        which ? of_pair(db[4 * s + e / 2], e) : of_pair(dg[4 * s + e / 2], e);
            __syncthreads();
            for (int i = threadIdx.x; i < width; i += row_block(W)) {
                // i counts (element of a lane, lane): the columns in the teams' order
                const int se = i / TL, li = i % TL, c = slot_col<VEC>(se / 8, se % 8, li, TL);
                float v = 0.0f;
#pragma unroll
                for (int t = 0; t < teams; ++t) v += sums[t * width + i];
                if (c < D) out[c] = v;
            }
        }
    }
}

// Adds the blocks' rows of partial sums, in order: out[c] = sum_r partials[r][c] over the 2 D
// columns (dgamma, then dbeta).  32 columns and 16 runs of rows per block (729 x 1152: 5.8 us for
// the whole backward pass; 8 runs 6.3).  `partials` is still being written when this kernel starts, so
// it carries no promise that would let its loads pass griddepcontrol.wait.
constexpr int kSumRuns = 16;
__global__ void __launch_bounds__(kSumRuns * 32) kt_ln_column_sums_kernel(const float* partials, int rows, int D, float* dgamma,
                                                                          float* dbeta) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float part[kSumRuns][32];
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    const int c = (int)blockIdx.x * 32 + lane;
    const int per = (rows + kSumRuns - 1) / kSumRuns, r1 = min(rows, (run + 1) * per);
    float v = 0.0f;
    if (c < 2 * D) {
#pragma unroll 4
        for (int r = run * per; r < r1; ++r) v += partials[(size_t)r * 2 * D + c];
    }
    part[run][lane] = v;
    __syncthreads();
    if (run == 0 && c < 2 * D) {
        v = part[0][lane];
#pragma unroll
        for (int i = 1; i < kSumRuns; ++i) v += part[i][lane];
        if (c < D)
            dgamma[c] = v;
        else
            dbeta[c - D] = v;
    }
}

}  // namespace

// As many blocks as are resident: each keeps 8 / W rows in flight and the next ones' loads behind them.
int ln_backward_blocks(int64_t M, int64_t D) {
    RowShape shape;
    if (M < 0 || D < 1 || !row_shape(D, &shape)) return 0;
    const int teams = row_block(shape.W) / (32 * shape.W);
    return (int)std::min<int64_t>((M + teams - 1) / teams, (int64_t)kMaxSms * ln_back_per_sm(shape.W, shape.V));
}

kt_status launch_ln_backward(int dtype, const LnBackward& p, int sms, int device, void* stream, const char** why) {
    RowShape shape;
    if (!row_shape(p.D, &shape)) {
        *why = "rows of this length are not supported";
        return KT_ERR_UNSUPPORTED;
    }
    const int grid = std::min(ln_backward_blocks(p.M, p.D), sms * ln_back_per_sm(shape.W, shape.V));
    cudaError_t e = cudaSuccess;
    if (grid > 0) {
        const auto al = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; };
        const bool vec = p.D % 8 == 0 && p.ldx % 8 == 0 && p.lddy % 8 == 0 && p.lddx % 8 == 0 && al(p.X) && al(p.dY) &&
                         al(p.dX) && al(p.gamma);
        auto go = [&](auto dt, auto v16) {
            return with_shape<decltype(v16)::value>(shape, [&](auto W, auto V) -> kt_status {
                constexpr int w = decltype(W)::value, v = decltype(V)::value, teams = row_block(w) / (32 * w);
                constexpr int t = decltype(dt)::value;
                constexpr bool al16 = decltype(v16)::value;
                constexpr size_t sums = (w == 16 ? 2 : teams == 1 ? 0 : teams) * (size_t)(32 * w * v * 8) * sizeof(float);
                constexpr size_t smem = std::max(sums, w <= kLnBackStagedWarps ? (size_t)staged_bytes(w, v) : 0);
                cudaError_t le = cudaSuccess;
                bool ring = false;
                if constexpr (al16 && w < 16 && ln_back_per_sm(w, v) == 1) {
                    // from three rows a team on they come through the ring
                    ring = (int64_t)p.M >= 3 * (int64_t)grid * teams;
                    if (ring) {
                        constexpr size_t staged = w <= kLnBackStagedWarps ? (size_t)staged_bytes(w, v) : 0;
                        constexpr size_t with_ring = std::max(sums, staged + RowRing<w, v, 2>::bytes);
                        static SmemOptIn opt_in;
                        auto kern = kt_ln_backward_kernel<t, w, v, true, true>;
                        le = opt_in(kern, (int)with_ring, device);
                        if (le == cudaSuccess) le = launch_pdl(kern, (unsigned)grid, row_block(w), with_ring, stream, p);
                    }
                }
                if (!ring) {
                    static SmemOptIn opt_in;
                    auto kern = kt_ln_backward_kernel<t, w, v, al16, false>;
                    if (smem > 32 * 1024) le = opt_in(kern, (int)smem, device);
                    if (le == cudaSuccess) le = launch_pdl(kern, (unsigned)grid, row_block(w), smem, stream, p);
                }
                if (le != cudaSuccess) {
                    *why = cudaGetErrorString(le);
                    return KT_ERR_CUDA;
                }
                return KT_OK;
            });
        };
        using F16 = std::integral_constant<int, KT_F16>;
        using BF16 = std::integral_constant<int, KT_BF16>;
        kt_status s;
        if (dtype == KT_F16)
            s = vec ? go(F16{}, std::true_type{}) : go(F16{}, std::false_type{});
        else
            s = vec ? go(BF16{}, std::true_type{}) : go(BF16{}, std::false_type{});
        if (s != KT_OK) return s;
    }
    if (p.dgamma) {
        e = launch_pdl(kt_ln_column_sums_kernel, (unsigned)((2 * (int64_t)p.D + 31) / 32), kSumRuns * 32, 0, stream, p.partials, grid,
                       p.D, p.dgamma, p.dbeta);
        if (e != cudaSuccess) {
            *why = cudaGetErrorString(e);
            return KT_ERR_CUDA;
        }
    }
    return KT_OK;
}

}  // namespace kt
