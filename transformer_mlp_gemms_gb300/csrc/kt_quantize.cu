// kt_quantize.cu -- each row of the activations in signed 8-bit integers with one scale:
//   v = act(x),  scale = max|v| / 127,  q = the integer nearest to v / scale, ties to even.
//
// Bound by HBM: 2 bytes read and 1 written per element.  The row stays in the registers of a
// team of warps (kt_rows.cuh) between its largest magnitude and its rounding, so it is read
// once; the grid is persistent and the next row's loads are in flight behind this row's
// reduction.  The magnitudes are compared as the integers that their bits are, which orders
// NaN above infinity above every number, so one maximum also tells whether the row is finite.
//
// The nearest integer is decided exactly without a division per element: v times the rounded
// inverse of the scale is off by less than 127 * 2^-22 = 3.1e-5, so only a product within
// 1e-4 of a half-integer can go to the wrong side, and the exact remainder of those few tells.
// (A 64-bit division there instead took 66 us for 16384 x 1152: bf16 values have many ties with
// their row's maximum, and this GPU has next to no 64-bit rate.)
#include "kt_ops_internal.h"
#include "kt_rows.cuh"

namespace kt {
namespace {

__device__ __noinline__ int nearest_by_division(float v, float scale) {
    const double t = rint((double)v / (double)scale);
    return (int)fmin(fmax(t, -127.0), 127.0);
}
// From the nearest integer n of a quotient that is off by less than 1e-4: the remainder
// v - n scale is exact in one fused step (a multiple of the smaller operand's last place, and
// hardly above half the scale), and twice it against the scale tells the side and the ties.
__device__ __forceinline__ int nearest_by_remainder(float v, float scale, int n) {
    const float twice = 2.0f * fmaf(-(float)n, scale, v);
    const int up = twice > scale || (twice == scale && (n & 1));
    const int down = twice < -scale || (twice == -scale && (n & 1));
    return n + up - down;
}

// The activation on 8 values (GEGLU: value v, gate g).
__device__ __forceinline__ void activate8(int act, float* v, const float* g) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const f32x2 x = f2(v[e], v[e + 1]);
        f32x2 y = x;
        if (act == KT_ACT_GEGLU) y = f2_mul<true>(x, gelu_erf_f2<true>(f2(g[e], g[e + 1])));
        else if (act == KT_ACT_GELU_ERF) y = gelu_erf_f2<true>(x);
        else if (act == KT_ACT_GELU_TANH) y = gelu_tanh_f2<true>(x);
        else if (act == KT_ACT_GELU_SIGMOID) y = gelu_sigmoid_f2<true>(x);
        else if (act == KT_ACT_SILU) y = silu_f2<true>(x);
        f2_split(y, v[e], v[e + 1]);
    }
}

template <int DT, int W, int V, bool VEC, bool ACT>
__global__ void __launch_bounds__(row_block(W), W == 16 || ACT ? 1 : 2) kt_quantize_kernel(const QuantRows p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int TL = 32 * W, teams = row_block(W) / TL;
    __shared__ TeamLines<W> lines;
    const int team = threadIdx.x / TL, l = threadIdx.x % TL;
    const uint16_t* X = static_cast<const uint16_t*>(p.X);
    const int K = p.K, step = (int)gridDim.x * teams;
    int row = (int)blockIdx.x * teams + team;
    if (row >= p.M) return;  // the whole team: its barriers are its own
    int turn = 0;
    uint4 c[V];
#pragma unroll
    for (int s = 0; s < V; ++s) c[s] = load_slot<VEC>(X + (int64_t)row * p.ldx, s, l, TL, K);
    for (;;) {
        const int next = p.M - row > step ? row + step : p.M;
        uint4 n[V];
        if (next < p.M) {
#pragma unroll
            for (int s = 0; s < V; ++s) n[s] = load_slot<VEC>(X + (int64_t)next * p.ldx, s, l, TL, K);
        }
        float a[ACT ? 8 * V : 8];  // ACT: the row's activated values
        uint32_t most = 0;
#pragma unroll
        for (int s = 0; s < V; ++s) {
            float* v = ACT ? a + 8 * s : a;
            unpack8<DT>(c[s], v);
            if constexpr (ACT) {
                float g[8] = {};
                if (p.act == KT_ACT_GEGLU)
                    unpack8<DT>(load_slot<VEC>(X + (int64_t)row * p.ldx + K, s, l, TL, K), g);
                activate8(p.act, v, g);  // a column past the row: act(0) = 0
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t bits = __float_as_uint(v[e]) & 0x7fffffffu;
                most = bits > most ? bits : most;
            }
        }
        most = team_max<W>(most, lines, turn, team);
        const bool finite = most < 0x7f800000u;
        const float scale = finite ? __fdiv_rn(__uint_as_float(most), 127.0f) : __uint_as_float(0x7fffffffu);
        if (l == 0) p.scale[row] = scale;
        // a scale whose inverse is out of range (a row of subnormals) divides every element
        const bool fast = scale > 1e-37f, zero = !finite || scale == 0.0f;
        const float inv = fast ? __fdiv_rn(1.0f, scale) : 0.0f;
        int8_t* qr = p.Q + (int64_t)row * p.ldq;
#pragma unroll
        for (int s = 0; s < V; ++s) {
            float* v = ACT ? a + 8 * s : a;
            if constexpr (!ACT) unpack8<DT>(c[s], v);
            uint32_t q[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // adding 1.5 * 2^23 rounds to the nearest integer, ties to even, in the low bits
                const float t = v[e] * inv, m = t + 12582912.0f;
                q[e] = __float_as_uint(m);
                const float off = fabsf(t - (m - 12582912.0f));
                if (zero) q[e] = 0;
                else if (!fast) q[e] = (uint32_t)nearest_by_division(v[e], scale);
                else if (off > 0.4999f) q[e] = (uint32_t)nearest_by_remainder(v[e], scale, (int)(m - 12582912.0f));
            }
            if constexpr (VEC) {
                const int col = slot_col<true>(s, 0, l, TL);
                if (col < K) {
                    const uint32_t lo = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
                    const uint32_t hi = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
                    *reinterpret_cast<uint2*>(qr + col) = make_uint2(lo, hi);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int col = slot_col<false>(s, e, l, TL);
                    if (col < K) qr[col] = (int8_t)q[e];
                }
            }
        }
        if (next >= p.M) break;
        row = next;
#pragma unroll
        for (int s = 0; s < V; ++s) c[s] = n[s];
    }
}

}  // namespace

kt_status launch_quantize(int dtype, const QuantRows& p, int sms, void* stream, const char** why) {
    RowShape shape;
    if (!row_shape(p.K, &shape)) {
        *why = "rows of this length are not supported";
        return KT_ERR_UNSUPPORTED;
    }
    const bool vec = p.K % 8 == 0 && p.ldx % 8 == 0 && p.ldq % 8 == 0 && (reinterpret_cast<uintptr_t>(p.X) & 15u) == 0 &&
                     (reinterpret_cast<uintptr_t>(p.Q) & 7u) == 0;
    auto go = [&](auto dt, auto v16, auto act) {
        return with_shape<decltype(v16)::value>(shape, [&](auto W, auto V) -> kt_status {
            constexpr int w = decltype(W)::value;
            const int teams = row_block(w) / (32 * w);
            const int64_t blocks = ((int64_t)p.M + teams - 1) / teams;
            const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)sms * (w == 16 || decltype(act)::value ? 1 : 2));
            cudaError_t e = launch_pdl(
                kt_quantize_kernel<decltype(dt)::value, w, decltype(V)::value, decltype(v16)::value, decltype(act)::value>,
                grid, row_block(w), 0, stream, p);
            if (e != cudaSuccess) {
                *why = cudaGetErrorString(e);
                return KT_ERR_CUDA;
            }
            return KT_OK;
        });
    };
    auto typed = [&](auto dt) {
        if (p.act == KT_ACT_NONE) return vec ? go(dt, std::true_type{}, std::false_type{}) : go(dt, std::false_type{}, std::false_type{});
        return vec ? go(dt, std::true_type{}, std::true_type{}) : go(dt, std::false_type{}, std::true_type{});
    };
    return dtype == KT_F16 ? typed(std::integral_constant<int, KT_F16>{}) : typed(std::integral_constant<int, KT_BF16>{});
}

}  // namespace kt
