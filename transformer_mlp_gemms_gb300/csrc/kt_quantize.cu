// kt_quantize.cu -- each row of the activations in signed 8-bit integers with one scale:
//   v = act(x),  scale = max|v| / 127,  q = the integer nearest to v / scale, ties to even.
//
// Bound by HBM: 2 bytes read and 1 written per element.  The row stays in the registers of a
// team of warps (kt_rows.cuh) between its largest magnitude and its rounding, so it is read
// once; the grid is persistent, and the next row's loads are in flight behind it.  The magnitudes
// are compared as the integers that their bits are, which orders NaN above infinity above every
// number, so one maximum (two 16-bit values at a time) also tells whether the row is finite.
//
// The nearest integer is decided exactly without a division per element: v times the rounded
// inverse of the scale is off by less than 127 * 2^-22 = 3.1e-5, so only a product within
// 1e-4 of a half-integer can go to the wrong side, and the exact remainder of those few tells.
// (A 64-bit division there instead took 66 us for 16384 x 1152: bf16 values have many ties with
// their row's maximum, and this GPU has next to no 64-bit rate.)  16384 x 1152 takes 14.3 us, 4.0
// TB/s, with 60% of the issue slots in use; 729 x 1152 2.9 us.
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

// 8 quotients as integers in the bytes of lo and hi; v holds the values.  `inv`: the scale's
// rounded inverse, in range.
__device__ __forceinline__ void quantize8(const f32x2 (&v)[4], float scale, float inv, uint32_t& lo, uint32_t& hi) {
    // adding 1.5 * 2^23 rounds to the nearest integer, ties to even, in the low bits
    constexpr float kMagic = 12582912.0f;
    uint32_t q[8];
    float off = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const f32x2 t = f2_mul<true>(v[e], f2(inv)), m = f2_add<true>(t, f2(kMagic));
        const f32x2 d = f2_sub<true>(t, f2_sub<true>(m, f2(kMagic)));
        off = fmaxf(off, fmaxf(fabsf(d.x), fabsf(d.y)));
        q[2 * e] = __float_as_uint(m.x);
        q[2 * e + 1] = __float_as_uint(m.y);
    }
    if (off > 0.4999f) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            q[2 * e] = (uint32_t)nearest_by_remainder(v[e].x, scale, (int)(__uint_as_float(q[2 * e]) - kMagic));
            q[2 * e + 1] = (uint32_t)nearest_by_remainder(v[e].y, scale, (int)(__uint_as_float(q[2 * e + 1]) - kMagic));
        }
    }
    lo = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
    hi = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
}
// The same for a scale whose inverse is out of range (a row of subnormals), 0 or NaN.
__device__ __noinline__ uint32_t quantize4_rare(float a, float b, float c, float d, float scale) {
    if (!(scale > 0.0f)) return 0u;
    return (uint32_t)(nearest_by_division(a, scale) & 255) | (uint32_t)(nearest_by_division(b, scale) & 255) << 8 |
           (uint32_t)(nearest_by_division(c, scale) & 255) << 16 | (uint32_t)(nearest_by_division(d, scale) & 255) << 24;
}

// Resident blocks per SM, as the registers allow.
constexpr int quant_per_sm(int W, bool ACT) { return ACT ? 1 : W == 16 ? 1 : 3; }

template <int DT, int W, int V, bool VEC, bool ACT>
__global__ void __launch_bounds__(row_block(W), quant_per_sm(W, ACT)) kt_quantize_kernel(const QuantRows p) {
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
        SlotAhead<VEC> n[V];  // the next row, on its way behind this one's reduction
        if (next < p.M) {
#pragma unroll
            for (int s = 0; s < V; ++s) n[s].load(X + (int64_t)next * p.ldx, s, l, TL, K);
        }
        f32x2 a[ACT ? 4 * V : 4];  // ACT: the row's activated values
        uint32_t most = 0;
        if constexpr (ACT) {
#pragma unroll
            for (int s = 0; s < V; ++s) {
                float v[8], g[8] = {};
                unpack8<DT>(c[s], v);
                if (p.act == KT_ACT_GEGLU) unpack8<DT>(load_slot<VEC>(X + (int64_t)row * p.ldx + K, s, l, TL, K), g);
                activate8(p.act, v, g);  // a column past the row: act(0) = 0
#pragma unroll
                for (int e = 0; e < 8; ++e) most = max(most, __float_as_uint(v[e]) & 0x7fffffffu);
#pragma unroll
                for (int e = 0; e < 4; ++e) a[4 * s + e] = f2(v[2 * e], v[2 * e + 1]);
            }
        } else {
            // the 16-bit patterns without their signs are ordered as the magnitudes are
            uint32_t m2 = 0;
#pragma unroll
            for (int s = 0; s < V; ++s)
                m2 = __vmaxu2(__vmaxu2(m2, __vmaxu2(c[s].x & 0x7fff7fffu, c[s].y & 0x7fff7fffu)),
                              __vmaxu2(c[s].z & 0x7fff7fffu, c[s].w & 0x7fff7fffu));
            float f[8];
            unpack8<DT>(make_uint4(max(m2 & 0xffffu, m2 >> 16), 0u, 0u, 0u), f);
            most = __float_as_uint(f[0]);
        }
        most = team_max<W>(most, lines, turn, team);
        const bool finite = most < 0x7f800000u;
        const float scale = finite ? __fdiv_rn(__uint_as_float(most), 127.0f) : __uint_as_float(0x7fffffffu);
        if (l == 0) p.scale[row] = scale;
        const bool fast = scale > 1e-37f;
        const float inv = fast ? __fdiv_rn(1.0f, scale) : 0.0f;
        int8_t* qr = p.Q + (int64_t)row * p.ldq;
#pragma unroll
        for (int s = 0; s < V; ++s) {
            f32x2 v[4];
            if constexpr (ACT) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = a[4 * s + e];
            } else {
                unpack_pairs<DT>(c[s], v);
            }
            uint32_t lo, hi;
            if (fast) {
                quantize8(v, scale, inv, lo, hi);
            } else {
                lo = quantize4_rare(v[0].x, v[0].y, v[1].x, v[1].y, scale);
                hi = quantize4_rare(v[2].x, v[2].y, v[3].x, v[3].y, scale);
            }
            if constexpr (VEC) {
                const int col = slot_col<true>(s, 0, l, TL);
                if (col < K) *reinterpret_cast<uint2*>(qr + col) = make_uint2(lo, hi);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int col = slot_col<false>(s, e, l, TL);
                    if (col < K) qr[col] = (int8_t)((e < 4 ? lo : hi) >> (8 * (e & 3)));
                }
            }
        }
        if (next >= p.M) break;
        row = next;
#pragma unroll
        for (int s = 0; s < V; ++s) c[s] = n[s].slot();
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
            constexpr int w = decltype(W)::value, t = decltype(dt)::value, v = decltype(V)::value;
            constexpr bool al16 = decltype(v16)::value, with_act = decltype(act)::value;
            constexpr int teams = row_block(w) / (32 * w), per_sm = quant_per_sm(w, with_act);
            const int64_t blocks = ((int64_t)p.M + teams - 1) / teams;
            const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)sms * per_sm);
            const cudaError_t e = launch_pdl(kt_quantize_kernel<t, w, v, al16, with_act>, grid, row_block(w), 0, stream, p);
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
