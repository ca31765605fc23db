// kt_rows.cuh -- one row of a matrix in the registers of a team of warps: what the layer
// norm kernels and the row quantiser share.
//
// A team of W warps (TL = 32 W lanes) holds a row of D 16-bit elements, V slots of 8
// elements per lane, packed in pairs.  With VEC a slot is one 16-byte load: slot s of lane l
// is columns 8 (s TL + l) .. + 7 (D a multiple of 8, every row 16-byte aligned).  Without it
// element e of slot s is column (8 s + e) TL + l: any D, pitch and alignment, 2-byte loads
// that still touch consecutive addresses across a warp.
#pragma once
#include "kt_gemm.cuh"
#include "kt_ops.h"

namespace kt {

constexpr int kRowThreads = 256;  // threads of a block: 8 / W teams (W = 16: 512, one team)
constexpr int row_block(int W) { return W * 32 > kRowThreads ? W * 32 : kRowThreads; }

// Team shape for rows of D columns: one warp with up to 5 slots (1280 columns), else the
// fewest warps that hold the row in 4.  Returns false where no team is large enough.
struct RowShape {
    int W, V;
};
inline bool row_shape(int64_t D, RowShape* out) {
    const int64_t vecs = (D + 7) / 8;
    int W = 1;
    if (vecs > 32 * 5) {
        W = 2;
        while (W < 16 && vecs > 32ll * W * 4) W *= 2;
        if (vecs > 32ll * W * 4) return false;
    }
    out->W = W;
    out->V = (int)((vecs + 32 * W - 1) / (32 * W));
    if (W > 1 && out->V < 3) out->V = 3;
    return true;
}

template <bool VEC>
__device__ __forceinline__ int slot_col(int s, int e, int l, int TL) {
    return VEC ? 8 * (s * TL + l) + e : (8 * s + e) * TL + l;
}

// Whether slot s is full for every lane at any D that gets this shape (row_shape, with_shape):
// with 16-byte loads all but the last of one warp's, and the first two of a wider team's.
template <bool VEC, int W, int V>
__device__ __forceinline__ constexpr bool slot_full(int s) {
    return VEC && (W == 1 ? s + 1 < V : s < 2);
}
// Sets the elements of slot s past the row's end to zero.
template <bool VEC, int W, int V>
__device__ __forceinline__ void clear_past_end(f32x2& d, int s, int pair, int l, int D) {
    if (slot_full<VEC, W, V>(s)) return;
    if (VEC) {  // a 16-byte slot is in the row or not as a whole
        if (slot_col<true>(s, 0, l, 32 * W) >= D) d = f2(0.0f);
    } else {
        if (slot_col<false>(s, 2 * pair, l, 32 * W) >= D) d.x = 0.0f;
        if (slot_col<false>(s, 2 * pair + 1, l, 32 * W) >= D) d.y = 0.0f;
    }
}

template <bool VEC>
__device__ __forceinline__ uint4 load_slot(const uint16_t* __restrict__ row, int s, int l, int TL, int D) {
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (VEC) {
        const int c = slot_col<true>(s, 0, l, TL);
        if (c < D) w = *reinterpret_cast<const uint4*>(row + c);
    } else {
        uint32_t u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = slot_col<false>(s, e, l, TL);
            u[e] = c < D ? (uint32_t)row[c] : 0u;
        }
        w = make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
    }
    return w;
}

template <bool VEC>
__device__ __forceinline__ void store_slot(uint16_t* __restrict__ row, int s, int l, int TL, int D, const uint4& w) {
    if constexpr (VEC) {
        const int c = slot_col<true>(s, 0, l, TL);
        if (c < D) *reinterpret_cast<uint4*>(row + c) = w;
    } else {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = slot_col<false>(s, e, l, TL);
            if (c < D) row[c] = (uint16_t)(u[e >> 1] >> (16 * (e & 1)));
        }
    }
}

// A slot's 8 values as pairs, for the paired fp32 instructions.
template <int DT>
__device__ __forceinline__ void unpack_pairs(const uint4& w, f32x2 (&f)[4]) {
    float t[8];
    unpack8<DT>(w, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2(t[2 * i], t[2 * i + 1]);
}
template <int DT>
__device__ __forceinline__ uint4 pack_pairs(const f32x2 (&f)[4]) {
    return make_uint4(pack2<DT>(f[0].x, f[0].y), pack2<DT>(f[1].x, f[1].y), pack2<DT>(f[2].x, f[2].y), pack2<DT>(f[3].x, f[3].y));
}
// Makes the next unpacking of these slots a new one: the unpacked values of an earlier pass would
// take four times the packed ones' registers to keep.
template <int V>
__device__ __forceinline__ void forget_unpacked(uint4 (&c)[V]) {
#pragma unroll
    for (int s = 0; s < V; ++s) asm volatile("" : "+r"(c[s].x), "+r"(c[s].y), "+r"(c[s].z), "+r"(c[s].w));
}

template <int DT>
__device__ __forceinline__ uint4 pack8(const float* y) {
    return make_uint4(pack2<DT>(y[0], y[1]), pack2<DT>(y[2], y[3]), pack2<DT>(y[4], y[5]), pack2<DT>(y[6], y[7]));
}

// Reductions over a team, the same bits in every lane.  Across warps they go through one of
// two shared-memory lines in turn, so one barrier per reduction is enough: a line is written
// again only after the next reduction's barrier, which every warp reaches after its reads.
template <int W>
struct TeamLines {
    float4 v[2][row_block(W) / 32];
};
template <int W>
__device__ __forceinline__ void team_barrier(int team) {
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(32 * W) : "memory");
}
__device__ __forceinline__ float warp_add(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
// Sums of a and b over the team.
template <int W>
__device__ __forceinline__ void team_add2(float& a, float& b, TeamLines<W>& lines, int& turn, int team) {
    a = warp_add(a);
    b = warp_add(b);
    if constexpr (W > 1) {
        const int warp = threadIdx.x >> 5;
        float4* line = lines.v[turn];
        if ((threadIdx.x & 31) == 0) line[warp] = make_float4(a, b, 0.0f, 0.0f);
        team_barrier<W>(team);
        a = b = 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float4 t = line[team * W + i];
            a += t.x;
            b += t.y;
        }
        turn ^= 1;
    }
}
// Largest of unsigned values over the team.
template <int W>
__device__ __forceinline__ uint32_t team_max(uint32_t x, TeamLines<W>& lines, int& turn, int team) {
    x = __reduce_max_sync(0xffffffffu, x);
    if constexpr (W > 1) {
        const int warp = threadIdx.x >> 5;
        float4* line = lines.v[turn];
        if ((threadIdx.x & 31) == 0) line[warp].x = __uint_as_float(x);
        team_barrier<W>(team);
        x = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const uint32_t t = __float_as_uint(line[team * W + i].x);
            x = t > x ? t : x;
        }
        turn ^= 1;
    }
    return x;
}

// Calls f(integral constants W, V) for the team shape; 13 shapes with 16-byte loads, 8 (the
// shapes' slot counts rounded up) without.
template <bool VEC, typename F>
kt_status with_shape(const RowShape& s, F&& f) {
#define KT_SHAPE(w, v) \
    if (s.W == w && s.V <= v) return f(std::integral_constant<int, w>{}, std::integral_constant<int, v>{})
    if constexpr (VEC) {
        KT_SHAPE(1, 1);
        KT_SHAPE(1, 2);
    } else {
        KT_SHAPE(1, 1);
    }
    KT_SHAPE(1, 3);
    if constexpr (VEC) KT_SHAPE(1, 4);
    KT_SHAPE(1, 5);
    if constexpr (VEC) {
        KT_SHAPE(2, 3);
        KT_SHAPE(4, 3);
        KT_SHAPE(8, 3);
        KT_SHAPE(16, 3);
    }
    KT_SHAPE(2, 4);
    KT_SHAPE(4, 4);
    KT_SHAPE(8, 4);
    KT_SHAPE(16, 4);
#undef KT_SHAPE
    return KT_ERR_UNSUPPORTED;
}

}  // namespace kt
