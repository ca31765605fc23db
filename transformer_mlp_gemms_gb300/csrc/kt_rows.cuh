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

// A slot on its way: the loads go out, and `slot` takes what came.  Without 16-byte loads the
// elements wait one by one: packing them where they are loaded would wait for them there (layer
// norm of 65536 x 642: 114 us, here 42; its gradients 107 and 85).
template <bool VEC>
struct SlotAhead {
    uint4 w;
    __device__ __forceinline__ void load(const uint16_t* __restrict__ row, int s, int l, int TL, int D) {
        w = load_slot<true>(row, s, l, TL, D);
    }
    __device__ __forceinline__ uint4 slot() const { return w; }
};
template <>
struct SlotAhead<false> {
    uint16_t u[8];
    __device__ __forceinline__ void load(const uint16_t* __restrict__ row, int s, int l, int TL, int D) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = slot_col<false>(s, e, l, TL);
            u[e] = 0;
            if (c < D) u[e] = row[c];
        }
    }
    __device__ __forceinline__ uint4 slot() const {
        return make_uint4(u[0] | (uint32_t)u[1] << 16, u[2] | (uint32_t)u[3] << 16, u[4] | (uint32_t)u[5] << 16, u[6] | (uint32_t)u[7] << 16);
    }
};

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

// Reductions over a team, the same bits in every lane.  Across warps they go through one of
// two shared-memory lines in turn, so one barrier per reduction is enough: a line is written
// again only after the next reduction's barrier, which every warp reaches after its reads.
template <int W>
struct TeamLines {
    float2 v[2][row_block(W) / 32];
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
        float2* line = lines.v[turn];
        if ((threadIdx.x & 31) == 0) line[warp] = make_float2(a, b);
        team_barrier<W>(team);
        a = b = 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float2 t = line[team * W + i];
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
        float2* line = lines.v[turn];
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

// Rows on their way from global memory in shared memory, `rows` of them ahead: each lane copies
// its own 16-byte slots asynchronously and reads only them, so nobody waits for another lane,
// and what is in flight costs no registers.  (One bulk copy per row by one lane of the team was
// slower than plain loads a row ahead: a copy takes its thread, and so its warp, about 0.1 us.)
template <int W, int V, int T>  // T tensors
struct RowRing {
    static constexpr int TL = 32 * W, teams = row_block(W) / TL;
    static constexpr int rows = V <= 2 ? 8 : V == 3 ? 6 : 4;
    static constexpr int bytes = rows * T * V * row_block(W) * 16;
    uint32_t base;  // this lane's first slot
    __device__ __forceinline__ void open(const uint8_t* smem, int team, int l) {
        base = smem_u32(smem) + (uint32_t)(team * rows * T * V * TL + l) * 16u;
    }
    __device__ __forceinline__ uint32_t at(int slot, int t, int s) const {
        return base + (uint32_t)(((slot * T + t) * V + s) * TL) * 16u;
    }
    __device__ __forceinline__ void copy(int slot, int t, const uint16_t* row, int l, int D) const {
#pragma unroll
        for (int s = 0; s < V; ++s) {
            const int c = 8 * (s * TL + l);
            // past the row's end: zeros, read from nowhere
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at(slot, t, s)), "l"(row + (c < D ? c : 0)), "r"(c < D ? 16 : 0)
                         : "memory");
        }
    }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    static __device__ __forceinline__ void wait_oldest() { asm volatile("cp.async.wait_group %0;" ::"n"(rows - 1) : "memory"); }
    __device__ __forceinline__ void read(int slot, int t, uint4 (&c)[V]) const {
#pragma unroll
        for (int s = 0; s < V; ++s)
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(c[s].x), "=r"(c[s].y), "=r"(c[s].z), "=r"(c[s].w) : "r"(at(slot, t, s)) : "memory");
    }
};

// gamma or beta as fp32 in shared memory, in the order in which the lanes read it: 16 bytes of
// slot s, half h (4 elements) of lane l at ((2 s + h) TL + l), so a warp's reads touch consecutive
// addresses.  Saves the registers that the packed values take and their unpacking in every row.
template <int DT, bool VEC, int W, int V>
__device__ __forceinline__ void stage_vector(const uint16_t* v, float4* to, int D) {
    constexpr int TL = 32 * W;
    for (int i = threadIdx.x; i < V * TL; i += row_block(W)) {
        const int s = i / TL, l = i % TL;
        float f[8];
        unpack8<DT>(load_slot<VEC>(v, s, l, TL, D), f);
        to[(2 * s) * TL + l] = make_float4(f[0], f[1], f[2], f[3]);
        to[(2 * s + 1) * TL + l] = make_float4(f[4], f[5], f[6], f[7]);
    }
}
template <int W>
__device__ __forceinline__ void staged_pairs(const float4* from, int s, int l, f32x2 (&f)[4]) {
    const float4 a = from[(2 * s) * 32 * W + l], b = from[(2 * s + 1) * 32 * W + l];
    f[0] = f2(a.x, a.y);
    f[1] = f2(a.z, a.w);
    f[2] = f2(b.x, b.y);
    f[3] = f2(b.z, b.w);
}
constexpr int staged_bytes(int W, int V) { return V * 32 * W * 8 * 4; }

// The same without 16-byte loads, for kernels whose lanes hold little else: from 2049
// columns on two slots per lane of more warps, as far as there are any, since the next row's elements
// take a register each (layer norm of 4000 x 4001: 25 us with four slots of 4 warps, here 20; below,
// the barriers cost more: 32768 x 1281 51 us with 2 warps, 78 with 4).
inline bool scalar_row_shape(int64_t D, RowShape* out) {
    if (!row_shape(D, out)) return false;
    if (out->W <= 2 || D > 32 * 16 * 2 * 8) return true;
    out->V = 2;
    for (out->W = 8; out->W < 16 && D > 32ll * out->W * 2 * 8;) out->W *= 2;
    return true;
}

// Calls f(integral constants W, V) for the team shape; 13 shapes with 16-byte loads, 8 (the
// shapes' slot counts rounded up; PAIRS: scalar_row_shape's) without.
template <bool VEC, bool PAIRS = false, typename F>
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
    if constexpr (PAIRS) {  // scalar_row_shape's
        KT_SHAPE(8, 2);
        KT_SHAPE(16, 2);
    } else {
        KT_SHAPE(4, 4);
        KT_SHAPE(8, 4);
    }
    KT_SHAPE(16, 4);
#undef KT_SHAPE
    return KT_ERR_UNSUPPORTED;
}

}  // namespace kt
