// kt_adamw.cu -- one AdamW step over many tensors in one launch, moments in fp32 or in 8 bits.
//
//   m = b1 m + (1 - b1) g,   v = b2 v + ((1 - b2) g) g,   r = sqrt(v),
//   p = p (1 - lr wd) - (m (lr / (1 - b1^t))) / (r / sqrt(1 - b2^t) + eps)
//
// in fp32 with every operation rounded on its own (no contraction), so that the step is the same bits
// whatever carries it out.  8-bit moments are e4m3 with a scale for each 256 values of a tensor: m, and r
// in the place of v, whose square would have twice the range; a root above zero is held as 2^-9 of its scale
// at least, since the step divides by it.
//
// Bound by memory with fp32 moments: 28 bytes per value with fp32 parameters, bf16 gradients and copies.  With 16-bit
// parameters and 8-bit moments there are 10 bytes and 59 instructions a value, and the instructions bind: 157 million
// values in 310 to 336 us, 4.7 to 5.1 TB/s, the schedulers busy 75 % of the time.  A warp takes 256 values at a time
// (a scale's block), eight consecutive ones per lane, and holds them in registers throughout: their
// largest magnitude is one warp reduction.  The tensors' addresses come as the launch's parameters, so no
// table is kept on the device, and a captured call carries its own.  A block takes every
// gridDim-th chunk, across tensors, so that what runs at a time lies together in memory.
#include <cuda_fp8.h>

#include "kt_ops_internal.h"
#include "kt_gemm.cuh"
#include "kt_exact.cuh"

namespace kt {
namespace {

constexpr int kAdBlock = 256, kAdWarps = 8, kAdChunk = kAdBlock * kAdWarps;  // values of a scale, of a thread block's round

template <int N>
struct AdTable {
    AdamwEntry e[N];
    int count;
    int64_t chunks;
    AdamwStep s;
};

// eight values as fp32, from consecutive elements or (STRIDED) from every 32nd, those past the end as zeros
template <int T, bool STRIDED>
__device__ __forceinline__ void ad_load(const void* at, int64_t i, int left, float* f) {
    if constexpr (!STRIDED) {
        if constexpr (T == KT_F32) {
            const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(at) + i);
            const float4 a = p[0], b = p[1];
            f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
        } else {
            unpack8<T>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(at) + i), f);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f[e] = 0.0f;
            if (32 * e < left) {
                if constexpr (T == KT_F32) {
                    f[e] = static_cast<const float*>(at)[i + 32 * e];
                } else {
                    float t[8];
                    unpack8<T>(make_uint4(static_cast<const uint16_t*>(at)[i + 32 * e], 0u, 0u, 0u), t);
                    f[e] = t[0];
                }
            }
        }
    }
}
template <int T, bool STRIDED>
__device__ __forceinline__ void ad_store(void* at, int64_t i, int left, const float* f) {
    if constexpr (!STRIDED) {
        if constexpr (T == KT_F32) {
            float4* p = reinterpret_cast<float4*>(static_cast<float*>(at) + i);
            p[0] = make_float4(f[0], f[1], f[2], f[3]);
            p[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(at) + i) =
                make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (32 * e < left) {
                if constexpr (T == KT_F32) static_cast<float*>(at)[i + 32 * e] = f[e];
                else static_cast<uint16_t*>(at)[i + 32 * e] = (uint16_t)(pack2<T>(f[e], 0.0f) & 0xffffu);
            }
    }
}

// eight e4m3 values
__device__ __forceinline__ void from_e4m3(uint2 w, float* f) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t u = j < 2 ? w.x : w.y;
        const float2 t = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u >> (16 * (j & 1))), __NV_E4M3)));
        f[2 * j] = t.x;
        f[2 * j + 1] = t.y;
    }
}
template <bool STRIDED>
__device__ __forceinline__ void ad_load8(const void* at, int64_t i, int left, float* f) {
    if constexpr (!STRIDED) {
        from_e4m3(*reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(at) + i), f);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f[e] = 0.0f;
            if (32 * e < left) f[e] = __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(at)[i + 32 * e], __NV_E4M3)));
        }
    }
}

// Eight values of this lane (32 lanes: a block of 256) in e4m3: the scale, most / 448, and each value times
// 448 / most, rounded to the nearest.  A block with no magnitude of 2^-100 or more is held as zeros (the
// quotient would overflow).  A NaN is the largest as bits, and makes the scale a NaN.  ROOT: what is above zero
// stays so (`positive`: all of this lane's are).
template <bool ROOT, bool STRIDED>
__device__ __forceinline__ void ad_store8(void* at, float* scale, int64_t i, int left, int lane, const float* f, bool positive) {
    float most = fabsf(f[0]);
#pragma unroll
    for (int e = 1; e < 8; ++e) most = max_nan(most, fabsf(f[e]));
    const float top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
    f32x2 both;  // most / 448, 448 / most
    if (top >= 0x1p-60f && top <= 0x1p60f) both = quotient_rn(f2(top, 448.0f), f2(448.0f, top), f2(-448.0f, -top));
    else both = top < 0x1p-100f ? f2(0.0f) : f2(__fdiv_rn(top, 448.0f), __fdiv_rn(448.0f, top));
    if (lane == 0) *scale = both.x;
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const f32x2 t = f2_mul<true>(f2(f[e], f[e + 1]), f2(both.y));
        q[e] = t.x, q[e + 1] = t.y;
    }
    if (ROOT) {
        if (positive) {
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] = max_nan(q[e], 0x1p-9f);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (q[e] > 0.0f) q[e] = fmaxf(q[e], 0x1p-9f);
        }
    }
    if constexpr (!STRIDED) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __nv_cvt_float2_to_fp8x2(make_float2(q[2 * j], q[2 * j + 1]), __NV_SATFINITE, __NV_E4M3);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(at) + i) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (32 * e < left) static_cast<uint8_t*>(at)[i + 32 * e] = __nv_cvt_float_to_fp8(q[e], __NV_SATFINITE, __NV_E4M3);
    }
}

// A lane's eight values of each kind on their way: copied into shared memory ahead of their turn, into places that
// this thread alone writes and reads.
template <int PT, int GT>
struct AdAhead {
    static constexpr int kStages = 3;
    static constexpr int kP = PT == KT_F32 ? 32 : 16, kG = GT == KT_F32 ? 32 : 16;
    static constexpr int kBytes = (kP + kG + 16) * kAdWarps * 32;  // of a stage: [16-byte piece][thread], m and v in one piece
    __device__ __forceinline__ static uint8_t* place(uint8_t* smem, int stage, int piece) {
        return smem + stage * kBytes + (piece * kAdWarps * 32 + (int)threadIdx.x) * 16;
    }
    __device__ __forceinline__ static void copy(uint8_t* to, const void* from) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
    }
    __device__ __forceinline__ static void copy8(uint8_t* to, const void* from) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(to)), "l"(from) : "memory");
    }
    __device__ __forceinline__ static void send(uint8_t* smem, int stage, const AdamwEntry& t, int64_t i) {
        const uint8_t *p = static_cast<const uint8_t*>(t.p) + i * (kP / 8), *g = static_cast<const uint8_t*>(t.g) + i * (kG / 8);
#pragma unroll
        for (int k = 0; k < kP / 16; ++k) copy(place(smem, stage, k), p + 16 * k);
#pragma unroll
        for (int k = 0; k < kG / 16; ++k) copy(place(smem, stage, kP / 16 + k), g + 16 * k);
        copy8(place(smem, stage, (kP + kG) / 16), static_cast<const uint8_t*>(t.m) + i);
        copy8(place(smem, stage, (kP + kG) / 16) + 8, static_cast<const uint8_t*>(t.v) + i);
    }
    template <int T>
    __device__ __forceinline__ static void take(uint8_t* smem, int stage, int piece, float* f) {
        const uint4 w = *reinterpret_cast<const uint4*>(place(smem, stage, piece));
        if constexpr (T == KT_F32) {
            const uint4 x = *reinterpret_cast<const uint4*>(place(smem, stage, piece + 1));
            const uint32_t u[8] = {w.x, w.y, w.z, w.w, x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(u[e]);
        } else {
            unpack8<T>(w, f);
        }
    }
};

// The step of 256 values of one tensor, from `at` on.  AHEAD: copied into the stage of shared memory before.
template <int PT, int GT, bool BITS8, bool STRIDED, bool AHEAD>
__device__ __forceinline__ void ad_block(const AdamwEntry& t, const AdamwStep& s, int64_t at, int lane, float rate, float root, float scale,
                                         uint8_t* smem, int stage, float2 scales) {
    const int64_t i = at + (STRIDED ? lane : 8 * lane);
    const int left = STRIDED ? (int)min((int64_t)kAdBlock, t.n - at) - lane : 256;
    float p[8], g[8], m[8], v[8], sm = 0.0f, sv = 0.0f;
    if constexpr (BITS8 && !AHEAD) {
        sm = t.ms[at / kAdBlock];
        sv = t.vs[at / kAdBlock];
    }
    if constexpr (AHEAD) {
        using A = AdAhead<PT, GT>;
        sm = scales.x;
        sv = scales.y;
        const uint4 w = *reinterpret_cast<const uint4*>(A::place(smem, stage, (A::kP + A::kG) / 16));
        from_e4m3(make_uint2(w.x, w.y), m);
        from_e4m3(make_uint2(w.z, w.w), v);
        A::template take<PT>(smem, stage, 0, p);
        A::template take<GT>(smem, stage, A::kP / 16, g);
    } else {
        ad_load<GT, STRIDED>(t.g, i, left, g);
        if constexpr (BITS8) {
            ad_load8<STRIDED>(t.m, i, left, m);
            ad_load8<STRIDED>(t.v, i, left, v);
        } else {
            ad_load<KT_F32, STRIDED>(t.m, i, left, m);
            ad_load<KT_F32, STRIDED>(t.v, i, left, v);
        }
        ad_load<PT, STRIDED>(t.p, i, left, p);
    }
    float r[8], a[8], d[8];  // the root; the step's numerator and the step, both with the other sign
    const f32x2 b1 = f2(s.b1), c1 = f2(s.c1), b2 = f2(s.b2), c2 = f2(s.c2), one = f2(s.one), minus_rate = f2(-rate);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        f32x2 gg = f2(g[e], g[e + 1]), mm = f2(m[e], m[e + 1]), vv = f2(v[e], v[e + 1]);
        if constexpr (BITS8) {
            mm = f2_mul<true>(mm, f2(sm));
            vv = f2_mul<true>(vv, f2(sv));
            vv = f2_mul<true>(vv, vv);
        }
        if (s.grad_scale) gg = f2_mul<true>(gg, f2(scale));
        mm = sum_rn(f2_mul<true>(mm, b1), f2_mul<true>(gg, c1), one);
        vv = sum_rn(f2_mul<true>(vv, b2), f2_mul<true>(f2_mul<true>(gg, c2), gg), one);
        const f32x2 aa = f2_mul<true>(mm, minus_rate);
        m[e] = mm.x, m[e + 1] = mm.y, v[e] = vv.x, v[e + 1] = vv.y, a[e] = aa.x, a[e + 1] = aa.y;
    }
    float v_least = v[0], v_most = v[0], a_least = fabsf(a[0]), a_most = fabsf(a[0]);
#pragma unroll
    for (int e = 1; e < 8; e += 2) {
        v_least = min3(v_least, v[e], v[e < 7 ? e + 1 : e]);
        v_most = max3(v_most, v[e], v[e < 7 ? e + 1 : e]);
        a_least = min3(a_least, fabsf(a[e]), fabsf(a[e < 7 ? e + 1 : e]));
        a_most = max3(a_most, fabsf(a[e]), fabsf(a[e < 7 ? e + 1 : e]));
    }
    // Within these the root lies in 2^-39 .. 2^30, the denominator in 2^-39 .. 2^51 (s.plain: eps and the correction are not
    // out of the way), the quotient in 2^-121 .. 2^99, and no residue is subnormal.  (A NaN may pass: it stays one.)
    const bool quick = s.plain && v_least >= 0x1p-78f && v_most <= 0x1p60f && a_least >= 0x1p-70f && a_most <= 0x1p60f;
    if (quick) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const f32x2 rr = root_rn(f2(v[e], v[e + 1]));
            const f32x2 w = f2_mul<true>(rr, f2(root));
            const f32x2 qq = quotient_rn(f2(a[e], a[e + 1]), sum_rn(w, f2(s.eps), one), sum_rn(w, f2(-s.eps), f2(-s.one)));
            r[e] = rr.x, r[e + 1] = rr.y, d[e] = qq.x, d[e + 1] = qq.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            r[e] = __fsqrt_rn(v[e]);
            d[e] = __fdiv_rn(a[e], __fadd_rn(__fmul_rn(r[e], root), s.eps));
        }
    }
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const f32x2 pp = sum_rn(f2_mul<true>(f2(p[e], p[e + 1]), f2(t.keep)), f2(d[e], d[e + 1]), one);
        p[e] = pp.x, p[e + 1] = pp.y;
    }
    ad_store<PT, STRIDED>(t.p, i, left, p);
    if (PT == KT_F32 && t.copy) {
        if (s.copy_dtype == KT_BF16) ad_store<KT_BF16, STRIDED>(t.copy, i, left, p);
        else ad_store<KT_F16, STRIDED>(t.copy, i, left, p);
    }
    if constexpr (BITS8) {
        if constexpr (STRIDED) {  // what is past the end has no part in the scale (its r would be the root of zero)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (32 * e >= left) m[e] = r[e] = 0.0f;
        }
        ad_store8<false, STRIDED>(t.m, t.ms + at / kAdBlock, i, left, lane, m, true);
        ad_store8<true, STRIDED>(t.v, t.vs + at / kAdBlock, i, left, lane, r, quick);
    } else {
        ad_store<KT_F32, STRIDED>(t.m, i, left, m);
        ad_store<KT_F32, STRIDED>(t.v, i, left, v);
    }
}

template <int PT, int GT, bool BITS8, int N>
__global__ void __launch_bounds__(kAdWarps * 32, 4) kt_adamw_kernel(const __grid_constant__ AdTable<N> tab) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const AdamwStep& s = tab.s;
    float rate = s.rate, root = s.root;
    if (s.step) {  // the step's number is on the device
        __shared__ float on_device[2];
        if (threadIdx.x == 0) {
            const double t = (double)*s.step;
            on_device[0] = (float)(s.lr / (1.0 - pow(s.beta1, t)));
            on_device[1] = (float)(1.0 / sqrt(1.0 - pow(s.beta2, t)));
        }
        __syncthreads();
        rate = on_device[0];
        root = on_device[1];
    }
    const float scale = s.grad_scale ? *s.grad_scale : 1.0f;
    int64_t c = blockIdx.x;
    const int64_t end = tab.chunks, step = gridDim.x;
    if (c >= end) return;
    int t = 0;
    for (int hi = tab.count; hi - t > 1;) {  // the last tensor whose first chunk is at or before c
        const int mid = (t + hi) >> 1;
        if (tab.e[mid].first <= c) t = mid;
        else hi = mid;
    }
    if constexpr (BITS8) {
        // chunks ahead of their turn, of their own tensor
        extern __shared__ __align__(16) uint8_t smem[];
        constexpr int kStages = AdAhead<PT, GT>::kStages;
        int ahead_t = t, ahead_stage = 0, stage = 0;
        float2 scales[kStages - 1] = {};  // of the chunks on their way
        auto send = [&](int64_t chunk, float2& s) {
            if (chunk < end) {
                while (ahead_t + 1 < tab.count && tab.e[ahead_t + 1].first <= chunk) ++ahead_t;
                const AdamwEntry& e = tab.e[ahead_t];
                const int64_t at = (chunk - e.first) * kAdChunk + warp * kAdBlock;
                if (e.wide && at + kAdBlock <= e.n) {
                    AdAhead<PT, GT>::send(smem, ahead_stage, e, at + 8 * lane);
                    s = make_float2(e.ms[at / kAdBlock], e.vs[at / kAdBlock]);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (++ahead_stage == kStages) ahead_stage = 0;
        };
#pragma unroll
        for (int k = 0; k < kStages - 1; ++k) send(c + k * step, scales[k]);
        for (; c < end; c += step) {
            const float2 now = scales[0];  // (moved on before the next are asked for, so that no move waits for a load)
#pragma unroll
            for (int k = 0; k + 2 < kStages; ++k) scales[k] = scales[k + 1];
            send(c + (kStages - 1) * step, scales[kStages - 2]);
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
            while (t + 1 < tab.count && tab.e[t + 1].first <= c) ++t;
            const AdamwEntry& e = tab.e[t];
            const int64_t at = (c - e.first) * kAdChunk + warp * kAdBlock;
            if (at < e.n) {
                if (e.wide && at + kAdBlock <= e.n) ad_block<PT, GT, true, false, true>(e, s, at, lane, rate, root, scale, smem, stage, now);
                else ad_block<PT, GT, true, true, false>(e, s, at, lane, rate, root, scale, nullptr, 0, float2{});
            }
            if (++stage == kStages) stage = 0;
        }
    } else {
        for (; c < end; c += step) {
            while (t + 1 < tab.count && tab.e[t + 1].first <= c) ++t;
            const AdamwEntry& e = tab.e[t];
            const int64_t at = (c - e.first) * kAdChunk + warp * kAdBlock;
            if (at >= e.n) continue;
            if (e.wide && at + kAdBlock <= e.n) ad_block<PT, GT, false, false, false>(e, s, at, lane, rate, root, scale, nullptr, 0, float2{});
            else ad_block<PT, GT, false, true, false>(e, s, at, lane, rate, root, scale, nullptr, 0, float2{});
        }
    }
}

template <int PT, int GT, bool BITS8, int N>
cudaError_t ad_launch(const AdamwEntry* e, int count, const AdamwStep& s, int sms, int device, void* stream) {
    AdTable<N> tab;
    int64_t chunks = 0;
    for (int i = 0; i < count; ++i) {
        tab.e[i] = e[i];
        tab.e[i].first = chunks;
        chunks += (e[i].n + kAdChunk - 1) / kAdChunk;
    }
    tab.count = count;
    tab.chunks = chunks;
    tab.s = s;
    if (chunks == 0) return cudaSuccess;
    const unsigned grid = (unsigned)std::min<int64_t>(chunks, (int64_t)sms * 16);
    constexpr int kSmem = BITS8 ? AdAhead<PT, GT>::kStages * AdAhead<PT, GT>::kBytes : 0;
    static SmemOptIn opt_in;
    if (const cudaError_t r = opt_in(kt_adamw_kernel<PT, GT, BITS8, N>, kSmem, device); r != cudaSuccess) return r;
    return launch_pdl(kt_adamw_kernel<PT, GT, BITS8, N>, grid, (unsigned)(kAdWarps * 32), (size_t)kSmem, stream, tab);
}

constexpr int kAdFew = 24, kAdMany = 360;
static_assert(sizeof(AdTable<kAdMany>) <= 32764, "a launch's parameters");

template <int PT, int GT, bool BITS8>
cudaError_t ad_all(const AdamwEntry* e, int count, const AdamwStep& s, int sms, int device, void* stream) {
    for (int at = 0; at < count; at += kAdMany) {
        const int n = std::min(count - at, kAdMany);
        const cudaError_t r = n <= kAdFew ? ad_launch<PT, GT, BITS8, kAdFew>(e + at, n, s, sms, device, stream)
                                          : ad_launch<PT, GT, BITS8, kAdMany>(e + at, n, s, sms, device, stream);
        if (r != cudaSuccess) return r;
    }
    return cudaSuccess;
}

template <int PT, int GT>
cudaError_t ad_bits(const AdamwEntry* e, int count, const AdamwStep& s, int sms, int device, void* stream) {
    return s.bits == 8 ? ad_all<PT, GT, true>(e, count, s, sms, device, stream) : ad_all<PT, GT, false>(e, count, s, sms, device, stream);
}
template <int PT>
cudaError_t ad_grads(const AdamwEntry* e, int count, const AdamwStep& s, int sms, int device, void* stream) {
    if (s.grad_dtype == KT_F32) return ad_bits<PT, KT_F32>(e, count, s, sms, device, stream);
    return s.grad_dtype == KT_BF16 ? ad_bits<PT, KT_BF16>(e, count, s, sms, device, stream) : ad_bits<PT, KT_F16>(e, count, s, sms, device, stream);
}

}  // namespace

kt_status launch_adamw(const AdamwEntry* e, int count, const AdamwStep& s, int sms, int device, void* stream, const char** why) {
    const cudaError_t r = s.param_dtype == KT_F32    ? ad_grads<KT_F32>(e, count, s, sms, device, stream)
                          : s.param_dtype == KT_BF16 ? ad_grads<KT_BF16>(e, count, s, sms, device, stream)
                                                     : ad_grads<KT_F16>(e, count, s, sms, device, stream);
    if (r != cudaSuccess) {
        *why = cudaGetErrorString(r);
        return KT_ERR_CUDA;
    }
    return KT_OK;
}

}  // namespace kt
