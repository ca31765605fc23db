// kt_glu.cu -- the elementwise part of a gated block's backward pass, with the bias gradient's sums:
//
//   p = [value | gate]:  dvalue = dh * act(gate),  dgate = dh * value * act'(gate),
//   db = the sums of [dvalue | dgate] over the rows, taken before the rounding to 16 bits;
//
// and, without p, the column sums of dh alone (a linear layer's bias gradient).
//
// Bound by memory: 10 bytes per hidden element (2 of dh, 4 of p, 4 of dp).  The two products behind it
// read dp from L2 or memory as their operand, so it has to be there as a 16-bit matrix: that rounding
// is the backward pass's one besides its results'.  16384 x 5120: 839 MB in 131 to 141 us, 6.0 to 6.4 TB/s.
#include "kt_ops_internal.h"
#include "kt_gemm.cuh"

namespace kt {
namespace {

constexpr int kGluThreads = 256, kGluAhead = 4;

// act(g) and act'(g) of a pair.  With s the sigmoid of c(g): act = g s, act' = s + g s (1 - s) c'; 1 - s
// is taken as s times the exponential, which keeps its digits where s is near 1.
template <int EPI>
__device__ __forceinline__ void gate_slopes(f32x2 g, f32x2& a, f32x2& da) {
    constexpr bool P = true;
    if constexpr (EPI == EPI_GELU_ERF) {
        // act = g Phi(g), act' = Phi(g) + g phi(g); Phi(-|g|) as in gelu_erf_f2
        using namespace erfc_fit;
        const f32x2 az = f2(fabsf(g.x), fabsf(g.y));
        const f32x2 u = f2_mul<P>(az, f2(kU)), nu = f2_mul<P>(az, f2(-kU));
        const f32x2 tp = f2_rcp(f2_fma<P>(u, f2(kA), f2(2.0f)));
        f32x2 q = f2_fma<P>(f2(kQ9), tp, f2(kQ8));
        q = f2_fma<P>(q, tp, f2(kQ7));
        q = f2_fma<P>(q, tp, f2(kQ6));
        q = f2_fma<P>(q, tp, f2(kQ5));
        q = f2_fma<P>(q, tp, f2(kQ4));
        q = f2_fma<P>(q, tp, f2(kQ3));
        q = f2_fma<P>(q, tp, f2(kQ2));
        q = f2_fma<P>(q, tp, f2(kQ1));
        q = f2_fma<P>(q, tp, f2(kQ0));
        const f32x2 tail = f2_mul<P>(tp, f2_ex2(f2_fma<P>(nu, u, q)));  // Phi(-|g|)
        const f32x2 rest = f2_sub<P>(f2(1.0f), tail);
        const f32x2 phi = f2(g.x >= 0.0f ? rest.x : tail.x, g.y >= 0.0f ? rest.y : tail.y);
        // the density: exp(-g^2 / 2) / sqrt(2 pi) = 2^(-u^2) / sqrt(2 pi)
        const f32x2 density = f2_mul<P>(f2_ex2(f2_mul<P>(nu, u)), f2(0.3989422804014327f));
        a = f2_mul<P>(g, phi);
        // an infinite gate's density is 0, and so is its term
        const f32x2 term = f2_mul<P>(g, density);
        da = f2_add<P>(phi, f2(density.x == 0.0f ? 0.0f : term.x, density.y == 0.0f ? 0.0f : term.y));
    } else if constexpr (EPI == EPI_NONE) {
        a = g;
        da = f2(1.0f);
    } else {
        f32x2 x, slope;  // the sigmoid's exponent in powers of two, and its argument's derivative
        if constexpr (EPI == EPI_GELU_TANH) {
            const f32x2 g2 = f2_mul<P>(g, g);
            x = f2_mul<P>(g, f2_fma<P>(f2(-0.1029432395800235f), g2, f2(-2.302208198144325f)));
            slope = f2_fma<P>(f2(0.21406571f), g2, f2(1.5957691216057308f));  // 2 sqrt(2/pi) (1 + 3 0.044715 g^2)
        } else {
            constexpr float c = EPI == EPI_SILU ? 1.0f : 1.702f;
            x = f2_mul<P>(g, f2(EPI == EPI_SILU ? -1.4426950408889634f : -2.4554669595930157f));
            slope = f2(c);
        }
        const f32x2 e = f2_ex2(x);
        const f32x2 s = f2_rcp(f2_add<P>(f2(1.0f), e));
        a = f2_mul<P>(g, s);
        // s (1 - s) = s^2 e; far out on the negative side e overflows where s is 0, and the term is 0
        const f32x2 term = f2_mul<P>(f2_mul<P>(a, slope), f2_mul<P>(s, e));
        da = f2_add<P>(s, f2(s.x == 0.0f || e.x == 0.0f ? 0.0f : term.x, s.y == 0.0f || e.y == 0.0f ? 0.0f : term.y));
    }
}

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

// The flags of the products behind this kernel.
__device__ __forceinline__ void zero_flags(int* at) {
    if (at && blockIdx.x == 0 && blockIdx.y == 0)
        for (int i = threadIdx.x; i < (int)(kGradientsFlags / sizeof(int)); i += blockDim.x) at[i] = 0;
}
__global__ void __launch_bounds__(256) kt_zero_kernel(int* at) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    zero_flags(at);
}

// Block (x, y): 8 << log columns, rows [y per, (y + 1) per); 1 << log lanes take a row, 8 columns each, and every
// (256 >> log)-th row, four of them on their way at a time.  EPI < 0: the sums of dh alone.
template <int DT, int EPI>
__global__ void __launch_bounds__(kGluThreads) kt_glu_backward_kernel(const GluBackward p, int per, int log) {
    constexpr bool GATED = EPI >= 0;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    zero_flags(p.zero);
    const int lane = threadIdx.x & ((1 << log) - 1), first = threadIdx.x >> log, across = kGluThreads >> log, cols = 8 << log;
    const int col = (int)blockIdx.x * cols + 8 * lane;
    const bool mine = col < p.F;
    const int row0 = (int)blockIdx.y * per, row1 = min(row0 + per, p.M);
    f32x2 sv[4], sg[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sv[i] = sg[i] = f2(0.0f);
    const uint16_t* dH = static_cast<const uint16_t*>(p.dH) + col;
    const uint16_t* P = static_cast<const uint16_t*>(p.P) + col;
    uint16_t* dP = static_cast<uint16_t*>(p.dP) + col;
    if (mine)
        for (int r = row0 + first; r < row1; r += across * kGluAhead) {
            uint4 h[kGluAhead], v[kGluAhead], g[kGluAhead];
#pragma unroll
            for (int j = 0; j < kGluAhead; ++j) {
                const int64_t row = r + j * across;
                if (row < row1) {
                    h[j] = *reinterpret_cast<const uint4*>(dH + row * p.lddh);
                    if constexpr (GATED) {
                        v[j] = *reinterpret_cast<const uint4*>(P + row * p.ldp);
                        g[j] = *reinterpret_cast<const uint4*>(P + row * p.ldp + p.F);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kGluAhead; ++j) {
                const int64_t row = r + j * across;
                if (row >= row1) break;
                f32x2 dh[4];
                unpack_pairs<DT>(h[j], dh);
                if constexpr (GATED) {
                    f32x2 val[4], gate[4], dv[4], dg[4];
                    unpack_pairs<DT>(v[j], val);
                    unpack_pairs<DT>(g[j], gate);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        f32x2 a, da;
                        gate_slopes<EPI>(gate[i], a, da);
                        dv[i] = f2_mul<true>(dh[i], a);
                        dg[i] = f2_mul<true>(f2_mul<true>(dh[i], val[i]), da);
                        sv[i] = f2_add<true>(sv[i], dv[i]);
                        sg[i] = f2_add<true>(sg[i], dg[i]);
                    }
                    *reinterpret_cast<uint4*>(dP + row * p.lddp) = pack_pairs<DT>(dv);
                    *reinterpret_cast<uint4*>(dP + row * p.lddp + p.F) = pack_pairs<DT>(dg);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) sv[i] = f2_add<true>(sv[i], dh[i]);
                }
            }
        }
    if (!p.partials) return;
    // the sums of the block's rows, in the order of the first ones
    __shared__ float sums[8 * kGluThreads];  // [across][cols]
    float* to = p.partials + (int64_t)blockIdx.y * (GATED ? 2 : 1) * p.F + (int64_t)blockIdx.x * cols;
    const int c = (int)threadIdx.x;
#pragma unroll
    for (int part = 0; part < (GATED ? 2 : 1); ++part) {
        const f32x2* s = part ? sg : sv;
        if (part) __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<float2*>(&sums[first * cols + 8 * lane + 2 * i]) = make_float2(s[i].x, s[i].y);
        __syncthreads();
        if (c < cols && (int)blockIdx.x * cols + c < p.F) {
            float t = 0.0f;
#pragma unroll 8
            for (int w = 0; w < across; ++w) t += sums[w * cols + c];
            to[(int64_t)part * p.F + c] = t;
        }
    }
}

// db[c] = the sum of `rows` partial sums (kMostRows at most), in a fixed order: a warp takes every eighth, all of them on
// their way at a time.
constexpr int kMostRows = 128;
__global__ void __launch_bounds__(256) kt_column_sums_kernel(const float* partials, float* db, int rows, int cols) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float sums[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = (int)blockIdx.x * 32 + lane;
    float x[kMostRows / 8];
#pragma unroll
    for (int i = 0; i < kMostRows / 8; ++i) x[i] = warp + 8 * i < rows && c < cols ? partials[(int64_t)(warp + 8 * i) * cols + c] : 0.0f;
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < kMostRows / 8; ++i) t += x[i];
    sums[warp][lane] = t;
    __syncthreads();
    if (warp || c >= cols) return;
    t = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += sums[w][lane];
    db[c] = t;
}

template <int DT, int EPI>
cudaError_t glu_launch(const GluBackward& p, int rows, int per, int log, void* stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.F + (8 << log) - 1) / (8 << log)), (unsigned)rows, 1);
    cfg.blockDim = dim3(kGluThreads, 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kt_glu_backward_kernel<DT, EPI>, p, per, log);
}

template <int DT>
cudaError_t glu_dispatch(const GluBackward& p, int rows, int per, int log, void* stream) {
    if (!p.P) return glu_launch<DT, -1>(p, rows, per, log, stream);
    switch (p.act) {
        case EPI_GELU_ERF: return glu_launch<DT, EPI_GELU_ERF>(p, rows, per, log, stream);
        case EPI_GELU_TANH: return glu_launch<DT, EPI_GELU_TANH>(p, rows, per, log, stream);
        case EPI_GELU_SIGMOID: return glu_launch<DT, EPI_GELU_SIGMOID>(p, rows, per, log, stream);
        case EPI_SILU: return glu_launch<DT, EPI_SILU>(p, rows, per, log, stream);
        default: return glu_launch<DT, EPI_NONE>(p, rows, per, log, stream);
    }
}

}  // namespace

// The columns of a block, as a power of two of lanes: 256, or 128 or 64 where that leaves a tenth fewer lanes without
// columns (16147 x 320, erf: 13.2 -> 9.1 us; 15673 x 72: 12.0 -> 6.8).
static int glu_log(int64_t F) {
    auto lanes = [&](int log) { return (F + (8 << log) - 1) / (8 << log) << log; };
    int best = 5;
    for (int log = 4; log >= 3; --log)
        if (10 * lanes(log) < 9 * lanes(best)) best = log;
    return best;
}

// Rows of blocks (and of partial sums): enough blocks for eight per SM, 32 rows each at least, and no more
// than kMostRows partial sums per column.
int column_sum_rows(int64_t M, int64_t F) {
    const int64_t cols = 8 << glu_log(F), across = (F + cols - 1) / cols, most = (M + 31) / 32;
    return (int)std::max<int64_t>(1, std::min({most, (1216 + across - 1) / across, (int64_t)kMostRows}));
}

kt_status launch_zero(int* at, void* stream, const char** why) {
    const cudaError_t e = launch_pdl(kt_zero_kernel, 1u, 256u, (size_t)0, stream, at);
    if (e == cudaSuccess) return KT_OK;
    *why = cudaGetErrorString(e);
    return KT_ERR_CUDA;
}

kt_status launch_glu_backward(int dtype, const GluBackward& p, void* stream, const char** why) {
    int rows = column_sum_rows(p.M, p.F);
    const int log = glu_log(p.F);
    const int per = (p.M + rows - 1) / rows;
    rows = (p.M + per - 1) / per;
    GluBackward q = p;
    if (p.partials && rows == 1) q.partials = p.db;
    cudaError_t e = dtype == KT_BF16 ? glu_dispatch<KT_BF16>(q, rows, per, log, stream) : glu_dispatch<KT_F16>(q, rows, per, log, stream);
    if (e == cudaSuccess && p.partials && rows > 1) {
        const int cols = p.P ? 2 * p.F : p.F;
        e = launch_pdl(kt_column_sums_kernel, (unsigned)((cols + 31) / 32), 256u, (size_t)0, stream, p.partials, p.db, rows, cols);
    }
    if (e != cudaSuccess) {
        *why = cudaGetErrorString(e);
        return KT_ERR_CUDA;
    }
    return KT_OK;
}

}  // namespace kt
