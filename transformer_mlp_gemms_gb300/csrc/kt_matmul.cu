// kt_matmul.cu -- products of 16-bit matrices in whichever order their operands lie in memory, for the
// training step of a feed-forward block:
//
//   C[M][N] = round(A . B^T (+ bias)),  A: [M][K] or, a_mn, [K][M];  B: [N][K] or, b_mn, [K][N]
//
// A linear layer is A = X, B = W; its gradient dX = dY W has B = W by its other side (b_mn), and
// dW = dY^T X both operands by theirs.  GATED (kt_glu_forward): B holds F value rows, then F gate rows;
// a tile takes value and gate rows of the same columns, so that its epilogue has both and stores
// h = value * act(gate), and p = [value | gate] where a backward pass will want it.
//
// The structure is kt_gemm.cuh's with both operands free in their order: TMA copies of 64-deep
// steps into a ring in shared memory (K-major boxes of 64 columns, or boxes of 64 rows along K and 64
// columns, both under the 128-byte swizzle), tcgen05.mma into one of two fp32 accumulators, and eight
// epilogue warps.  One CTA per tile of 128 rows or a pair per 256 (cta_group::2); persistent, the
// tiles in bands of kBand tile rows so that what runs at a time shares its operands in L2.
//   warp 0: copies of A, and each step's byte count; warp 10: copies of B; warp 1: products;
//   warps 2-9: epilogue.
// SPLIT: few tiles with long sums (a gradient's dX of few tokens): a cluster per tile, each CTA with its
// share of the steps; the fp32 sums meet in the cluster's shared memory, added in the order of the ranks.
//
// Every wait is bounded: one that runs out leaves an error word and NaN in the elements that the call
// could not compute.
#include "kt_ops_internal.h"
#include "kt_gemm.cuh"
#include "kt_matmul.cuh"

namespace kt {

__device__ int g_matmul_error;

namespace {

constexpr int kMmThreads = 11 * 32;
constexpr int kMmEpi = 8;
constexpr uint32_t kMmABytes = 128 * 128;  // one step of 128 rows

struct MmParams {
    int M, N;                 // of the output (GATED: N = F)
    int BN, tiles_m, tiles_n, kblocks, stages;
    int a_mn, b_mn, act, has_p;
    uint32_t idesc, b_bytes;  // b_bytes: one step of this CTA's share of B
    const void* bias;
    unsigned long long wait_limit_ns, stall_ns;
};

// GATED: the activation of 32 gates times their values, packed.
template <int DT, int EPI>
__device__ __forceinline__ void gate32(const float* v, const float* g, uint32_t* w) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const f32x2 h = f2_mul<true>(f2(v[2 * i], v[2 * i + 1]), act_f2<EPI, true>(f2(g[2 * i], g[2 * i + 1])));
        w[i] = pack2<DT>(h.x, h.y);
    }
}

template <int DT>
__device__ __forceinline__ void pack32(const float* v, uint32_t* w) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack2<DT>(v[2 * i], v[2 * i + 1]);
}

template <int DT, int PAIR, bool GATED, bool SPLIT>
__global__ void __launch_bounds__(kMmThreads, 1)
    kt_matmul_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmG, const __grid_constant__ MmParams p) {
    static_assert(!(SPLIT && (GATED || PAIR == 2)), "a split tile is one CTA's, not gated");
    extern __shared__ uint8_t raw[];
    uint8_t* const at = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t base = smem_u32(at);
    const uint32_t stage_bytes = kMmABytes + p.b_bytes;
    const uint32_t staging = base + (uint32_t)p.stages * stage_bytes;  // two 2 KB buffers per epilogue warp
    const uint32_t bars = staging + kMmEpi * 4096u;
    const uint32_t bar_full = bars, bar_empty = bars + 64u, bar_accf = bars + 128u, bar_acce = bars + 144u, bar_drain = bars + 160u,
                   bar_stall = bars + 168u;
    uint32_t* const words = reinterpret_cast<uint32_t*>(at + (bars - base) + 176u);
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(words + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned long long limit = p.wait_limit_ns;
    const uint32_t rank = PAIR == 2 ? (cluster_ctarank() & 1u) : 0u;
    const int splits = SPLIT ? (int)cluster_size() : 1, part = SPLIT ? (int)cluster_ctarank() : 0;
    const bool leader = rank == 0;
    const int unit0 = (int)blockIdx.x / (PAIR * splits), units = (int)gridDim.x / (PAIR * splits);
    const int tiles = p.tiles_m * p.tiles_n;
    const int kb_from = SPLIT ? (int)((int64_t)p.kblocks * part / splits) : 0;
    const int kb_to = SPLIT ? (int)((int64_t)p.kblocks * (part + 1) / splits) : p.kblocks;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(bar_full + 8u * s, 1);
            mbar_init(bar_empty + 8u * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_accf + 8u * b, 1);
            mbar_init(bar_acce + 8u * b, kMmEpi * PAIR);
        }
        mbar_init(bar_drain, 1);
        mbar_init(bar_stall, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
        prefetch_tmap(&tmC);
    }
    if (warp == 1) tmem_alloc<PAIR>(smem_u32(words), kTmemCols);
    tc_fence_before();
    __syncthreads();
    if (PAIR == 2) cluster_sync_relaxed();  // the other CTA's barriers are initialised before any signal to them
    tc_fence_after();
    const uint32_t tmem = words[0];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // first row of A and first row of B (GATED: value row) of this CTA's part of tile t
    auto origin = [&](int t, int& m, int& n) {
        int tm, tn;
        band_tile(t, p.tiles_m, p.tiles_n, tm, tn);
        m = (tm * PAIR + (int)rank) * 128;
        n = tn * (GATED ? p.BN / 2 : p.BN) + (int)rank * (GATED ? p.BN / 2 / PAIR : p.BN / PAIR);
    };

    if (warp == 0 || warp == 10) {
        // ------------------- copies -------------------
        if (lane == 0) {
            const bool a_role = warp == 0;
            uint32_t stage = 0, phase = 0, used = 0, used_phase = 0;
            if (a_role && p.stall_ns && blockIdx.x == 0)  // the tests' hook: nobody signals this barrier
                wait_phase(bar_stall, 0, abort_flag, &g_matmul_error, DEV_INJECTED_STALL, p.stall_ns);
            for (int t = unit0; t < tiles && !*abort_flag; t += units) {
                int m, n;
                origin(t, m, n);
                for (int kb = kb_from; kb < kb_to; ++kb) {
                    if (!wait_phase(bar_empty + 8u * stage, phase ^ 1u, abort_flag, &g_matmul_error, DEV_TIMEOUT_PRODUCER, limit)) break;
                    const uint32_t sA = base + stage * stage_bytes, sB = sA + kMmABytes;
                    const uint32_t fb = PAIR == 2 ? mapa_rank(bar_full + 8u * stage, 0) : bar_full + 8u * stage;
                    auto load = [&](uint32_t dst, const CUtensorMap* tm, int x, int y) {
                        if constexpr (PAIR == 2) tma_load_2d_pair(dst, tm, fb, x, y);
                        else tma_load_2d(dst, tm, fb, x, y);
                    };
                    const int k = kb * kAtomK;
                    if (a_role) {
                        if (leader) mbar_arrive_expect_tx(bar_full + 8u * stage, PAIR * stage_bytes);
                        if (p.a_mn) {
                            load(sA, &tmA, m, k);
                            load(sA + 8192u, &tmA, m + 64, k);
                        } else {
                            load(sA, &tmA, k, m);
                        }
                        used |= 1u << stage;
                        used_phase = (used_phase & ~(1u << stage)) | (phase << stage);
                    } else if (GATED) {
                        load(sB, &tmB, k, n);
                        load(sB + p.b_bytes / 2, &tmB, k, p.N + n);
                    } else if (p.b_mn) {
                        for (uint32_t j = 0; j < p.b_bytes; j += 8192u) load(sB + j, &tmB, n + (int)(j / 128u), k);
                    } else {
                        load(sB, &tmB, k, n);
                    }
                    if (++stage == (uint32_t)p.stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (*abort_flag) {
                // no copy may still be on its way into memory that is about to be released: the byte
                // counts cover both CTAs' copies, and what was never counted gets 100 us to land
                if (a_role && leader)
                    for (int s = 0; s < p.stages; ++s)
                        if (used & (1u << s)) wait_drain(bar_full + 8u * s, (used_phase >> s) & 1u, 100000000ull);
                const unsigned long long t0 = global_ns();
                while (global_ns() - t0 < 100000ull) __nanosleep(1000);
            }
        }
    } else if (warp == 1) {
        // ------------------- products -------------------
        if (lane == 0 && leader) {
            uint32_t stage = 0, phase = 0;
            const uint64_t ad0 = smem_desc(base, p.a_mn ? 8192u : 16u, 1024u);
            const uint64_t bd0 = smem_desc(base + kMmABytes, p.b_mn ? 8192u : 16u, 1024u);
            // 16 columns of K further: 32 bytes of a K-major row, 16 rows of an MN-major box
            const uint32_t a_step = p.a_mn ? 128u : 2u, b_step = p.b_mn ? 128u : 2u, stage16 = stage_bytes >> 4;
            bool ok = true, any = false;
            int local = 0;
            for (int t = unit0; t < tiles && ok; t += units, ++local) {
                const uint32_t buf = local & 1, d = tmem + buf * (uint32_t)kAccSlot;
                if (!wait_phase<PAIR == 2>(bar_acce + 8u * buf, ((local >> 1) & 1u) ^ 1u, abort_flag, &g_matmul_error, DEV_TIMEOUT_MMA, limit)) break;
                tc_fence_after();
                for (int kb = kb_from; kb < kb_to; ++kb) {
                    const uint32_t fb = bar_full + 8u * stage;
                    if (!mbar_test_wait(fb, phase) && !wait_phase(fb, phase, abort_flag, &g_matmul_error, DEV_TIMEOUT_MMA, limit)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = ad0 + stage * stage16, bd = bd0 + stage * stage16;
#pragma unroll
                    for (uint32_t k = 0; k < 4; ++k) {
                        const uint32_t acc = kb > kb_from || k > 0;
                        if constexpr (PAIR == 2) mma_f16_pair(d, ad + k * a_step, bd + k * b_step, p.idesc, acc);
                        else mma_f16(d, ad + k * a_step, bd + k * b_step, p.idesc, acc);
                    }
                    any = true;
                    if constexpr (PAIR == 2) mma_commit_pair(bar_empty + 8u * stage);
                    else mma_commit(bar_empty + 8u * stage);
                    if (++stage == (uint32_t)p.stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                if constexpr (PAIR == 2) mma_commit_pair(bar_accf + 8u * buf);
                else mma_commit(bar_accf + 8u * buf);
            }
            if (*abort_flag && any) {  // no product may still be running when tensor memory is freed
                if constexpr (PAIR == 2) mma_commit_pair(bar_drain);
                else mma_commit(bar_drain);
                wait_drain(bar_drain, 0u, 100000000ull);
            }
        }
        __syncwarp();
    } else {
        // ------------------- epilogue -------------------
        const int ew = warp - 2, q = warp & 3, half = ew >> 2;  // this warp's lanes of tensor memory, its column groups
        const uint32_t stg = staging + (uint32_t)ew * 4096u;
        uint32_t stores = 0;
        bool ok = true;
        int local = 0;
        for (int t = unit0; t < tiles; t += units, ++local) {
            const uint32_t buf = local & 1;
            ok = ok && wait_phase(bar_accf + 8u * buf, (local >> 1) & 1u, abort_flag, &g_matmul_error, DEV_TIMEOUT_EPILOGUE, limit);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            int m, n;
            origin(t, m, n);
            if (PAIR == 2) n -= (int)rank * (GATED ? p.BN / 4 : p.BN / 2);  // every column of the tile
            const int y = m + 32 * q;
            const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + buf * (uint32_t)kAccSlot;
            // 32 columns of the accumulator (NaN where there is none), with their bias
            auto columns = [&](uint32_t from, const uint16_t* bias, int col, int limit_col, float* v) {
                uint32_t r[32];
                if (ok) {
                    tmem_ld32(acc + from, r);
                    tmem_wait_ld_only();
                    reg_fence32(r);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) r[i] = 0x7fffffffu;
                }
                if (bias) {
                    bias32<DT>(bias, col, limit_col, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] += __uint_as_float(r[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
                }
            };
            auto store = [&](const CUtensorMap* tm, const uint32_t* w, int col) {
                stage_and_store_packed(tm, stg + (stores++ & 1u) * 2048u, lane, w, col, y, true);
            };
            const uint16_t* bias = static_cast<const uint16_t*>(p.bias);
            if constexpr (SPLIT) {
                // the sums go where the operands were (every product has read them): 32 x 32 units of
                // [4 columns][32 rows], 16 bytes each
                for (int g = half; g < p.BN / 32; g += 2) {
                    uint32_t r[32];
                    if (ok) {
                        tmem_ld32(acc + 32u * g, r);
                        tmem_wait_ld_only();
                        reg_fence32(r);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        st_shared_v4(base + (uint32_t)(4 * g + q) * 4096u + (uint32_t)(i * 512 + lane * 16), ok ? r[4 * i] : 0x7fffffffu,
                                     ok ? r[4 * i + 1] : 0x7fffffffu, ok ? r[4 * i + 2] : 0x7fffffffu, ok ? r[4 * i + 3] : 0x7fffffffu);
                }
            } else if constexpr (GATED) {
                const int share = p.BN / PAIR, hs = share / 2;  // accumulator: per share its value columns, then its gates
                for (int g = half; g < p.BN / 64; g += 2) {
                    const int c = 32 * g, col = n + c;
                    if (col >= p.N || y >= p.M) continue;
                    const uint32_t from = (uint32_t)(c / hs * share + c % hs);
                    float v[32], gt[32];
                    uint32_t w[16];
                    columns(from, bias, col, p.N, v);
                    if (p.has_p) {
                        pack32<DT>(v, w);
                        store(&tmV, w, col);
                    }
                    columns(from + (uint32_t)hs, bias ? bias + p.N : nullptr, col, p.N, gt);
                    if (p.has_p) {
                        pack32<DT>(gt, w);
                        store(&tmG, w, col);
                    }
                    switch (p.act) {
                        case EPI_GELU_ERF: gate32<DT, EPI_GELU_ERF>(v, gt, w); break;
                        case EPI_GELU_TANH: gate32<DT, EPI_GELU_TANH>(v, gt, w); break;
                        case EPI_GELU_SIGMOID: gate32<DT, EPI_GELU_SIGMOID>(v, gt, w); break;
                        case EPI_SILU: gate32<DT, EPI_SILU>(v, gt, w); break;
                        default: gate32<DT, EPI_NONE>(v, gt, w); break;
                    }
                    store(&tmC, w, col);
                }
            } else {
                for (int g = half; g < p.BN / 32; g += 2) {
                    const int col = n + 32 * g;
                    if (col >= p.N || y >= p.M) continue;
                    float v[32];
                    uint32_t w[16];
                    columns(32u * g, bias, col, p.N, v);
                    pack32<DT>(v, w);
                    store(&tmC, w, col);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR == 2) mbar_arrive_cluster_relaxed(mapa_rank(bar_acce + 8u * buf, 0));
                else mbar_arrive_relaxed(bar_acce + 8u * buf);
            }
        }
        if constexpr (!SPLIT) {
            if (lane == 0) bulk_wait0();
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (SPLIT) {
        if (*abort_flag)  // no sums from this CTA: NaN in their place, and so in the whole tile
            for (int i = threadIdx.x; i < 128 * p.BN; i += kMmThreads) reinterpret_cast<uint32_t*>(at)[i] = 0x7fffffffu;
        cluster_sync_all();  // every CTA's sums are there
        if (warp >= 2 && warp < 10) {
            const int ew = warp - 2;
            const uint32_t stg = staging + (uint32_t)ew * 4096u;
            int m, n;
            origin(unit0, m, n);
            for (int u = part + splits * ew; u < p.BN / 8; u += splits * kMmEpi) {  // units of this CTA: every splits-th
                const int q = u & 3, col = n + 32 * (u >> 2), y = m + 32 * q;
                if (col >= p.N || y >= p.M) continue;
                float v[32];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t from = base + (uint32_t)u * 4096u + (uint32_t)(i * 512 + lane * 16);
                    float4 x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < splits) x[j] = ld_cluster4(mapa_rank(from, (uint32_t)j));
#pragma unroll
                    for (int j = 1; j < 8; ++j)
                        if (j < splits) {
                            x[0].x += x[j].x;
                            x[0].y += x[j].y;
                            x[0].z += x[j].z;
                            x[0].w += x[j].w;
                        }
                    v[4 * i] = x[0].x;
                    v[4 * i + 1] = x[0].y;
                    v[4 * i + 2] = x[0].z;
                    v[4 * i + 3] = x[0].w;
                }
                if (p.bias) {
                    float b[32];
                    bias32<DT>(p.bias, col, p.N, b);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] += b[i];
                }
                uint32_t w[16];
                pack32<DT>(v, w);
                stage_and_store_packed(&tmC, stg, lane, w, col, y);
            }
            if (lane == 0) bulk_wait0();
            __syncwarp();
        }
    }
    if (PAIR == 2 || SPLIT) cluster_sync_all();  // neither leaves while another may still signal or read it
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc<PAIR>(tmem, kTmemCols);
    }
}

constexpr int kMmSmem = kSmemBudget;
// what the ring may take: alignment, staging, barriers beside it
constexpr int kMmRing = kMmSmem - 1024 - kMmEpi * 4096 - 256;

int mm_stages(const MatmulShape& s) { return std::min(8, kMmRing / (int)(kMmABytes + s.BN / s.pair * 128)); }

template <int DT, int PAIR, bool GATED, bool SPLIT>
cudaError_t mm_prepare(int device) {
    static SmemOptIn opt_in;
    return opt_in(kt_matmul_kernel<DT, PAIR, GATED, SPLIT>, kMmSmem, device);
}

cudaLaunchConfig_t mm_config(int grid, int cluster, void* stream, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(kMmThreads, 1, 1);
    cfg.dynamicSmemBytes = kMmSmem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cfg;
}

// Clusters of ks CTAs that the device holds at once; 0 if it cannot say.
int mm_clusters(int ks, int device) {
    static std::atomic<int> known[64][9];  // + 1
    int n = known[device & 63][ks].load(std::memory_order_relaxed) - 1;
    if (n >= 0) return n;
    n = 0;
    if (mm_prepare<KT_F16, 1, false, true>(device) == cudaSuccess) {
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t cfg = mm_config(ks, ks, nullptr, attr);
        if (cudaOccupancyMaxActiveClusters(&n, kt_matmul_kernel<KT_F16, 1, false, true>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
    }
    known[device & 63][ks].store(n + 1, std::memory_order_relaxed);
    return n;
}

template <int DT, int PAIR, bool GATED, bool SPLIT>
cudaError_t mm_launch(const CUtensorMap* tm, const MmParams& p, int grid, int cluster, int device, void* stream) {
    cudaError_t e = mm_prepare<DT, PAIR, GATED, SPLIT>(device);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = mm_config(grid, cluster, stream, attr);
    return cudaLaunchKernelEx(&cfg, kt_matmul_kernel<DT, PAIR, GATED, SPLIT>, tm[0], tm[1], tm[2], tm[3], tm[4], p);
}

template <int DT>
cudaError_t mm_dispatch(const CUtensorMap* tm, const MmParams& p, const MatmulShape& s, bool gated, int sms, int device, void* stream) {
    const int tiles = p.tiles_m * p.tiles_n;
    if (s.splits > 1) return mm_launch<DT, 1, false, true>(tm, p, tiles * s.splits, s.splits, device, stream);
    const int grid = std::min(tiles, sms / s.pair) * s.pair;
    if (gated) return s.pair == 2 ? mm_launch<DT, 2, true, false>(tm, p, grid, 2, device, stream) : mm_launch<DT, 1, true, false>(tm, p, grid, 1, device, stream);
    return s.pair == 2 ? mm_launch<DT, 2, false, false>(tm, p, grid, 2, device, stream) : mm_launch<DT, 1, false, false>(tm, p, grid, 1, device, stream);
}

int64_t mm_tiles(const Matmul& a, int bn, int pair) {
    const int64_t cols = a.gated ? bn / 2 : bn;
    return (int64_t)((a.M + 128 * pair - 1) / (128 * pair)) * ((a.N + cols - 1) / cols);
}

}  // namespace

MatmulShape matmul_shape(const Matmul& a, int sms, int device) {
    const int steps = (a.K + kAtomK - 1) / kAtomK;
    struct {
        int pair, bn;
        double step, round;
    } const kinds[] = {{2, 256, 0.30, 4.0}, {2, 128, 0.21, 3.5}, {1, 128, 0.25, 3.0}, {1, 64, 0.20, 3.0}};
    MatmulShape best = {};
    double least = 1e30;
    for (const auto& k : kinds) {
        const int64_t t = mm_tiles(a, k.bn, k.pair), units = sms / k.pair, rounds = (t + units - 1) / units;
        const double time = rounds * (steps * k.step + 0.5) + k.round;
        if (time < least) {
            least = time;
            best = {k.pair, k.bn, 1};
        }
        if (a.gated || k.pair == 2) continue;
        for (int ks = 2; ks <= 8; ks *= 2) {
            if (t * ks > sms || steps < 2 * ks || t > mm_clusters(ks, device)) continue;
            const double split = (steps + ks - 1) / ks * k.step + k.round + 2.5;
            if (split < least) {
                least = split;
                best = {1, k.bn, ks};
            }
        }
    }
    return best;
}

kt_status launch_matmul_as(int dtype, const Matmul& a, const MatmulShape& s, int sms, int device, void* stream, const char** why) {
    MmParams p = {};
    p.M = a.M;
    p.N = a.N;
    p.BN = s.BN;
    const int cols = a.gated ? s.BN / 2 : s.BN;
    p.tiles_m = (a.M + 128 * s.pair - 1) / (128 * s.pair);
    p.tiles_n = (a.N + cols - 1) / cols;
    p.kblocks = (a.K + kAtomK - 1) / kAtomK;
    p.stages = mm_stages(s);
    p.a_mn = a.a_mn;
    p.b_mn = a.b_mn;
    p.act = a.act;
    p.has_p = a.P != nullptr;
    p.idesc = make_idesc(dtype, s.BN, 128 * s.pair, !a.b_mn) | (a.a_mn ? 1u << 15 : 0u);
    p.b_bytes = (uint32_t)(s.BN / s.pair) * 128u;
    p.bias = a.bias;
    p.wait_limit_ns = a.wait_limit_ns;
    p.stall_ns = a.stall_ns;
    CUtensorMap tm[5];
    // a [rows][cols] matrix of pitch ld, in boxes of box_rows x box_cols
    auto encode = [&](CUtensorMap* m, const void* at, int64_t ld, int64_t rows, int64_t columns, int box_rows, int box_cols, int swizzle) {
        const uint64_t dims[2] = {(uint64_t)columns, (uint64_t)rows}, strides[1] = {(uint64_t)ld * 2};
        const uint32_t box[2] = {(uint32_t)box_cols, (uint32_t)box_rows};
        return encode_tmap_nd(m, at, dtype, 2, dims, strides, box, swizzle, why);
    };
    const int b_rows = a.gated ? s.BN / s.pair / 2 : s.BN / s.pair;
    if (!(a.a_mn ? encode(tm, a.A, a.lda, a.K, a.M, 64, 64, 128) : encode(tm, a.A, a.lda, a.M, a.K, 128, 64, 128)) ||
        !(a.b_mn ? encode(tm + 1, a.B, a.ldb, a.K, a.N, 64, 64, 128)
                 : encode(tm + 1, a.B, a.ldb, a.gated ? 2 * (int64_t)a.N : a.N, a.K, b_rows, 64, 128)) ||
        !encode(tm + 2, a.C, a.ldc, a.M, a.N, 32, kStoreCols, 64))
        return KT_ERR_CUDA;
    tm[3] = tm[4] = tm[2];
    if (a.P) {
        uint16_t* P = static_cast<uint16_t*>(a.P);
        if (!encode(tm + 3, P, a.ldp, a.M, a.N, 32, kStoreCols, 64) || !encode(tm + 4, P + a.N, a.ldp, a.M, a.N, 32, kStoreCols, 64))
            return KT_ERR_CUDA;
    }
    const cudaError_t e = dtype == KT_BF16 ? mm_dispatch<KT_BF16>(tm, p, s, a.gated, sms, device, stream)
                                           : mm_dispatch<KT_F16>(tm, p, s, a.gated, sms, device, stream);
    if (e != cudaSuccess) {
        *why = cudaGetErrorString(e);
        return KT_ERR_CUDA;
    }
    return KT_OK;
}

kt_status launch_matmul(int dtype, const Matmul& a, int sms, int device, void* stream, const char** why) {
    return launch_matmul_as(dtype, a, matmul_shape(a, sms, device), sms, device, stream, why);
}

kt_status matmul_status(void* stream, int* word, const char** why) { return error_word(g_matmul_error, stream, word, why); }

}  // namespace kt
