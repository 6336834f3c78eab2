// mxfp4_gemm.cu -- Y[M,N] = X[M,K] * W[N,K]^T with both operands MXFP4, on
// the block-scaled 4-bit tensor cores (tcgen05 kind::mxf4).
//
// Products of two E2M1 numbers and their powers of two are exact in fp32; the
// tensor core adds them in fp32, so the sum's rounding is the only error.
// The weight is the MMA's A operand (its 128 rows are the accumulator's
// lanes), the activations its B operand, so that a warp's lanes hold
// consecutive n of one row of Y and a store is one contiguous run, and a few
// activation rows cost an MMA of few columns.
//   * a producer thread brings the tiles of a 256-k step with bulk copies;
//   * one thread copies the step's scales from shared to tensor memory (each
//     ring slot has its own columns there) and issues four MMAs of K = 64;
//   * four epilogue warps drain the accumulator and store Y.
#include <cstring>

#include "mxfp4_layout.cuh"
#include "mxfp4_tcgen05.cuh"

namespace {

using namespace q4dev;
using q4::kMxCodeBytes;
using q4::kMxTileBytes;

constexpr int kThreads = 192;

struct GemmParams {
    const uint8_t *W, *X;
    void *Y;
    unsigned *err;
    int64_t M, N, kt;
    int64_t tiles_n, tiles_m;
    int bf16;
};

// XR: activation rows a CTA's tile holds (32, 128 or 256)
template <int XR>
struct Cfg {
    static constexpr int kXCodes = XR * 128;
    static constexpr int kXTiles = (XR + 127) / 128;
    static constexpr int kSlot = kMxTileBytes + kXCodes + 1024 * kXTiles;
    static constexpr int kStages = XR == 32 ? 9 : XR == 128 ? 6 : 4;
    static constexpr int kDCols = XR;
    static constexpr int kSfCols = 8 + 8 * kXTiles;   // tensor-memory columns of a slot's scales
    static constexpr int kTmemCols = kDCols + kStages * kSfCols <= 256 ? 256 : 512;
    static_assert(kDCols + kStages * kSfCols <= kTmemCols, "tensor memory");
};

template <int XR>
struct Smem {
    uint8_t slot[Cfg<XR>::kStages][Cfg<XR>::kSlot];
    uint64_t full[Cfg<XR>::kStages], empty[Cfg<XR>::kStages];
    uint64_t d_full, d_empty, mma_done;
    uint32_t tmem_base;
    int abort_flag;
};

__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, int *abort_flag, unsigned *err) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_ns();
    while (!mbar_try_wait_suspend(bar, parity)) {
        if (*reinterpret_cast<volatile int *>(abort_flag)) return false;
        if (global_ns() - t0 > kWaitLimitNs) {
            atomicOr(err, (unsigned)Q4_DEVERR_WAIT_TIMEOUT);
            *reinterpret_cast<volatile int *>(abort_flag) = 1;
            return false;
        }
    }
    return true;
}

template <int XR>
__global__ void __launch_bounds__(kThreads, 1) mx_gemm_kernel(const GemmParams P) {
    using C = Cfg<XR>;
    extern __shared__ uint8_t smem_raw[];
    Smem<XR> &S = *reinterpret_cast<Smem<XR> *>(align_smem<1024>(smem_raw));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t tiles = P.tiles_n * P.tiles_m;
    const int kt = static_cast<int>(P.kt);

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&S.full[s], 1);
            mbar_init(&S.empty[s], 1);
        }
        mbar_init(&S.d_full, 1);
        mbar_init(&S.d_empty, 4);
        mbar_init(&S.mma_done, 1);
        S.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(&S.tmem_base, C::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem_base;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t c = 0;
            bool ok = true;
            for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                const int64_t tn = t % P.tiles_n, m0 = t / P.tiles_n * XR;
                // the tile's activation rows, in whole groups of eight (rows
                // past M lie in the matrix's padding)
                const int rows = static_cast<int>((P.M - m0 < XR ? P.M - m0 : XR) + 7) & ~7;
                const uint8_t *w = P.W + tn * kt * kMxTileBytes;
                const uint8_t *x = P.X + (m0 >> 7) * kt * kMxTileBytes + (m0 & 127) * 128;
                for (int i = 0; i < kt; ++i, ++c) {
                    const int s = c % C::kStages;
                    if (!(ok = wait_or_abort(&S.empty[s], ((c / C::kStages) & 1) ^ 1, &S.abort_flag, P.err))) break;
                    uint8_t *slot = S.slot[s];
                    const int xt = (rows + 127) / 128;
                    mbar_arrive_expect_tx(&S.full[s], kMxTileBytes + rows * 128 + 1024 * xt);
                    bulk_g2s(slot, w + (int64_t)i * kMxTileBytes, kMxTileBytes, &S.full[s]);
                    for (int j = 0; j < xt; ++j) {
                        const uint8_t *xs = x + ((int64_t)j * kt + i) * kMxTileBytes;
                        const int rj = rows - 128 * j < 128 ? rows - 128 * j : 128;
                        bulk_g2s(slot + kMxTileBytes + j * kMxCodeBytes, xs, rj * 128, &S.full[s]);
                        bulk_g2s(slot + kMxTileBytes + C::kXCodes + 1024 * j, xs - (m0 & 127) * 128 + kMxCodeBytes, 1024,
                                 &S.full[s]);
                    }
                }
            }
            if (!ok)   // let the copies already issued land (bounded) before the CTA can exit
                for (uint32_t i = 0; i < C::kStages && i < c; ++i) {
                    const uint32_t q = c - 1 - i;
                    mbar_wait(&S.full[q % C::kStages], (q / C::kStages) & 1, P.err);
                }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            uint32_t c = 0, dc = 0;
            bool ok = true;
            for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++dc) {
                const int64_t m0 = t / P.tiles_n * XR;
                const int rows = static_cast<int>((P.M - m0 < XR ? P.M - m0 : XR) + 7) & ~7;
                if (!(ok = wait_or_abort(&S.d_empty, (dc & 1) ^ 1, &S.abort_flag, P.err))) break;
                tc_fence_after();
                const uint32_t idesc = mxf4_idesc(128, rows, 0);
                for (int i = 0; i < kt; ++i, ++c) {
                    const int s = c % C::kStages;
                    if (!(ok = wait_or_abort(&S.full[s], (c / C::kStages) & 1, &S.abort_flag, P.err))) break;
                    tc_fence_after();
                    const uint32_t base = smem_addr(S.slot[s]);
                    const uint32_t sfa = tmem + C::kDCols + s * C::kSfCols, sfb = sfa + 8;
                    #pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        tc_cp_scales(sfa + 4 * g, scales_desc(base + kMxCodeBytes + 512 * g));
                        #pragma unroll
                        for (int j = 0; j < C::kXTiles; ++j)
                            if (j == 0 || rows > 128)
                                tc_cp_scales(sfb + 4 * C::kXTiles * g + 4 * j,
                                             scales_desc(base + kMxTileBytes + C::kXCodes + 1024 * j + 512 * g));
                    }
                    const uint64_t a = sw128_kmajor_desc(base), b = sw128_kmajor_desc(base + kMxTileBytes);
                    #pragma unroll
                    for (int j = 0; j < 4; ++j)
                        tc_mma_mxf4(tmem, a + 2 * j, b + 2 * j, idesc | ((j & 1) ? mxf4_idesc(0, 0, 2) : 0u),
                                    sfa + 4 * (j >> 1), sfb + 4 * C::kXTiles * (j >> 1), (i | j) != 0);
                    tc_commit(&S.empty[s]);
                }
                if (ok) tc_commit(&S.d_full);
            }
            tc_commit(&S.mma_done);   // every MMA issued so far has completed once this arrives
            wait_or_abort(&S.mma_done, 0, &S.abort_flag, P.err) || mbar_wait(&S.mma_done, 0, P.err);
        }
    } else {
        const int quad = warp & 3;
        uint32_t dc = 0;
        for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x, ++dc) {
            const int64_t m0 = t / P.tiles_n * XR, n = t % P.tiles_n * 128 + 32 * quad + lane;
            const int rows = static_cast<int>(P.M - m0 < XR ? P.M - m0 : XR);
            if (!wait_or_abort(&S.d_full, dc & 1, &S.abort_flag, P.err)) break;
            tc_fence_after();
            #pragma unroll 1
            for (int c = 0; c < rows; c += 32) {
                float v[32];
                tc_ld_32(tmem + (uint32_t(32 * quad) << 16) + c, v);
                if (n < P.N) {
                    #pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (c + j < rows) {
                            const int64_t at = (m0 + c + j) * P.N + n;
                            if (P.bf16) static_cast<__nv_bfloat16 *>(P.Y)[at] = __float2bfloat16_rn(v[j]);
                            else __stcs(static_cast<float *>(P.Y) + at, v[j]);
                        }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.d_empty);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

// ---------------------------------------------------------------- few rows

// The split kernel: a cluster of `split` CTAs takes one tile of 128 weight
// rows x up to 128 activation rows, each CTA a run of its 256-k steps.  The
// ranks' sums meet in shared memory: rank q adds columns [q*cpr, (q+1)*cpr)
// over all ranks, in rank order, so the result does not depend on timing.
struct SplitParams {
    const uint8_t *W, *X;
    void *Y;
    unsigned *err;
    int64_t M, N;
    int kt, tiles_n;
    int split;        // CTAs of a cluster
    int slots;        // ring slots
    int xcap;         // activation rows a slot has room for (a multiple of 8)
    int bf16;
};

constexpr int kMaxSlots = 12;
constexpr int kSplitTmemCols = 256;

struct SplitSmem {
    uint64_t full[kMaxSlots], empty[kMaxSlots];
    uint64_t d_full, mma_done, red_full;
    uint32_t tmem_base;
    int abort_flag;
};

__host__ __device__ constexpr int split_x_bytes(int xcap) { return (xcap * 128 + 1023) & ~1023; }
__host__ __device__ constexpr int split_slot_bytes(int xcap) { return kMxTileBytes + split_x_bytes(xcap) + 1024; }
// the ranks' sums of one rank's columns, [source rank][column][weight row]
__host__ __device__ constexpr int split_red_bytes(int xcap, int split) {
    return split > 1 ? split * ((xcap + split - 1) / split) * 512 : 0;
}
__host__ __device__ constexpr int split_d_cols(int xcap) { return (xcap + 15) & ~15; }

__device__ __forceinline__ uint32_t remote_addr(uint32_t local, uint32_t rank) {
    uint32_t ra;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(local), "r"(rank));
    return ra;
}

__device__ __forceinline__ bool wait_cluster_or_abort(uint64_t *bar, uint32_t parity, int *abort_flag, unsigned *err) {
    const unsigned long long t0 = global_ns();
    for (;;) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
            " selp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok)
            : "r"(smem_addr(bar)), "r"(parity), "r"(kSuspendHintNs)
            : "memory");
        if (ok) return true;
        if (*reinterpret_cast<volatile int *>(abort_flag)) return false;
        if (global_ns() - t0 > kWaitLimitNs) {
            atomicOr(err, (unsigned)Q4_DEVERR_WAIT_TIMEOUT);
            *reinterpret_cast<volatile int *>(abort_flag) = 1;
            return false;
        }
    }
}

__device__ __forceinline__ void store_y(const SplitParams &P, int64_t m, int64_t n, float v) {
    const int64_t at = m * P.N + n;
    if (P.bf16) static_cast<__nv_bfloat16 *>(P.Y)[at] = __float2bfloat16_rn(v);
    else static_cast<float *>(P.Y)[at] = v;
}

__global__ void __launch_bounds__(kThreads, 2) mx_split_kernel(const __grid_constant__ SplitParams P) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ SplitSmem S;
    uint8_t *const ring = align_smem<1024>(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slot_bytes = split_slot_bytes(P.xcap), x_bytes = split_x_bytes(P.xcap);
    float *const red = reinterpret_cast<float *>(ring + P.slots * slot_bytes);
    const int rank = static_cast<int>(blockIdx.x) % P.split;      // clusters are consecutive blocks
    const int tile = static_cast<int>(blockIdx.x) / P.split;
    const int tn = tile % P.tiles_n;
    const int64_t m0 = static_cast<int64_t>(tile / P.tiles_n) * 128;
    const int live = static_cast<int>(P.M - m0 < 128 ? P.M - m0 : 128);
    const int rows = (live + 7) & ~7;
    const int k0 = static_cast<int>(static_cast<int64_t>(P.kt) * rank / P.split);
    const int k1 = static_cast<int>(static_cast<int64_t>(P.kt) * (rank + 1) / P.split);

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int s = 0; s < P.slots; ++s) {
            mbar_init(&S.full[s], 1);
            mbar_init(&S.empty[s], 1);
        }
        mbar_init(&S.d_full, 1);
        mbar_init(&S.mma_done, 1);
        mbar_init(&S.red_full, 4 * P.split);
        S.abort_flag = 0;
        fence_mbar_init();
        // the first weight tiles on their way to L2 while the kernel before
        // this one ends
        const uint8_t *w = P.W + (static_cast<int64_t>(tn) * P.kt + k0) * kMxTileBytes;
        for (int i = 0; i < P.slots && k0 + i < k1; ++i) bulk_prefetch_l2(w + static_cast<int64_t>(i) * kMxTileBytes, kMxTileBytes);
    }
    if (warp == 1) tmem_alloc(&S.tmem_base, kSplitTmemCols);
    tc_fence_before();
    __syncthreads();
    if (P.split > 1)   // every CTA's barrier exists before another CTA arrives on it
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    tc_fence_after();
    const uint32_t tmem = S.tmem_base;

    if (warp == 0) {
        if (lane == 0) {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            const uint8_t *w = P.W + (static_cast<int64_t>(tn) * P.kt + k0) * kMxTileBytes;
            const uint8_t *x = P.X + ((m0 >> 7) * P.kt + k0) * kMxTileBytes;
            bool ok = true;
            int c = 0;
            for (; c < k1 - k0; ++c, w += kMxTileBytes, x += kMxTileBytes) {
                const int s = c % P.slots;
                if (!(ok = wait_or_abort(&S.empty[s], ((c / P.slots) & 1) ^ 1, &S.abort_flag, P.err))) break;
                uint8_t *slot = ring + s * slot_bytes;
                mbar_arrive_expect_tx(&S.full[s], kMxTileBytes + rows * 128 + 1024);
                bulk_g2s(slot, w, kMxTileBytes, &S.full[s]);
                bulk_g2s(slot + kMxTileBytes, x, rows * 128, &S.full[s]);
                bulk_g2s(slot + kMxTileBytes + x_bytes, x + kMxCodeBytes, 1024, &S.full[s]);
            }
            if (!ok)   // let the copies already issued land (bounded) before the CTA can exit
                for (int i = 0; i < P.slots && i < c; ++i)
                    mbar_wait(&S.full[(c - 1 - i) % P.slots], ((c - 1 - i) / P.slots) & 1, P.err);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            bool ok = true;
            const uint32_t idesc = mxf4_idesc(128, rows, 0);
            const uint32_t sf0 = tmem + split_d_cols(P.xcap);
            for (int c = 0; c < k1 - k0; ++c) {
                const int s = c % P.slots;
                if (!(ok = wait_or_abort(&S.full[s], (c / P.slots) & 1, &S.abort_flag, P.err))) break;
                tc_fence_after();
                const uint32_t base = smem_addr(ring + s * slot_bytes);
                const uint32_t sfa = sf0 + 16 * s, sfb = sfa + 8;
                #pragma unroll
                for (int g = 0; g < 2; ++g) {
                    tc_cp_scales(sfa + 4 * g, scales_desc(base + kMxCodeBytes + 512 * g));
                    tc_cp_scales(sfb + 4 * g, scales_desc(base + kMxTileBytes + x_bytes + 512 * g));
                }
                const uint64_t a = sw128_kmajor_desc(base), b = sw128_kmajor_desc(base + kMxTileBytes);
                #pragma unroll
                for (int j = 0; j < 4; ++j)
                    tc_mma_mxf4(tmem, a + 2 * j, b + 2 * j, idesc | ((j & 1) ? mxf4_idesc(0, 0, 2) : 0u),
                                sfa + 4 * (j >> 1), sfb + 4 * (j >> 1), (c | j) != 0);
                tc_commit(&S.empty[s]);
            }
            if (ok) tc_commit(&S.d_full);
            tc_commit(&S.mma_done);   // every MMA issued so far has completed once this arrives
            wait_or_abort(&S.mma_done, 0, &S.abort_flag, P.err) || mbar_wait(&S.mma_done, 0, P.err);
        }
    } else {
        const int quad = warp & 3, row = 32 * quad + lane;
        const int64_t n = static_cast<int64_t>(tn) * 128 + row;
        const uint32_t d = tmem + (uint32_t(32 * quad) << 16);
        if (wait_or_abort(&S.d_full, 0, &S.abort_flag, P.err)) {
            tc_fence_after();
            if (P.split == 1) {
                #pragma unroll 1
                for (int c = 0; c < live; c += 8) {
                    float v[8];
                    tc_ld_cols<8>(d + c, v);
                    tc_wait_ld();
                    if (n < P.N) {
                        #pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (c + j < live) store_y(P, m0 + c + j, n, v[j]);
                    }
                }
            } else {
                const int cpr = (P.xcap + P.split - 1) / P.split;   // columns a rank adds
                const uint32_t mine = smem_addr(red + rank * cpr * 128 + row);
                int dest = 0, at = 0;
                #pragma unroll 1
                for (int c = 0; c < live; c += 8) {
                    float v[8];
                    tc_ld_cols<8>(d + c, v);
                    tc_wait_ld();
                    #pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if (c + j < live)
                            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote_addr(mine + at * 512, dest)), "f"(v[j])
                                         : "memory");
                        if (++at == cpr) { at = 0; ++dest; }
                    }
                }
                asm volatile("fence.acq_rel.cluster;" ::: "memory");
                __syncwarp();
                if (lane < P.split)
                    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                                     remote_addr(smem_addr(&S.red_full), lane))
                                 : "memory");
                if (rank * cpr < live && wait_cluster_or_abort(&S.red_full, 0, &S.abort_flag, P.err) && n < P.N) {
                    #pragma unroll 1
                    for (int c = rank * cpr; c < live && c < (rank + 1) * cpr; ++c) {
                        const float *p = red + (c - rank * cpr) * 128 + row;
                        float v = 0.f;
                        for (int q = 0; q < P.split; ++q) v += p[q * cpr * 128];
                        store_y(P, m0 + c, n, v);
                    }
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kSplitTmemCols);
    }
    if (P.split > 1)   // no CTA leaves while another of the cluster may still reach its shared memory
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

constexpr int kSplitSmemMax = 220 * 1024, kSplitSmemHalf = 111 * 1024;

cudaError_t launch_split(const uint8_t *W, const uint8_t *X, void *Y, bool bf16, int64_t M, int64_t N, int kt,
                         const q4::DeviceInfo &dev, cudaStream_t s) {
    static q4::DeviceOnce configured;
    cudaError_t e = configured.run(dev.device, [] {
        return cudaFuncSetAttribute(mx_split_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSplitSmemMax);
    });
    if (e != cudaSuccess) return e;
    SplitParams p{W, X, Y, dev.err, M, N, kt, static_cast<int>(q4::mx_row_tiles(N)), 1, 1, 0, bf16};
    p.xcap = static_cast<int>((M < 128 ? M : 128) + 7) & ~7;
    const int64_t tiles = p.tiles_n * q4::mx_row_tiles(M);
    // SPLIT RULE
    int split = 1;
    while (split < 8 && split < kt && tiles * (split + 1) <= 2 * dev.sm_count) ++split;
    p.split = split;
    const int budget = tiles * split <= dev.sm_count ? kSplitSmemMax : kSplitSmemHalf;
    const int need = (kt + split - 1) / split;
    int slots = (budget - 1024 - split_red_bytes(p.xcap, split)) / split_slot_bytes(p.xcap);
    if (slots > (kSplitTmemCols - split_d_cols(p.xcap)) / 16) slots = (kSplitTmemCols - split_d_cols(p.xcap)) / 16;
    if (slots > kMaxSlots) slots = kMaxSlots;
    if (slots > need) slots = need;
    p.slots = slots < 1 ? 1 : slots;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = 1024 + p.slots * split_slot_bytes(p.xcap) + split_red_bytes(p.xcap, split);
    cfg.stream = s;
    cfg.attrs = attr;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, mx_split_kernel, p);
}

template <int XR>
cudaError_t launch(GemmParams p, const q4::DeviceInfo &dev, cudaStream_t s) {
    constexpr size_t bytes = sizeof(Smem<XR>) + 1024;
    static_assert(bytes <= 232448, "shared memory");
    static q4::DeviceOnce configured;
    const cudaError_t e = configured.run(dev.device, [] {
        return cudaFuncSetAttribute(mx_gemm_kernel<XR>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    });
    if (e != cudaSuccess) return e;
    p.tiles_m = (p.M + XR - 1) / XR;
    const int64_t tiles = p.tiles_n * p.tiles_m;
    mx_gemm_kernel<XR><<<static_cast<int>(tiles < dev.sm_count ? tiles : dev.sm_count), kThreads, bytes, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

namespace q4 {

cudaError_t launch_mx_gemm(const uint8_t *W, const uint8_t *X, void *Y, int y_type, int64_t M, int64_t N, int64_t K,
                           const DeviceInfo &dev, cudaStream_t s) {
    GemmParams p{W, X, Y, dev.err, M, N, mx_k_tiles(K), mx_row_tiles(N), 0, y_type == Q4_TYPE_BF16};
    if (M <= 128) return launch_split(W, X, Y, y_type == Q4_TYPE_BF16, M, N, static_cast<int>(p.kt), dev, s);
    return launch<256>(p, dev, s);
}

}  // namespace q4
