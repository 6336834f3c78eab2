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
    return M <= 32 ? launch<32>(p, dev, s) : M <= 128 ? launch<128>(p, dev, s) : launch<256>(p, dev, s);
}

}  // namespace q4
