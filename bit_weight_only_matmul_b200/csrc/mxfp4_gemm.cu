// mxfp4_gemm.cu -- Y[M,N] = X[M,K] * W[N,K]^T with both operands MXFP4, on
// the block-scaled 4-bit tensor cores (tcgen05 kind::mxf4).
//
// Products of two E2M1 numbers and their powers of two are exact in fp32; the
// tensor core adds them in fp32, so the sum's rounding is the only error.
// The weight is the MMA's A operand (its rows are the accumulator's lanes),
// the activations its B operand, so that a warp's lanes hold consecutive n of
// one row of Y and a store is one contiguous run, and a few activation rows
// cost an MMA of few columns.  Both kernels have
//   * producer warps that bring the tiles of a 256-k step with bulk copies. A
//     warp issues one copy in about 100 cycles plus one for each 77 bytes (one
//     warp 52 bytes a cycle in copies of 16 KB, two 68), so each of the step's
//     larger copies has a warp of its own;
//   * a warp that copies the step's scales from shared to tensor memory (each
//     ring slot has its own columns there) and issues four MMAs of K = 64.
//     The whole warp walks the loop and one elected lane issues, so that the
//     operands of the instructions stay in uniform registers: a step takes
//     214 cycles at 8 activation rows and 516 at 256 (the tensor cores' full
//     rate), where a loop under `if (lane == 0)` took 733 and 738;
//   * epilogue warps that drain the accumulator and store Y.
// mx_split_kernel (few rows) is paced by the weight stream from HBM: 1 x 131072 x
// 5120 54.7 us, 6.5 TB/s; 32 x 16384 x 5120 9.7 us, of which 3 are start and end.
// mx_pair_kernel (many) is paced by the tensor cores under the power cap: 4096 x
// 16384 x 5120 with bf16 Y 120 to 126 us (5.5 PFLOP/s) in a burst of 24, 140 to
// 147 (4.8) in 4000 one after the other, and the same between its quantizes.
#include <cstring>
#include <type_traits>

#include "mxfp4_layout.cuh"
#include "mxfp4_tcgen05.cuh"
#include "q4_0_tmap.cuh"

namespace {

using namespace q4dev;
using q4::kMxCodeBytes;
using q4::kMxTileBytes;

// One try at phase `parity`: the thread may be suspended while it is
// incomplete.  CLUSTER: the phase is completed by another CTA of the cluster.
template <bool CLUSTER>
__device__ __forceinline__ bool try_phase(uint64_t *bar, uint32_t parity) {
    if (!CLUSTER) return mbar_try_wait_suspend(bar, parity);
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(kSuspendHintNs)
        : "memory");
    return ok != 0;
}

// Bounded wait that also gives up when another role has aborted.  The global
// timer is read, and the error word at hand, only once a wait has failed often
// enough to be out of the ordinary.
template <bool CLUSTER>
__device__ __noinline__ bool long_wait(uint64_t *bar, uint32_t parity, int *abort_flag, unsigned *err) {
    const unsigned long long t0 = global_ns();
    while (!try_phase<CLUSTER>(bar, parity)) {
        if (*reinterpret_cast<volatile int *>(abort_flag)) return false;
        if (global_ns() - t0 > kWaitLimitNs) {
            atomicOr(err, (unsigned)Q4_DEVERR_WAIT_TIMEOUT);
            *reinterpret_cast<volatile int *>(abort_flag) = 1;
            return false;
        }
    }
    return true;
}
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, int *abort_flag, unsigned *err) {
    if (!CLUSTER && mbar_try_wait(bar, parity)) return true;
    #pragma unroll 1
    for (int i = 0; i < 32; ++i)
        if (try_phase<CLUSTER>(bar, parity)) return true;
    return long_wait<CLUSTER>(bar, parity, abort_flag, err);
}

// The same answer in all lanes of a warp that waits as a whole.
__device__ __forceinline__ bool all_lanes(bool ok) { return __all_sync(0xffffffffu, ok); }

// After an abort: the copies a producer has issued land (bounded) before its
// CTA can exit.  `count` slots of a ring of `slots` were filled.
__device__ __forceinline__ void drain(uint64_t *full, int slots, int count, unsigned *err) {
    for (int i = 1; i <= slots && i <= count; ++i)
        mbar_wait(&full[(count - i) % slots], ((count - i) / slots) & 1, err, 20000000ull);
}

// One lane of a converged warp, in a form the compiler knows to be a single one.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}

// ---------------------------------------------------------------- few rows

// The split kernel: a cluster of `split` CTAs takes 128 weight rows and all
// activation rows (up to 128), each CTA a run of the 256-k steps.  The ranks'
// sums meet in shared memory: rank q adds columns [q*cpr, (q+1)*cpr) over all
// ranks, in rank order, so the result does not depend on timing.  They travel
// in groups of four columns, 16 bytes a lane (128 x 1024 x 5120 8.4 us one by one,
// 7.5 in groups), one or two columns one by one (1 x 5120 x 8192 7.2 and 7.3).
struct SplitParams {
    const uint8_t *W, *X;
    void *Y;
    unsigned *err;
    int64_t N;
    int M, kt;
    int split;        // CTAs of a cluster
    int slots;        // ring slots
    int xcap;         // M in whole groups of eight rows (the rest lies in X's padding)
    int bf16;
};

constexpr int kThreads = 224;
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
// columns a rank adds, in whole groups of four
__host__ __device__ constexpr int split_cpr(int xcap, int split) { return ((xcap + split - 1) / split + 3) & ~3; }
// the ranks' sums of one rank's columns, [source rank][group][weight row][column of the group]
__host__ __device__ constexpr int split_red_bytes(int xcap, int split) { return split > 1 ? split * split_cpr(xcap, split) * 512 : 0; }
__host__ __device__ constexpr int split_d_cols(int xcap) { return (xcap + 15) & ~15; }

__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote_addr(uint32_t local, uint32_t rank) {
    uint32_t ra;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(local), "r"(rank));
    return ra;
}

__device__ __forceinline__ void put(float *y, float v) { *y = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *y, float v) { *y = __float2bfloat16_rn(v); }

// A warp's 32 lanes of the accumulator to column n of Y's rows.
template <class T>
__device__ __forceinline__ void store_columns(const SplitParams &P, uint32_t d, int64_t n) {
    T *y = static_cast<T *>(P.Y) + n;
    #pragma unroll 1
    for (int c = 0; c < P.M; c += 8) {
        float v[8];
        tc_ld_cols<8>(d + c, v);
        tc_wait_ld();
        #pragma unroll
        for (int j = 0; j < 8; ++j, y += P.N)
            if (n < P.N && c + j < P.M) put(y, v[j]);
    }
}

// A warp's 32 lanes of the accumulator to the ranks that add their columns, in
// groups of G; `mine` is the lane's row in this rank's first group.
template <int G>
__device__ __forceinline__ void send_columns(const SplitParams &P, SplitSmem &S, int cpr, uint32_t d, uint32_t mine) {
    int dest = 0, at = 0;
    #pragma unroll 1
    for (int c = 0; c < P.M; c += 8) {
        float v[8];
        tc_ld_cols<8>(d + c, v);
        tc_wait_ld();
        #pragma unroll
        for (int j = 0; j < 8; j += G) {
            if (c + j < P.M) {
                if (Q4_DEBUG_BAD(dest < P.split && at + G <= cpr, P.err, &S.abort_flag)) return;
                const uint32_t to = remote_addr(mine + at * 512, dest);
                if constexpr (G == 4)
                    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(v[j]), "f"(v[j + 1]),
                                 "f"(v[j + 2]), "f"(v[j + 3])
                                 : "memory");
                else
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(v[j]) : "memory");
            }
            if ((at += G) == cpr) { at = 0; ++dest; }
        }
    }
}

// A rank's columns [first, last): the ranks' sums of one weight row in rank
// order.  `red` is that row's place in the first group of the first rank.
template <int G, class T>
__device__ __forceinline__ void store_sums(const SplitParams &P, const float *red, int first, int last, int cpr, int64_t n) {
    T *y = static_cast<T *>(P.Y) + first * P.N + n;
    for (int c = first; c < last; c += G, red += G * 128) {
        float sum[G] = {};
        const float *p = red;
        for (int q = 0; q < P.split; ++q, p += cpr * 128) {
            if constexpr (G == 4) {
                const float4 v = *reinterpret_cast<const float4 *>(p);
                sum[0] += v.x; sum[1] += v.y; sum[2] += v.z; sum[3] += v.w;
            } else {
                sum[0] += *p;
            }
        }
        #pragma unroll
        for (int j = 0; j < G; ++j, y += P.N)
            if (c + j < last) put(y, sum[j]);
    }
}

// A warp's part in the meeting of the sums.
template <int G>
__device__ __forceinline__ void meet(const SplitParams &P, SplitSmem &S, float *red, int rank, int row, uint32_t d, int64_t n) {
    const int cpr = split_cpr(P.xcap, P.split);
    send_columns<G>(P, S, cpr, d, smem_addr(red + rank * cpr * 128 + G * row));
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
    __syncwarp();
    const int lane = threadIdx.x & 31;
    if (lane < P.split)
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                         remote_addr(smem_addr(&S.red_full), lane))
                     : "memory");
    if (rank * cpr < P.M && wait_or_abort<true>(&S.red_full, 0, &S.abort_flag, P.err) && n < P.N) {
        const int first = rank * cpr, last = min(first + cpr, P.M);
        if (P.bf16) store_sums<G, __nv_bfloat16>(P, red + G * row, first, last, cpr, n);
        else store_sums<G, float>(P, red + G * row, first, last, cpr, n);
    }
}

__global__ void __launch_bounds__(kThreads, 2) mx_split_kernel(const __grid_constant__ SplitParams P) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ SplitSmem S;
    uint8_t *const ring = align_smem<1024>(smem_raw);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int slot_bytes = split_slot_bytes(P.xcap), x_bytes = split_x_bytes(P.xcap);
    float *const red = reinterpret_cast<float *>(ring + P.slots * slot_bytes);
    const int rank = static_cast<int>(blockIdx.x) % P.split;      // clusters are consecutive blocks
    const int tn = static_cast<int>(blockIdx.x) / P.split;
    const int rows = P.xcap;
    const int k0 = static_cast<int>(static_cast<int64_t>(P.kt) * rank / P.split);
    const int k1 = static_cast<int>(static_cast<int64_t>(P.kt) * (rank + 1) / P.split);

    if (threadIdx.x == 0) {
        for (int s = 0; s < P.slots; ++s) {
            mbar_init(&S.full[s], 2);
            mbar_init(&S.empty[s], 1);
        }
        mbar_init(&S.d_full, 1);
        mbar_init(&S.mma_done, 1);
        mbar_init(&S.red_full, 4 * P.split);
        S.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp >= 2 && lane == 0) {
        // the first weight tiles on their way to L2 while the kernel before
        // this one ends: as many as the ring takes where K is short or split
        // (behind a norm, 2 x 5120 x 4096 8.6 us without, 8.1 with; behind a
        // quantize, 8 x 8192 x 2048 6.1 and 5.6).  A whole K of more steps soon
        // keeps HBM busy, and copies that wait for a prefetch cost more than
        // others: two tiles (behind a quantize, 32 x 16384 x 5120 11.5 us without,
        // 11.3 with two tiles, 12.5 with nine)
        const int ahead = P.split == 1 && P.kt > P.slots ? min(2, P.slots) : P.slots;
        const uint8_t *w = P.W + (static_cast<int64_t>(tn) * P.kt + k0) * kMxTileBytes;
        for (int i = warp - 2; i < ahead && k0 + i < k1; i += 5) bulk_prefetch_l2(w + static_cast<int64_t>(i) * kMxTileBytes, kMxTileBytes);
    }
    if (warp == 1) tmem_alloc(&S.tmem_base, kSplitTmemCols);
    tc_fence_before();
    __syncthreads();
    if (P.split > 1) cluster_sync_all();   // every CTA's barrier exists before another CTA arrives on it
    tc_fence_after();
    begin_dependent();   // all warps: their waits are bounded, the kernel before is not
    const uint32_t tmem = S.tmem_base;

    if (warp == 0) {
        // the weight tiles
        if (lane == 0) {
            const uint8_t *w = P.W + (static_cast<int64_t>(tn) * P.kt + k0) * kMxTileBytes;
            int c = 0;
            for (; c < k1 - k0; ++c, w += kMxTileBytes) {
                const int s = c % P.slots;
                if (!wait_or_abort(&S.empty[s], ((c / P.slots) & 1) ^ 1, &S.abort_flag, P.err)) break;
                if (Q4_DEBUG_BAD(s < kMaxSlots && tn < (P.N + 127) / 128 && k0 + c < P.kt, P.err, &S.abort_flag)) break;
                mbar_arrive_expect_tx(&S.full[s], kMxTileBytes);
                bulk_g2s(ring + s * slot_bytes, w, kMxTileBytes, &S.full[s]);
            }
            if (c < k1 - k0) drain(S.full, P.slots, c, P.err);
        }
    } else if (warp == 6) {
        // the activation rows and their scales
        if (lane == 0) {
            const uint8_t *x = P.X + static_cast<int64_t>(k0) * kMxTileBytes;
            int c = 0;
            for (; c < k1 - k0; ++c, x += kMxTileBytes) {
                const int s = c % P.slots;
                if (!wait_or_abort(&S.empty[s], ((c / P.slots) & 1) ^ 1, &S.abort_flag, P.err)) break;
                if (Q4_DEBUG_BAD(s < kMaxSlots && rows <= 128 && k0 + c < P.kt, P.err, &S.abort_flag)) break;
                uint8_t *slot = ring + s * slot_bytes + kMxTileBytes;
                mbar_arrive_expect_tx(&S.full[s], rows * 128 + 1024);
                bulk_g2s(slot, x, rows * 128, &S.full[s]);
                bulk_g2s(slot + x_bytes, x + kMxCodeBytes, 1024, &S.full[s]);
            }
            if (c < k1 - k0) drain(S.full, P.slots, c, P.err);
        }
    } else if (warp == 1) {
        const uint32_t idesc = mxf4_idesc(128, rows, 0);
        const uint32_t sf0 = tmem + split_d_cols(P.xcap);
        int s = 0;
        uint32_t parity = 0;
        for (int c = 0; c < k1 - k0; ++c) {
            if (!all_lanes(wait_or_abort(&S.full[s], parity, &S.abort_flag, P.err))) break;
            tc_fence_after();
            const uint32_t base = smem_addr(ring) + s * slot_bytes;
            const uint32_t sfa = sf0 + 16 * s, sfb = sfa + 8;
            if (Q4_DEBUG_BAD(split_d_cols(P.xcap) + 16 * s + 16 <= kSplitTmemCols, P.err, &S.abort_flag)) break;
            const uint64_t a = sw128_kmajor_desc(base), b = sw128_kmajor_desc(base + kMxTileBytes);
            const uint64_t da = scales_desc(base + kMxCodeBytes), db = scales_desc(base + kMxTileBytes + x_bytes);
            __syncwarp();
            if (elect_one()) {
                #pragma unroll
                for (int g = 0; g < 2; ++g) {   // 512 bytes on: 32 in the descriptor's units
                    tc_cp_scales(sfa + 4 * g, da + 32 * g);
                    tc_cp_scales(sfb + 4 * g, db + 32 * g);
                }
                #pragma unroll
                for (int j = 0; j < 4; ++j)
                    tc_mma_mxf4(tmem, a + 2 * j, b + 2 * j, idesc | ((j & 1) ? mxf4_idesc(0, 0, 2) : 0u),
                                sfa + 4 * (j >> 1), sfb + 4 * (j >> 1), (c | j) != 0);
                tc_commit(&S.empty[s]);
                if (c == k1 - k0 - 1) tc_commit(&S.d_full);
            }
            __syncwarp();
            if (++s == P.slots) { s = 0; parity ^= 1; }
        }
        // every MMA issued so far has completed once this commit arrives
        if (elect_one()) tc_commit(&S.mma_done);
        __syncwarp();
        wait_or_abort(&S.mma_done, 0, &S.abort_flag, P.err) || mbar_wait(&S.mma_done, 0, P.err);
    }
    const int quad = warp & 3, row = 32 * quad + lane;
    const int64_t n = static_cast<int64_t>(tn) * 128 + row;
    const uint32_t d = tmem + (uint32_t(32 * quad) << 16);
    if (warp >= 2 && warp < 6 && all_lanes(wait_or_abort(&S.d_full, 0, &S.abort_flag, P.err))) {
        tc_fence_after();
        if (P.split == 1) {
            if (P.bf16) store_columns<__nv_bfloat16>(P, d, n);
            else store_columns<float>(P, d, n);
        } else if (P.M <= 2) {
            meet<1>(P, S, red, rank, row, d, n);
        } else {
            meet<4>(P, S, red, rank, row, d, n);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kSplitTmemCols);
    }
    if (P.split > 1) cluster_sync_all();   // no CTA leaves while another of the cluster may still reach its shared memory
}

// Shared memory of a CTA: alone on an SM, one of two, and the least it asks
// for.  The least keeps a third CTA of this kernel, and any CTA of the other
// tensor-memory kernels of this library (180 KB and more), off an SM that
// holds two: their 2 x 256 columns are all there is, and a CTA that had to
// wait for columns while the rest of its cluster holds some could wait for
// another cluster that waits for it.
constexpr int kSplitSmemMax = 220 * 1024, kSplitSmemHalf = 111 * 1024, kSplitSmemMin = 80 * 1024;

// Clusters of `parts` CTAs with an SM each that run at one time: a cluster lies
// within a group of SMs, whose number need not be a multiple of it (128 x 2048 x
// 5120 in 16 clusters of 8, two waves: 14.8 us, in clusters of 4 7.9).
int clusters_at_once(int parts, const q4::DeviceInfo &dev) {
    static q4::DeviceValue resident[9];
    return resident[parts].get(dev.device, [&] {
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = parts;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(dev.sm_count / parts * parts);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSplitSmemMax;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, mx_split_kernel, &cfg) != cudaSuccess) n = 0;
        (void)cudaGetLastError();
        return n > 0 ? n : 1;
    });
}

cudaError_t launch_split(const uint8_t *W, const uint8_t *X, void *Y, bool bf16, int64_t M, int64_t N, int64_t kt64,
                         const q4::DeviceInfo &dev, cudaStream_t s) {
    static q4::DeviceOnce configured;
    cudaError_t e = configured.run(dev.device, [] {
        return cudaFuncSetAttribute(mx_split_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSplitSmemMax);
    });
    if (e != cudaSuccess) return e;
    const int kt = static_cast<int>(kt64), xcap = static_cast<int>(M + 7) & ~7;
    const int64_t tiles = q4::mx_row_tiles(N);
    // K is split into the number of parts that a model of the time favours, of
    // those that leave each CTA an SM of its own; for more than 32 rows, whose
    // CTAs take all of an SM's memory, of those whose clusters run all at once
    // (up to 32 rows two CTAs fit an SM, and a cluster finds room beside
    // another).  The model
    // (ns) is a fit to 150 shapes, each with every number of parts: a step of
    // a CTA costs 260 and two thirds of a row, the meeting of the sums 800 and
    // more with the rows and the CTAs; on 150 others its choice is 0.9 % slower
    // than the best on average, 11 % at worst.  Measured, us, whole and split: 1 x 5120 x 8192 11.0
    // and 7.2 (3 parts), 1 x 256 x 5120 7.1 and 3.6 (8), 16 x 4096 x 4096 6.8 and
    // 5.3 (4), 64 x 1024 x 5120 8.2 and 5.6 (8); whole by the rule: 16 x 5120 x 2048
    // 4.2 and 4.9 (3), 128 x 5120 x 5120 9.5 and 10.6 (3).
    int split = 1;
    int64_t least = 0;
    for (int parts = 1; parts <= 8 && parts <= kt && (parts == 1 || tiles * parts <= dev.sm_count); ++parts) {
        // of 61 shapes 5 or 7 parts were the best for 2, by 1.1 % at most, and 7
        // parts of more than 32 rows twice as slow where 4 or 6 still ran at once
        if (parts == 5 || parts == 7) continue;
        if (parts > 1 && M > 32 && tiles > clusters_at_once(parts, dev)) continue;
        int64_t cost = (260 + 2 * M / 3) * ((kt + parts - 1) / parts);
        if (parts > 1) cost += 800 + 20 * M + tiles * parts * (40 + M) / 10;
        if (parts == 1 || cost < least) {
            split = parts;
            least = cost;
        }
    }
    // a CTA that has its SM to itself takes the memory of two, but where a few
    // rows' split ones do with less and leave room for the next launch's CTAs
    const int budget = tiles <= dev.sm_count && (split == 1 || M > 32) ? kSplitSmemMax : kSplitSmemHalf;
    const int need = (kt + split - 1) / split, red = split_red_bytes(xcap, split);
    int slots = (budget - 1024 - red) / split_slot_bytes(xcap);
    if (slots > (kSplitTmemCols - split_d_cols(xcap)) / 16) slots = (kSplitTmemCols - split_d_cols(xcap)) / 16;
    if (slots > kMaxSlots) slots = kMaxSlots;
    if (slots > need) slots = need;
    const SplitParams p{W, X, Y, dev.err, N, static_cast<int>(M), kt, split, slots, xcap, bf16};
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = 1024 + slots * split_slot_bytes(xcap) + red;
    if (cfg.dynamicSmemBytes < kSplitSmemMin) cfg.dynamicSmemBytes = kSplitSmemMin;
    cfg.stream = s;
    cfg.attrs = attr;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, mx_split_kernel, p);
}

// ---------------------------------------------------------------- many rows

// The pair kernel: two CTAs of a cluster work one tile of 256 weight rows x
// 256 activation rows as one MMA (cta_group::2): each holds 128 weight rows,
// 128 activation rows and the accumulator of its weight rows for all 256
// activation rows, so that a step costs a CTA 35 KB of loads instead of the
// 52 KB of a 128 x 256 tile of its own.  Persistent, one CTA an SM.
//   * each CTA's producers fill its own ring, and the copies of both CTAs
//     complete on the first one's barrier (which only copies through a tensor
//     map can: the matrices are mapped as rows of 1 KB).  Passing the second
//     CTA's filled slots on by remote arrivals instead held a step to 0.6 us;
//   * warp 1 of the first CTA issues for both and releases slots and
//     accumulators in both with multicast commits;
//   * eight epilogue warps take the accumulator into registers at once, so
//     that the next tile's MMAs wait for that only, and store from there.
struct alignas(64) PairParams {
    CUtensorMap map_w, map_x, map_xs;   // boxes: a tile, a tile's codes, a tile's scales
    void *Y;
    unsigned *err;
    int64_t M, N;
    int kt, wt, xt;           // 256-k steps, 128-row tiles of W and of X
    int tiles_n, tiles_m, tiles;   // tiles of 256 x XN: along N, along M, in all
};

constexpr int kPairThreads = 384;

// XN: activation rows of a tile, 256 or 128
template <int XN>
struct Pair {
    static constexpr int kXCodes = XN / 2 * 128;        // a CTA's half of the rows
    static constexpr int kXScales = XN / 128 * 1024;    // both CTAs need those of all rows
    static constexpr int kSlotBytes = kMxTileBytes + kXCodes + kXScales;
    static constexpr int kSlots = XN == 256 ? 6 : 8;
    static constexpr int kSfCols = 8 + XN / 16;         // tensor-memory columns of a slot's scales
    static constexpr int kSmemBytes = kSlots * kSlotBytes + 1024;
    static_assert(XN + kSlots * kSfCols <= 512, "tensor memory");
    static_assert(kSmemBytes + 256 <= 232448, "shared memory");
};

constexpr int kPairMaxSlots = 8;
struct PairSmem {
    uint64_t full[kPairMaxSlots], empty[kPairMaxSlots];
    uint64_t d_full, d_empty, mma_done;
    uint32_t tmem_base;
    int abort_flag;
};

// Says that this warp has read its part of the accumulator.  Relaxed: what it
// read is in registers (tcgen05.wait::ld), it hands over no memory, and a
// release would wait for the last tile's stores of Y.
__device__ __forceinline__ void arrive_remote(uint64_t *bar, uint32_t rank) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote_addr(smem_addr(bar), rank))
                 : "memory");
}

// Tile t's place: bands of up to kBand tiles along M, within a band M fastest,
// so that the tiles worked at one time form a near square and share their
// weight and activation tiles in L2 (4096 x 16384 x 5120, us: bands of 4 131,
// of 8 129, of 16 125; one band of all tiles along N first 213 against 200 when
// it was tried).
constexpr int kBand = 16;
struct TilePlace {
    int n, m;
};
__device__ __forceinline__ TilePlace place_of(const PairParams &P, int t) {
    const int per_band = kBand * P.tiles_n, band = t / per_band, r = t - band * per_band;
    const int rows = min(kBand, P.tiles_m - band * kBand), n = r / rows;
    return {n, band * kBand + r - n * rows};
}

// A producer warp's walk: `copy(place, slot, step, barrier)` for each step of
// each tile, once the slot is free; `bytes` land in each CTA.  A tile past the
// last of W or X is the last one again, for rows or columns that are not
// stored.
template <int SLOTS, class Copy>
__device__ __forceinline__ void produce(const PairParams &P, PairSmem &S, int first, int step, int rank, int bytes, Copy &&copy) {
    if ((threadIdx.x & 31) != 0) return;
    int s = 0, issued = 0;
    uint32_t parity = 1;
    for (int t = first; t < P.tiles; t += step) {
        const TilePlace at = place_of(P, t);
        for (int i = 0; i < P.kt; ++i, ++issued) {
            if (!wait_or_abort(&S.empty[s], parity, &S.abort_flag, P.err)) {
                if (rank == 0) drain(S.full, SLOTS, issued, P.err);
                return;
            }
            if (rank == 0) mbar_arrive_expect_tx(&S.full[s], 2 * bytes);
            copy(at, s, i, remote_addr(smem_addr(&S.full[s]), 0));
            if (++s == SLOTS) { s = 0; parity ^= 1; }
        }
    }
}

template <bool BF16, int XN>
__global__ void __launch_bounds__(kPairThreads, 1) __cluster_dims__(2, 1, 1) mx_pair_kernel(const __grid_constant__ PairParams P) {
    using C = Pair<XN>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ PairSmem S;
    uint8_t *const ring = align_smem<1024>(smem_raw);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = static_cast<int>(blockIdx.x) & 1;
    const int first = static_cast<int>(blockIdx.x) >> 1, step = static_cast<int>(gridDim.x) >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kSlots; ++s) {
            mbar_init(&S.full[s], 3);   // the first CTA's producers, which answer for both CTAs' bytes
            mbar_init(&S.empty[s], 1);
        }
        mbar_init(&S.d_full, 1);
        mbar_init(&S.d_empty, 16);                      // the epilogue warps of both CTAs
        mbar_init(&S.mma_done, 1);
        S.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc_pair(&S.tmem_base, 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();   // the other CTA's barriers exist
    tc_fence_after();
    begin_dependent();   // all warps: their waits are bounded, the kernel before is not
    const uint32_t tmem = S.tmem_base;

    if (warp == 0) {
        produce<C::kSlots>(P, S, first, step, rank, kMxTileBytes, [&](const TilePlace &at, int s, int i, uint32_t bar) {
            const int y = 17 * (min(2 * at.n + rank, P.wt - 1) * P.kt + i);
            if (Q4_DEBUG_BAD(s < C::kSlots && y >= 0 && y + 17 <= 17 * P.wt * P.kt, P.err, &S.abort_flag)) return;
            tma_load_pair(smem_addr(ring) + s * C::kSlotBytes, &P.map_w, y, bar);
        });
    } else if (warp == 10) {
        produce<C::kSlots>(P, S, first, step, rank, C::kXCodes, [&](const TilePlace &at, int s, int i, uint32_t bar) {
            const int y = XN == 256 ? 17 * (min(2 * at.m + rank, P.xt - 1) * P.kt + i) : 17 * (at.m * P.kt + i) + 8 * rank;
            if (Q4_DEBUG_BAD(s < C::kSlots && y >= 0 && y + C::kXCodes / 1024 < 17 * P.xt * P.kt, P.err, &S.abort_flag)) return;
            tma_load_pair(smem_addr(ring) + s * C::kSlotBytes + kMxTileBytes, &P.map_x, y, bar);
        });
    } else if (warp == 11) {
        produce<C::kSlots>(P, S, first, step, rank, C::kXScales, [&](const TilePlace &at, int s, int i, uint32_t bar) {
            #pragma unroll
            for (int h = 0; h < XN / 128; ++h) {
                const int y = 17 * (min(XN / 128 * at.m + h, P.xt - 1) * P.kt + i) + 16;
                if (Q4_DEBUG_BAD(s < C::kSlots && y >= 0 && y < 17 * P.xt * P.kt, P.err, &S.abort_flag)) return;
                tma_load_pair(smem_addr(ring) + s * C::kSlotBytes + kMxTileBytes + C::kXCodes + 1024 * h, &P.map_xs, y, bar);
            }
        });
    } else if (warp == 1 && rank == 0) {
        constexpr uint32_t idesc = mxf4_idesc(256, XN, 0);
        int s = 0;
        uint32_t parity = 0, dpar = 1;
        bool ok = true;
        for (int t = first; t < P.tiles && ok; t += step, dpar ^= 1) {
            if (!(ok = all_lanes(wait_or_abort(&S.d_empty, dpar, &S.abort_flag, P.err)))) break;
            tc_fence_after();
            for (int i = 0; i < P.kt; ++i) {
                if (!(ok = all_lanes(wait_or_abort(&S.full[s], parity, &S.abort_flag, P.err)))) break;
                tc_fence_after();
                const uint32_t base = smem_addr(ring) + s * C::kSlotBytes;
                const uint32_t sfa = tmem + XN + C::kSfCols * s, sfb = sfa + 8;
                const uint64_t a = sw128_kmajor_desc(base), b = sw128_kmajor_desc(base + kMxTileBytes);
                const uint64_t da = scales_desc(base + kMxCodeBytes), db = scales_desc(base + kMxTileBytes + C::kXCodes);
                __syncwarp();
                if (elect_one()) {
                    #pragma unroll
                    for (int g = 0; g < 2; ++g) {   // 512 bytes on: 32 in the descriptor's units
                        tc_cp_scales_pair(sfa + 4 * g, da + 32 * g);
                        #pragma unroll
                        for (int h = 0; h < XN / 128; ++h) tc_cp_scales_pair(sfb + XN / 32 * g + 4 * h, db + 64 * h + 32 * g);
                    }
                    #pragma unroll
                    for (int j = 0; j < 4; ++j)
                        tc_mma_mxf4_pair(tmem, a + 2 * j, b + 2 * j, idesc | ((j & 1) ? mxf4_idesc(0, 0, 2) : 0u),
                                         sfa + 4 * (j >> 1), sfb + XN / 32 * (j >> 1), (i | j) != 0);
                    tc_commit_pair(&S.empty[s]);
                    if (i == P.kt - 1) tc_commit_pair(&S.d_full);
                }
                __syncwarp();
                if (++s == C::kSlots) { s = 0; parity ^= 1; }
            }
        }
        // every MMA issued so far has completed once this commit arrives
        if (elect_one()) tc_commit_pair_own(&S.mma_done);
        __syncwarp();
        wait_or_abort(&S.mma_done, 0, &S.abort_flag, P.err) || mbar_wait(&S.mma_done, 0, P.err);
    } else if (warp >= 2) {
        const int quad = warp & 3, half = (warp - 2) >> 2;   // lanes [32 quad, +32), columns [XN/2 half, +XN/2)
        uint32_t parity = 0;
        for (int t = first; t < P.tiles; t += step, parity ^= 1) {
            if (!all_lanes(wait_or_abort(&S.d_full, parity, &S.abort_flag, P.err))) break;
            tc_fence_after();
            float v[XN / 64][32];
            #pragma unroll
            for (int c = 0; c < XN / 64; ++c)
                tc_ld_cols<32>(tmem + (uint32_t(32 * quad) << 16) + XN / 2 * half + 32 * c, v[c]);
            tc_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_remote(&S.d_empty, 0);
            const TilePlace at_tile = place_of(P, t);
            const int64_t n = static_cast<int64_t>(2 * at_tile.n + rank) * 128 + 32 * quad + lane;
            const int64_t m = static_cast<int64_t>(at_tile.m) * XN + XN / 2 * half;
            if (n < P.N && m < P.M) {
                // whole tiles without a test for each row: with one, storing a
                // tile took longer (9600 cycles) than the MMAs of 18 steps
                using T = typename std::conditional<BF16, __nv_bfloat16, float>::type;
                T *y = static_cast<T *>(P.Y) + m * P.N + n;
                const int live = static_cast<int>(P.M - m < XN / 2 ? P.M - m : XN / 2);
                if (live == XN / 2) {
                    #pragma unroll
                    for (int c = 0; c < XN / 64; ++c)
                        #pragma unroll
                        for (int j = 0; j < 32; ++j, y += P.N) put(y, v[c][j]);
                } else {
                    #pragma unroll
                    for (int c = 0; c < XN / 64; ++c)
                        #pragma unroll
                        for (int j = 0; j < 32; ++j, y += P.N)
                            if (32 * c + j < live) put(y, v[c][j]);
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();   // no MMA or copy of either CTA is left
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
    cluster_sync_all();
}

template <bool BF16, int XN>
cudaError_t launch_pair(PairParams &p, const q4::DeviceInfo &dev, cudaStream_t s) {
    constexpr int bytes = Pair<XN>::kSmemBytes;
    static q4::DeviceOnce configured;
    static q4::DeviceValue resident;
    const cudaError_t e = configured.run(dev.device, [] {
        return cudaFuncSetAttribute(mx_pair_kernel<BF16, XN>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int pairs = resident.get(dev.device, [&] {
        cudaLaunchConfig_t c = cfg;
        cudaLaunchAttribute cl;
        cl.id = cudaLaunchAttributeClusterDimension;
        cl.val.clusterDim.x = 2;
        cl.val.clusterDim.y = cl.val.clusterDim.z = 1;
        c.gridDim = dim3(dev.sm_count / 2 * 2);
        c.stream = nullptr;
        c.attrs = &cl;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, mx_pair_kernel<BF16, XN>, &c) != cudaSuccess) n = 0;
        (void)cudaGetLastError();
        return n > 0 ? n : dev.sm_count / 2;
    });
    cfg.gridDim = dim3(2 * (p.tiles < pairs ? p.tiles : pairs));
    return cudaLaunchKernelEx(&cfg, mx_pair_kernel<BF16, XN>, p);
}

}  // namespace

namespace q4 {

cudaError_t launch_mx_gemm(const uint8_t *W, const uint8_t *X, void *Y, int y_type, int64_t M, int64_t N, int64_t K,
                           const DeviceInfo &dev, cudaStream_t s) {
    const int64_t kt = mx_k_tiles(K), wt = mx_row_tiles(N), xt = mx_row_tiles(M);
    const bool bf16 = y_type == Q4_TYPE_BF16;
    // up to 128 rows, one tile of X, the pair kernel's weight tiles are as many
    // but go to half as many places, and it cannot split K (us, split and pair:
    // 64 x 16384 x 5120 10.2 and 10.9, 64 x 5120 x 8192 10.0 and 11.4, 64 x 1024 x 5120
    // 5.6 and 8.3, 64 x 32768 x 5120 16.9 and 21.2, 128 x 16384 x 5120 11.1 and 11.5,
    // 128 x 2048 x 2048 5.6 and 6.2; the other way 128 x 8192 x 5120 9.8 and 9.5)
    if (M <= q4::kMxTileRows) return launch_split(W, X, Y, bf16, M, N, kt, dev, s);
    const int64_t tiles_n = (wt + 1) / 2;
    // tiles of 128 activation rows while they all run at once, of 256 beyond
    // (us, 128 and 256: 333 x 5003 x 4128 8.9 and 11.3, 512 x 2048 x 2048 6.2 and
    // 7.9; 256 x 16384 x 5120 15.9 and 13.6, 600 x 5120 x 4096 12.6 and 11.3)
    const bool wide = tiles_n * xt > dev.sm_count / 2;
    const int64_t tiles_m = wide ? (xt + 1) / 2 : xt, tiles = tiles_n * tiles_m;
    if (tiles > 0x7fffffff || 17 * wt * kt > 0x7fffffff || 17 * xt * kt > 0x7fffffff) return cudaErrorInvalidValue;
    PairParams p;
    if (!encode_1k_rows_map(&p.map_w, W, 17 * wt * kt, 17) || !encode_1k_rows_map(&p.map_x, X, 17 * xt * kt, wide ? 16 : 8) ||
        !encode_1k_rows_map(&p.map_xs, X, 17 * xt * kt, 1))
        return cudaErrorInvalidValue;
    p.Y = Y;
    p.err = dev.err;
    p.M = M;
    p.N = N;
    p.kt = static_cast<int>(kt);
    p.wt = static_cast<int>(wt);
    p.xt = static_cast<int>(xt);
    p.tiles_n = static_cast<int>(tiles_n);
    p.tiles_m = static_cast<int>(tiles_m);
    p.tiles = static_cast<int>(tiles);
    if (wide) return bf16 ? launch_pair<true, 256>(p, dev, s) : launch_pair<false, 256>(p, dev, s);
    return bf16 ? launch_pair<true, 128>(p, dev, s) : launch_pair<false, 128>(p, dev, s);
}

}  // namespace q4
