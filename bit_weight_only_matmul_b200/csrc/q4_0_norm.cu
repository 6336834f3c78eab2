// q4_0_norm.cu -- the step between two products of a decoder: the norm of a
// block's output, its gate and residual scale, the residual add and the norm
// in front of the next block, in one pass.
//
//     h  = y                        or  y / sqrt(mean(y^2) + eps) * post
//     r' = r + scale * gate * h     (r' = r without y)
//     x  = r' / sqrt(mean(r'^2) + eps) * pre
//
// Memory-bound: y and r are read once and r' and x written once, everything
// in between stays in registers.  A row belongs to a CTA; a thread holds G
// groups of eight values, a group being two runs of four, 128 values apart,
// in the 256 values of its warp: every load and store of a warp is one
// contiguous piece, and a warp's group is one row of an MXFP4 tile, so that x
// can be written as MXFP4.  The two sums go through shuffles and one line of
// shared memory and are added in a fixed order.  All arithmetic is fp32; r' is
// rounded once to r's type, and x is taken from r' before that rounding.
//
// Two kernels.  block_norm_kernel keeps a row's values in registers from the
// load on: for few rows, where one row's time is all there is.
// block_norm_many_kernel lands them in shared memory first (each thread copies
// what it will read itself, so nobody waits for anybody), which leaves room on
// an SM for twice as many rows: a row's time is mostly waiting, for memory and
// for its two sums.  Keeping all values in registers, 4096 x 8192 fp32 took
// 97 us against 77 (6.1 TB/s); a persistent kernel with a ring of rows in shared
// memory 80, and more than this one for shorter rows (4096 x 5120 80 against 55).
#include "mxfp4_layout.cuh"

namespace {

using namespace q4dev;

struct NormParams {
    const void *y, *r;
    void *r_out, *x;
    const float *post, *gate, *pre;
    int64_t M, gate_span;
    int D, kt;
    float scale, eps;
    int x_type;
};

__device__ __forceinline__ float warp_sum(float v) {
    #pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The sum over the CTA, the same bits in all lanes: every warp adds the line
// itself, in the same order.
__device__ __forceinline__ float block_sum(float v, float *part, int warps) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum((threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : 0.f);
}

__device__ __forceinline__ void quad(float4 a, float (&v)[8], int h) {
    v[4 * h] = a.x; v[4 * h + 1] = a.y; v[4 * h + 2] = a.z; v[4 * h + 3] = a.w;
}

// A group as it lies in memory, its first run at `p`; a
// run past the row's end (low, high: there is a first, a second one) stays zero.
template <class T> struct Raw;
template <> struct Raw<float> {
    float4 q[2];
    __device__ __forceinline__ void load(const float *p, bool low, bool high) {
        if (low) q[0] = __ldcs(reinterpret_cast<const float4 *>(p));
        if (high) q[1] = __ldcs(reinterpret_cast<const float4 *>(p + 128));
    }
    __device__ __forceinline__ void get(float (&v)[8]) const { quad(q[0], v, 0); quad(q[1], v, 1); }
};
template <> struct Raw<__nv_bfloat16> {
    uint2 q[2];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, bool low, bool high) {
        if (low) q[0] = __ldcs(reinterpret_cast<const uint2 *>(p));
        if (high) q[1] = __ldcs(reinterpret_cast<const uint2 *>(p + 128));
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        #pragma unroll
        for (int h = 0; h < 2; ++h)
            quad(make_float4(__uint_as_float(q[h].x << 16), __uint_as_float(q[h].x & 0xFFFF0000u),
                             __uint_as_float(q[h].y << 16), __uint_as_float(q[h].y & 0xFFFF0000u)), v, h);
    }
};

__device__ __forceinline__ void load_weights(const float *p, bool low, bool high, float (&v)[8]) {
    quad(low ? __ldg(reinterpret_cast<const float4 *>(p)) : make_float4(0.f, 0.f, 0.f, 0.f), v, 0);
    quad(high ? __ldg(reinterpret_cast<const float4 *>(p + 128)) : make_float4(0.f, 0.f, 0.f, 0.f), v, 1);
}

// One run of a group.
__device__ __forceinline__ void store_run(float *p, const float *v) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store_run(__nv_bfloat16 *p, const float *v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

// What a thread does with its G groups of a row.  Column of run h of group j:
// first + 256 * warps * j + 128 * h.
template <int G>
struct Lane {
    int first, step;   // step: 256 * warps
    __device__ __forceinline__ Lane(int warp, int lane, int warps) : first(256 * warp + 4 * lane), step(256 * warps) {}
    __device__ __forceinline__ int column(int j, int h) const { return first + step * j + 128 * h; }
};

template <int G>
__device__ __forceinline__ float square_sum(const float (&v)[G][8]) {
    float ss[4] = {};   // four chains: one would wait for itself at every step
    #pragma unroll
    for (int j = 0; j < G; ++j)
        #pragma unroll
        for (int i = 0; i < 8; ++i) ss[i & 3] = fmaf(v[j][i], v[j][i], ss[i & 3]);
    return (ss[0] + ss[1]) + (ss[2] + ss[3]);
}

// w = post * gate of a group (1 where one is missing).
__device__ __forceinline__ void block_weights(const NormParams &P, const float *gate, int k, float (&w)[8]) {
    const bool low = k < P.D, high = k + 128 < P.D;
    if (P.post) load_weights(P.post + k, low, high, w);
    else if (gate) load_weights(gate + k, low, high, w);
    else {
        #pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 1.f;
    }
    if (P.post && gate) {
        float g[8];
        load_weights(gate + k, low, high, g);
        #pragma unroll
        for (int i = 0; i < 8; ++i) w[i] *= g[i];
    }
}

__device__ __forceinline__ const float *gate_row(const NormParams &P, int64_t row) {
    return !P.gate ? nullptr : P.gate + (P.gate_span ? row / P.gate_span : 0) * P.D;
}

// r' of a group from h, its weight and r.
__device__ __forceinline__ void add_block(float (&h)[8], const float (&w)[8], float fy, const float (&r)[8]) {
    #pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = fmaf(h[i] * w[i], fy, r[i]);
}

template <int G, class T>
__device__ __forceinline__ void store_row(void *p, int64_t at, const Lane<G> &L, int D, const float (&v)[G][8]) {
    T *q = static_cast<T *>(p) + at;
    #pragma unroll
    for (int j = 0; j < G; ++j) {
        const int k = L.column(j, 0);
        if (k < D) store_run(q + k, v[j]);
        if (k + 128 < D) store_run(q + k + 128, v[j] + 4);
    }
}

// x as one row of an MXFP4 matrix: a block is one run of eight lanes, and whole
// warps take part (blocks past D: zero codes and a zero scale byte).
template <int G>
__device__ __forceinline__ void store_mxfp4(const NormParams &P, int64_t row, const Lane<G> &L, int lane, const float (&v)[G][8]) {
    uint32_t a[G][2];   // the blocks' largest magnitudes, all on their way at once
    #pragma unroll
    for (int j = 0; j < G; ++j)
        #pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float *u = v[j] + 4 * h;
            a[j][h] = magnitude_bits(max_abs(max_abs(u[0], u[1], u[2]), u[3], u[3]));
        }
    #pragma unroll
    for (int o = 1; o < 8; o <<= 1)
        #pragma unroll
        for (int j = 0; j < G; ++j)
            #pragma unroll
            for (int h = 0; h < 2; ++h) a[j][h] = max(a[j][h], __shfl_xor_sync(0xffffffffu, a[j][h], o));
    const int r = static_cast<int>(row & 127);
    uint8_t *const tiles = static_cast<uint8_t *>(P.x) + (row >> 7) * P.kt * q4::kMxTileBytes;
    #pragma unroll
    for (int j = 0; j < G; ++j) {
        const int k = L.column(j, 0), tile_k = k >> 8;   // the same in the whole warp
        if (tile_k < P.kt) {
            uint8_t *tile = tiles + static_cast<int64_t>(tile_k) * q4::kMxTileBytes;
            #pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool live = k + 128 * h < P.D;
                const uint32_t byte = live ? mx_scale_byte(a[j][h]) : 0u;
                const float inv = mx_inverse_scale(a[j][h]);
                const float *u = v[j] + 4 * h;
                const uint32_t code = live ? e2m1x4(u[0] * inv, u[1] * inv, u[2] * inv, u[3] * inv) : 0u;
                const int b = 4 * h + (lane >> 3);
                *reinterpret_cast<uint16_t *>(tile + mx_code_offset(r, b) + 2 * (lane & 7)) = static_cast<uint16_t>(code);
                if ((lane & 7) == 0) tile[mx_scale_offset(r, h) + (lane >> 3)] = static_cast<uint8_t>(byte);
            }
        }
    }
}

template <int G>
__device__ __forceinline__ void store_x(const NormParams &P, int64_t row, const Lane<G> &L, int lane, const float (&v)[G][8]) {
    if (P.x_type == Q4_TYPE_MXFP4) store_mxfp4<G>(P, row, L, lane, v);
    else if (P.x_type == Q4_TYPE_BF16) store_row<G, __nv_bfloat16>(P.x, row * P.D, L, P.D, v);
    else store_row<G, float>(P.x, row * P.D, L, P.D, v);
}

// ---------------------------------------------------------------- a row a CTA

// EAGER: the weights are on their way with the rows; where they would not fit
// in the registers as well they are loaded when they are needed.
template <int G, int T, bool EAGER, class YT, class RT>
__global__ void __launch_bounds__(T) block_norm_kernel(const __grid_constant__ NormParams P) {
    __shared__ float part[2][32];
    begin_dependent();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const Lane<G> L(warp, lane, warps);
    const int64_t row = blockIdx.x, at = row * P.D;
    const float *gate = gate_row(P, row);
    float v[G][8], w[EAGER ? G : 1][8], pre[EAGER ? G : 1][8];
    Raw<RT> q[G] = {};
    {
        Raw<YT> y[G] = {};
        #pragma unroll
        for (int j = 0; j < G; ++j) {
            const int k = L.column(j, 0);
            if (P.y) y[j].load(static_cast<const YT *>(P.y) + at + k, k < P.D, k + 128 < P.D);
        }
        #pragma unroll
        for (int j = 0; j < G; ++j) {
            const int k = L.column(j, 0);
            q[j].load(static_cast<const RT *>(P.r) + at + k, k < P.D, k + 128 < P.D);
        }
        if (EAGER) {
            #pragma unroll
            for (int j = 0; j < G; ++j) {
                const int k = L.column(j, 0);
                if (P.y) block_weights(P, gate, k, w[j]);
                if (P.pre) load_weights(P.pre + k, k < P.D, k + 128 < P.D, pre[j]);
            }
        }
        #pragma unroll
        for (int j = 0; j < G; ++j) y[j].get(v[j]);
    }
    float fy = P.scale;
    if (P.y && P.post) fy *= rsqrtf(block_sum(square_sum<G>(v), part[0], warps) / static_cast<float>(P.D) + P.eps);
    #pragma unroll
    for (int j = 0; j < G; ++j) {
        float r[8];
        q[j].get(r);
        if (P.y) {
            if (!EAGER) block_weights(P, gate, L.column(j, 0), w[0]);
            add_block(v[j], w[EAGER ? j : 0], fy, r);
        } else {
            #pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] = r[i];
        }
    }
    if (P.r_out) store_row<G, RT>(P.r_out, at, L, P.D, v);
    if (P.x) {
        const float fx = rsqrtf(block_sum(square_sum<G>(v), part[1], warps) / static_cast<float>(P.D) + P.eps);
        #pragma unroll
        for (int j = 0; j < G; ++j) {
            const int k = L.column(j, 0);
            if (!EAGER && P.pre) load_weights(P.pre + k, k < P.D, k + 128 < P.D, pre[0]);
            #pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] = P.pre ? v[j][i] * fx * pre[EAGER ? j : 0][i] : v[j][i] * fx;
        }
        store_x<G>(P, row, L, lane, v);
    }
}

// ---------------------------------------------------------------- many rows

// One run of a group from global to shared memory: 16 bytes of fp32, 8 of bf16.
__device__ __forceinline__ void copy_run(uint32_t dst, const float *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_run(uint32_t dst, const __nv_bfloat16 *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void get_run(const float *p, float *v) {
    const float4 a = *reinterpret_cast<const float4 *>(p);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ void get_run(const __nv_bfloat16 *p, float *v) {
    const uint2 a = *reinterpret_cast<const uint2 *>(p);
    v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xFFFF0000u);
    v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xFFFF0000u);
}

// A thread's groups of a row between global memory, shared memory and
// registers; run (j, h) of thread t at (2j + h) * threads + t.
template <int G, class T>
struct Landing {
    T *mine;
    int gap;
    __device__ __forceinline__ Landing(uint8_t *base) : mine(reinterpret_cast<T *>(base) + 4 * threadIdx.x), gap(4 * blockDim.x) {}
    __device__ __forceinline__ void copy(const T *row, const Lane<G> &L, int D) const {
        #pragma unroll
        for (int j = 0; j < G; ++j)
            #pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = L.column(j, h);
                if (k < D) copy_run(smem_addr(mine + (2 * j + h) * gap), row + k);
            }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __device__ __forceinline__ void get(const Lane<G> &L, int D, int j, float (&v)[8]) const {
        #pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (L.column(j, h) < D) {
                get_run(mine + (2 * j + h) * gap, v + 4 * h);
            } else {
                #pragma unroll
                for (int i = 0; i < 4; ++i) v[4 * h + i] = 0.f;
            }
        }
    }
};

// CTAs that an SM's registers must leave room for, by groups and threads.
constexpr int many_ctas(int G, int T) { return T == 256 ? 3 : G == 4 ? 1 : 2; }

template <int G, int T, class YT, class RT>
__global__ void __launch_bounds__(T, many_ctas(G, T)) block_norm_many_kernel(const __grid_constant__ NormParams P) {
    extern __shared__ __align__(16) uint8_t landing[];
    __shared__ float part[2][32];
    begin_dependent();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const Lane<G> L(warp, lane, warps);
    const int64_t row = blockIdx.x, at = row * P.D;
    const Landing<G, YT> y(landing);
    const Landing<G, RT> r(landing + (P.y ? blockDim.x * G * 8 * sizeof(YT) : 0));
    if (P.y) y.copy(static_cast<const YT *>(P.y) + at, L, P.D);
    r.copy(static_cast<const RT *>(P.r) + at, L, P.D);
    const float *gate = gate_row(P, row);
    float v[G][8];
    float fy = P.scale;
    if (P.y) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        #pragma unroll
        for (int j = 0; j < G; ++j) y.get(L, P.D, j, v[j]);
        if (P.post) fy *= rsqrtf(block_sum(square_sum<G>(v), part[0], warps) / static_cast<float>(P.D) + P.eps);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    #pragma unroll
    for (int j = 0; j < G; ++j) {
        float q[8];
        r.get(L, P.D, j, q);
        if (P.y) {
            float w[8];
            block_weights(P, gate, L.column(j, 0), w);
            add_block(v[j], w, fy, q);
        } else {
            #pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] = q[i];
        }
    }
    if (P.r_out) store_row<G, RT>(P.r_out, at, L, P.D, v);
    if (P.x) {
        const float fx = rsqrtf(block_sum(square_sum<G>(v), part[1], warps) / static_cast<float>(P.D) + P.eps);
        #pragma unroll
        for (int j = 0; j < G; ++j) {
            float w[8];
            const int k = L.column(j, 0);
            if (P.pre) load_weights(P.pre + k, k < P.D, k + 128 < P.D, w);
            #pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] = P.pre ? v[j][i] * fx * w[i] : v[j][i] * fx;
        }
        store_x<G>(P, row, L, lane, v);
    }
}

// ---------------------------------------------------------------- host side

template <class F>
cudaError_t by_types(const q4_0_block &b, F &&f) {
    using B = __nv_bfloat16;
    const bool yf = !b.y || b.y_type == Q4_TYPE_F32, rf = b.r_type == Q4_TYPE_F32;
    if (yf) return rf ? f(float(), float()) : f(float(), B());
    return rf ? f(B(), float()) : f(B(), B());
}

template <int G, int T, bool EAGER>
cudaError_t launch_rows(const q4_0_block &b, const NormParams &p, int warps, cudaStream_t s) {
    return by_types(b, [&](auto y, auto r) {
        return launch_dependent(block_norm_kernel<G, T, EAGER, decltype(y), decltype(r)>, p.M, 32 * warps, s, p);
    });
}

template <int G, int T>
cudaError_t launch_many(const q4_0_block &b, const NormParams &p, int warps, const q4::DeviceInfo &dev, cudaStream_t s) {
    return by_types(b, [&](auto y, auto r) {
        const auto kernel = block_norm_many_kernel<G, T, decltype(y), decltype(r)>;
        constexpr int most = T * G * 8 * (sizeof(y) + sizeof(r));
        if (most > 47 * 1024) {   // more than a CTA gets unasked, with the sums beside it
            static q4::DeviceOnce configured;
            const cudaError_t e = configured.run(dev.device, [&] {
                return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
            });
            if (e != cudaSuccess) return e;
        }
        const size_t bytes = static_cast<size_t>(32 * warps) * G * 8 * ((p.y ? sizeof(y) : 0) + sizeof(r));
        return launch_dependent_smem(kernel, p.M, 32 * warps, bytes, s, p);
    });
}

}  // namespace

namespace q4 {

cudaError_t launch_block_norm(const q4_0_block &b, const DeviceInfo &dev, cudaStream_t s) {
    NormParams p;
    p.y = b.y;
    p.r = b.r;
    p.r_out = b.r_out;
    p.x = b.x;
    p.post = b.post_weight;
    p.gate = b.gate;
    p.pre = b.pre_weight;
    p.M = b.M;
    p.gate_span = b.gate_span;
    p.D = static_cast<int>(b.D);
    p.kt = static_cast<int>(mx_k_tiles(b.D));
    p.scale = b.scale;
    p.eps = b.eps;
    p.x_type = b.x_type;
    const int groups = p.kt;   // of a warp: 256 values
    // More rows than SMs: fewer warps a row, so that more rows are in flight.
    // Two groups a thread, four for the longest rows (us, two and four: 1001 x
    // 4128 bf16 10.2 and 11.6, 4096 x 5120 46.9 and 50.9, 4096 x 6144 bf16 and
    // fp32 49.0 and 51.8; 4096 x 8192 74.0 and 75.8, in bf16 59.4 and 55.4).
    if (b.M > dev.sm_count && groups <= 64) {
        if (groups <= 4) return launch_many<1, 512>(b, p, groups, dev, s);
        if (groups <= 24) return launch_many<2, 512>(b, p, (groups + 1) / 2, dev, s);
        if (groups <= 32) return launch_many<4, 256>(b, p, (groups + 3) / 4, dev, s);
        return launch_many<4, 512>(b, p, (groups + 3) / 4, dev, s);
    }
    // as many warps as the row has groups, for the shortest time of a row
    if (groups <= 16) return launch_rows<1, 512, true>(b, p, groups, s);
    if (groups <= 32) return launch_rows<1, 1024, true>(b, p, groups, s);
    if (groups <= 64) return launch_rows<2, 1024, true>(b, p, (groups + 1) / 2, s);
    // rows above 16384 values, of any number: y and r of 32768 in fp32 are more
    // than an SM's shared memory, so there is no landing them.  With 1024 threads
    // of 64 registers each some values spill (40 to 68 bytes a thread for two
    // groups, 104 to 224 for four): 2000 x 20000 fp32 165 us, 3.4 TB/s, where 2000 x
    // 16384 lands and takes 96 (4.8 TB/s); 1 x 16384 6.0 us, 1 x 32768 13.2
    return launch_rows<4, 1024, false>(b, p, (groups + 3) / 4, s);
}

}  // namespace q4
