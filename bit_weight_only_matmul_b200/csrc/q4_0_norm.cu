// q4_0_norm.cu -- the step between two products of a decoder: the norm of a
// block's output, its gate and residual scale, the residual add and the norm
// in front of the next block, in one pass.
//
//     h  = y                        or  y / sqrt(mean(y^2) + eps) * post
//     r' = r + scale * gate * h     (r' = r without y)
//     x  = r' / sqrt(mean(r'^2) + eps) * pre
//
// Memory-bound: y and r are read once and r' and x written once, everything
// in between stays in registers.  A CTA takes a row; a thread holds G groups
// of eight consecutive values, so that a warp's group is one row of an MXFP4
// tile (256 k) and x can be written as MXFP4 with the code that
// mxfp4_quantize uses.  The two sums go through shuffles and one line of
// shared memory and are added in a fixed order.  All arithmetic is fp32; r'
// is rounded once to r's type, and x is taken from r' before that rounding.
#include "mxfp4_layout.cuh"

namespace {

using namespace q4dev;

struct NormParams {
    const void *y, *r;
    void *r_out, *x;
    const float *post, *gate, *pre;
    int64_t M, D, gate_span, kt;
    float scale, eps;
    int y_type, r_type, x_type;
};

__device__ __forceinline__ float block_sum(float v, float *part) {
    #pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    // every warp adds the line itself: the same order, the same bits in all lanes
    float s = (threadIdx.x & 31) < (blockDim.x >> 5) ? part[threadIdx.x & 31] : 0.f;
    #pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

__device__ __forceinline__ void weights8(const float *p, float (&v)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ void store8_any(void *p, int type, int64_t at, const float (&v)[8]) {
    if (type == Q4_TYPE_F32) {
        float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + at);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint32_t w[4];
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p) + at) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// G: groups of eight values a thread holds; T: threads at most; YT, RT: the
// types of y and r.
template <int G, int T, class YT, class RT>
__global__ void __launch_bounds__(T, G == 2 && T == 512 ? 2 : 1) block_norm_kernel(const __grid_constant__ NormParams P) {
    __shared__ float part[2][32];
    begin_dependent();
    const int lane = threadIdx.x & 31;
    const int D = static_cast<int>(P.D), gap = 8 * blockDim.x;
    for (int64_t row = blockIdx.x; row < P.M; row += gridDim.x) {
        const int64_t at = row * P.D;
        // both rows on their way before the first sum
        Raw8<YT> y[G];
        Raw8<RT> r[G];
        #pragma unroll
        for (int j = 0; j < G; ++j) {
            const int k = 8 * threadIdx.x + j * gap;
            if (k < D && P.y) y[j].load(P.y, at + k);
        }
        #pragma unroll
        for (int j = 0; j < G; ++j) {
            const int k = 8 * threadIdx.x + j * gap;
            if (k < D) r[j].load(P.r, at + k);
        }
        float fy = P.scale;
        if (P.y && P.post) {
            float ss = 0.f;
            #pragma unroll
            for (int j = 0; j < G; ++j)
                if (8 * threadIdx.x + j * gap < D) {
                    float v[8];
                    y[j].get(v);
                    #pragma unroll
                    for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
                }
            fy *= rsqrtf(block_sum(ss, part[0]) / static_cast<float>(D) + P.eps);
        }
        const float *gate = P.gate ? P.gate + (P.gate_span ? row / P.gate_span : 0) * P.D : nullptr;
        float v[G][8];   // r'
        float ss = 0.f;
        #pragma unroll
        for (int j = 0; j < G; ++j) {
            const int k = 8 * threadIdx.x + j * gap;
            if (k < D) {
                r[j].get(v[j]);
                if (P.y) {
                    float h[8], w[8];
                    y[j].get(h);
                    if (P.post) {
                        weights8(P.post + k, w);
                        #pragma unroll
                        for (int i = 0; i < 8; ++i) h[i] *= w[i];
                    }
                    if (gate) {
                        weights8(gate + k, w);
                        #pragma unroll
                        for (int i = 0; i < 8; ++i) h[i] *= w[i];
                    }
                    #pragma unroll
                    for (int i = 0; i < 8; ++i) v[j][i] = fmaf(h[i], fy, v[j][i]);
                }
                if (P.r_out) store8_any(P.r_out, P.r_type, at + k, v[j]);
                #pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(v[j][i], v[j][i], ss);
            }
        }
        if (P.x) {
            const float fx = rsqrtf(block_sum(ss, part[1]) / static_cast<float>(D) + P.eps);
            #pragma unroll
            for (int j = 0; j < G; ++j) {
                const int k = 8 * threadIdx.x + j * gap;
                const bool live = k < D;
                if (live) {
                    if (P.pre) {
                        float w[8];
                        weights8(P.pre + k, w);
                        #pragma unroll
                        for (int i = 0; i < 8; ++i) v[j][i] = v[j][i] * fx * w[i];
                    } else {
                        #pragma unroll
                        for (int i = 0; i < 8; ++i) v[j][i] *= fx;
                    }
                    if (P.x_type != Q4_TYPE_MXFP4) store8_any(P.x, P.x_type, at + k, v[j]);
                }
                if (P.x_type == Q4_TYPE_MXFP4 && (k >> 8) < P.kt) {   // the whole warp: k >> 8 is the warp's tile
                    if (!live) {
                        #pragma unroll
                        for (int i = 0; i < 8; ++i) v[j][i] = 0.f;
                    }
                    uint32_t byte;
                    const uint32_t code = mx_encode8(v[j], byte);
                    const uint32_t word = mx_scale_word(live ? byte : 0u, lane);
                    uint8_t *tile = static_cast<uint8_t *>(P.x) + ((row >> 7) * P.kt + (k >> 8)) * q4::kMxTileBytes;
                    const int rr = static_cast<int>(row & 127);
                    *reinterpret_cast<uint32_t *>(tile + mx_code_offset(rr, lane >> 2) + 4 * (lane & 3)) = code;
                    if ((lane & 15) == 0) *reinterpret_cast<uint32_t *>(tile + mx_scale_offset(rr, lane >> 4)) = word;
                }
            }
        }
        if (gridDim.x < P.M) __syncthreads();   // the sums' line is written again for the next row
    }
}

template <int G, int T>
cudaError_t launch(const NormParams &p, int threads, int64_t grid, cudaStream_t s) {
    const bool yf = p.y_type == Q4_TYPE_F32, rf = p.r_type == Q4_TYPE_F32;
    using B = __nv_bfloat16;
    return yf ? rf ? launch_dependent(block_norm_kernel<G, T, float, float>, grid, threads, s, p)
                   : launch_dependent(block_norm_kernel<G, T, float, B>, grid, threads, s, p)
              : rf ? launch_dependent(block_norm_kernel<G, T, B, float>, grid, threads, s, p)
                   : launch_dependent(block_norm_kernel<G, T, B, B>, grid, threads, s, p);
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
    p.D = b.D;
    p.gate_span = b.gate_span;
    p.kt = mx_k_tiles(b.D);
    p.scale = b.scale;
    p.eps = b.eps;
    p.y_type = b.y ? b.y_type : Q4_TYPE_F32;
    p.r_type = b.r_type;
    p.x_type = b.x_type;
    // few rows: as many threads as the row has groups, for the shortest time
    // of a row; many: two or four groups a thread, so that a CTA's sums hold
    // up fewer warps and several CTAs fit on an SM
    const int64_t groups = b.D / 8;
    const bool few = b.M <= dev.sm_count;
    const int G = groups <= (few ? 1024 : 256) ? 1 : groups <= (few ? 2048 : 1024) ? 2 : 4;
    const int threads = static_cast<int>(((groups + G - 1) / G + 31) / 32 * 32);
    const int64_t cap = static_cast<int64_t>(dev.sm_count) * 64, grid = b.M < cap ? b.M : cap;
    if (G == 1) return launch<1, 1024>(p, threads, grid, s);
    if (threads <= 512) return G == 2 ? launch<2, 512>(p, threads, grid, s) : launch<4, 512>(p, threads, grid, s);
    return G == 2 ? launch<2, 1024>(p, threads, grid, s) : launch<4, 1024>(p, threads, grid, s);
}

}  // namespace q4
