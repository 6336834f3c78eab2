// mxfp4_quantize.cu -- values to an MXFP4 matrix and back, and an MXFP4
// checkpoint's codes and scales into the library's layout.  All three are one
// pass over memory.
//
// A warp takes two or eight consecutive rows of a tile (256 k, 8 values a
// lane, four lanes a block).  It reads 512 or 1024 contiguous bytes of each
// row, all rows before it works on the first (pack: each row as it stores it),
// finds each block's largest magnitude with two shuffles, and writes each
// row's 128 bytes of codes as one line and its eight scale bytes from eight
// lanes.
//
// Quantize and dequant are bound by HBM (16384 x 5120: quantize of fp32 57.8
// us, 6.6 TB/s, dequant to bf16 34.0 us, 6.2 TB/s), and for 16-bit values by
// the instructions too (quantize of 8192 x 8192 bf16 29.8 us, 5.7 TB/s).  Eight
// rows a warp keep more in flight where there are warps enough (that quantize
// 35.7 us against 39.9 with two rows when it was chosen, dequant to bf16 35.1
// against 44.2); two spread few rows over the SMs (1003 x 4128 fp16 quantize
// 4.3 us against 5.9, now 3.7), and are enough for fp32, whose rows are twice as
// many bytes (16384 x 5120 quantize 57.8 against 59.0 us, dequant 65 against
// 72.5).  Pack, which runs once for a checkpoint, has one row's loads of a warp
// in flight and is bound by their latency: 16384 x 5120 55 us, 1.6 TB/s.
#include "mxfp4_layout.cuh"

namespace {

using namespace q4dev;
using q4::kMxTileBytes;

constexpr int kWarps = 4;       // warps of a CTA

// A warp's part of the matrix, ROWS rows or the last few of one tile column.
// ROWS divides 8, so that row i of the part is row (r & 7) | i of its group of
// eight in the swizzle, and r + i stays within 32 rows of scales.
struct Part {
    int64_t at;        // the lane's first value of the first row
    int rows;
    uint8_t *codes;    // the first row's codes
    uint8_t *scales;   // the first row's scales, blocks 0 to 3
    uint8_t *scale;    // the lane's block's scale byte of the first row
    int word;          // the lane's code word in a row, swizzled as in the first
    bool live;         // the lane's values lie within K
};

template <int ROWS>
__device__ __forceinline__ bool part_of(Part &p, const uint8_t *W, int64_t R, int64_t K, int kt) {
    static_assert(8 % ROWS == 0, "a part lies in a group of eight rows");
    const int lane = threadIdx.x & 31, b = lane >> 2;
    const uint32_t u = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const uint32_t g = u / static_cast<uint32_t>(kt), t = u - g * kt;
    const int64_t row = static_cast<int64_t>(g) * ROWS, k = static_cast<int64_t>(t) * 256 + 8 * lane;
    if (row >= R) return false;
    p.rows = R - row < ROWS ? static_cast<int>(R - row) : ROWS;
    const int r = static_cast<int>(row & 127);
    uint8_t *tile = const_cast<uint8_t *>(W) + ((row >> 7) * kt + t) * kMxTileBytes;
    p.codes = tile + 128 * r;
    p.word = mx_code_offset(r, b) - 128 * r + 4 * (lane & 3);
    p.scales = tile + mx_scale_offset(r, 0);
    p.scale = p.scales + 512 * (b >> 2) + (b & 3);
    p.live = k < K;
    p.at = row * K + k;
    return true;
}

__device__ __forceinline__ uint32_t *code_word(const Part &p, int i) {
    return reinterpret_cast<uint32_t *>(p.codes + 128 * i + (p.word ^ (i << 4)));
}

template <typename T, int ROWS>
__global__ void __launch_bounds__(32 * kWarps, 8)
    mx_quantize_kernel(const T *__restrict__ X, uint8_t *__restrict__ W, int64_t R, int64_t K, int kt) {
    begin_dependent();
    const int lane = threadIdx.x & 31;
    Part p;
    if (!part_of<ROWS>(p, W, R, K, kt)) return;
    Raw8<T> x[ROWS];
    #pragma unroll
    for (int i = 0; i < ROWS; ++i)
        if (p.live && i < p.rows) x[i].load(X, p.at + i * K);
    #pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        if (i < p.rows) {   // the same in all lanes
            float v[8] = {};
            if (p.live) x[i].get(v);
            uint32_t byte;
            const uint32_t code = mx_encode8(v, byte);
            *code_word(p, i) = code;
            if ((lane & 3) == 0) p.scale[16 * i] = static_cast<uint8_t>(byte);   // 0 for a block past K
        }
    }
}

__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
    uint32_t w[4];
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ void store8(__half *p, const float (&v)[8]) {
    uint32_t w[4];
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
}

// E2M1 code to its value: the two exponent bits and the mantissa bit of
// codes 2..7 are those of a float of exponent bias 1; codes 0 and 1 are 0
// and a half.  (c & 7) << 22 is the value's bits times 2^-126 in every case,
// the two subnormal codes included, and one multiplication by a power of two
// makes both adjustments at once, exactly.
__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const float m = __uint_as_float((c & 7u) << 22) * __uint_as_float(253u << 23);
    return __uint_as_float(__float_as_uint(m) | ((c & 8u) << 28));
}

template <typename T, int ROWS>
__global__ void __launch_bounds__(32 * kWarps) mx_dequant_kernel(const uint8_t *__restrict__ W, T *__restrict__ out, int64_t R,
                                                                 int64_t K, int kt) {
    begin_dependent();
    Part p;
    if (!part_of<ROWS>(p, W, R, K, kt)) return;
    uint32_t code[ROWS];
    #pragma unroll
    for (int i = 0; i < ROWS; ++i) code[i] = i < p.rows ? __ldcs(code_word(p, i)) : 0u;
    // lane 2i + g has the scales of row i's blocks 4g .. 4g+3
    const int lane = threadIdx.x & 31;
    const uint32_t words =
        lane < 2 * p.rows ? __ldcs(reinterpret_cast<const uint32_t *>(p.scales + 16 * (lane >> 1) + 512 * (lane & 1))) : 0u;
    T *o = out + p.at;
    #pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const uint32_t word = __shfl_sync(0xffffffffu, words, 2 * i + (lane >> 4));
        if (i < p.rows && p.live) {
            const float s = mx_scale((word >> (8 * ((lane >> 2) & 3))) & 255u);
            float v[8];
            #pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = e2m1_value(code[i] >> (4 * j)) * s;
            store8(o + i * K, v);
        }
    }
}

template <int ROWS>
__global__ void __launch_bounds__(32 * kWarps) mx_pack_kernel(const uint8_t *__restrict__ codes,
                                                              const uint8_t *__restrict__ scales, uint8_t *__restrict__ W,
                                                              int64_t R, int64_t K, int kt) {
    begin_dependent();
    const int lane = threadIdx.x & 31;
    Part p;
    if (!part_of<ROWS>(p, W, R, K, kt)) return;
    #pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        if (i < p.rows) {
            const int64_t at = p.at + i * K;
            *code_word(p, i) = p.live ? __ldcs(reinterpret_cast<const uint32_t *>(codes + at / 2)) : 0u;
            if ((lane & 3) == 0) p.scale[16 * i] = p.live ? scales[at / 32] : 0;
        }
    }
}

// CTAs of a pass over R rows in kt tile columns, `rows` rows a warp; 0 if they
// do not fit a grid (no device memory holds such a matrix).
int64_t grid_for(int64_t R, int64_t kt, int rows) {
    const int64_t parts = (R + rows - 1) / rows * kt;
    return parts > 0x7fffffff ? 0 : (parts + kWarps - 1) / kWarps;
}

// Eight rows a warp where that leaves every SM as many warps as it holds.
bool eight_rows(int type, int64_t R, int64_t kt, const q4::DeviceInfo &dev) {
    return type != Q4_TYPE_F32 && R / 8 * kt >= 64LL * dev.sm_count;
}

template <typename T, int ROWS>
cudaError_t quantize(const void *X, uint8_t *W, int64_t R, int64_t K, int64_t kt, cudaStream_t s) {
    return launch_dependent(mx_quantize_kernel<T, ROWS>, grid_for(R, kt, ROWS), 32 * kWarps, s, static_cast<const T *>(X), W,
                            R, K, static_cast<int>(kt));
}

template <typename T, int ROWS>
cudaError_t dequant(const uint8_t *W, void *out, int64_t R, int64_t K, int64_t kt, cudaStream_t s) {
    return launch_dependent(mx_dequant_kernel<T, ROWS>, grid_for(R, kt, ROWS), 32 * kWarps, s, W, static_cast<T *>(out), R, K,
                            static_cast<int>(kt));
}

}  // namespace

namespace q4 {

cudaError_t launch_mx_quantize(const void *X, int type, uint8_t *W, int64_t R, int64_t K, const DeviceInfo &dev,
                               cudaStream_t s) {
    const int64_t kt = mx_k_tiles(K);
    if (type == Q4_TYPE_F32) return quantize<float, 2>(X, W, R, K, kt, s);
    if (eight_rows(type, R, kt, dev))
        return type == Q4_TYPE_BF16 ? quantize<__nv_bfloat16, 8>(X, W, R, K, kt, s) : quantize<__half, 8>(X, W, R, K, kt, s);
    return type == Q4_TYPE_BF16 ? quantize<__nv_bfloat16, 2>(X, W, R, K, kt, s) : quantize<__half, 2>(X, W, R, K, kt, s);
}

cudaError_t launch_mx_dequant(const uint8_t *W, void *out, int type, int64_t R, int64_t K, const DeviceInfo &dev,
                              cudaStream_t s) {
    const int64_t kt = mx_k_tiles(K);
    if (type == Q4_TYPE_F32) return dequant<float, 2>(W, out, R, K, kt, s);
    if (eight_rows(type, R, kt, dev))
        return type == Q4_TYPE_BF16 ? dequant<__nv_bfloat16, 8>(W, out, R, K, kt, s) : dequant<__half, 8>(W, out, R, K, kt, s);
    return type == Q4_TYPE_BF16 ? dequant<__nv_bfloat16, 2>(W, out, R, K, kt, s) : dequant<__half, 2>(W, out, R, K, kt, s);
}

cudaError_t launch_mx_pack(const uint8_t *codes, const uint8_t *scales, uint8_t *W, int64_t R, int64_t K, cudaStream_t s) {
    const int64_t kt = mx_k_tiles(K);
    return launch_dependent(mx_pack_kernel<2>, grid_for(R, kt, 2), 32 * kWarps, s, codes, scales, W, R, K, static_cast<int>(kt));
}

}  // namespace q4
