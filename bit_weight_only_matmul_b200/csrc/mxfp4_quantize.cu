// mxfp4_quantize.cu -- values to an MXFP4 matrix and back, and an MXFP4
// checkpoint's codes and scales into the library's layout.  All three are one
// pass over memory.
//
// A warp takes one row of a tile (256 k, 8 values a lane, four lanes a block):
// it reads 512 or 1024 contiguous bytes, finds each block's largest magnitude
// with two shuffles, and writes the row's 128 bytes of codes as one line and
// its eight scale bytes as two words.
#include "mxfp4_layout.cuh"

namespace {

using namespace q4dev;
using q4::kMxTileBytes;

template <typename T>
__global__ void mx_quantize_kernel(const T *__restrict__ X, uint8_t *__restrict__ W, int64_t R, int64_t K, int64_t kt) {
    const int lane = threadIdx.x & 31;
    const int64_t warp0 = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5;
    const int64_t warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    for (int64_t u = warp0; u < R * kt; u += warps) {
        const int64_t row = u / kt, t = u - row * kt, k = t * 256 + 8 * lane;
        float v[8] = {};
        if (k < K) load8(X + row * K + k, v);
        uint32_t byte;
        const uint32_t code = mx_encode8(v, byte);
        const uint32_t word = mx_scale_word(k < K ? byte : 0u, lane);
        uint8_t *tile = W + ((row >> 7) * kt + t) * kMxTileBytes;
        const int r = static_cast<int>(row & 127);
        *reinterpret_cast<uint32_t *>(tile + mx_code_offset(r, lane >> 2) + 4 * (lane & 3)) = code;
        if ((lane & 15) == 0) *reinterpret_cast<uint32_t *>(tile + mx_scale_offset(r, lane >> 4)) = word;
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

template <typename T>
__global__ void mx_dequant_kernel(const uint8_t *__restrict__ W, T *__restrict__ out, int64_t R, int64_t K, int64_t kt) {
    const int lane = threadIdx.x & 31;
    const int64_t warp0 = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5;
    const int64_t warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    for (int64_t u = warp0; u < R * kt; u += warps) {
        const int64_t row = u / kt, t = u - row * kt, k = t * 256 + 8 * lane;
        if (k >= K) continue;
        const uint8_t *tile = W + ((row >> 7) * kt + t) * kMxTileBytes;
        const int r = static_cast<int>(row & 127), b = lane >> 2;
        const uint32_t code = __ldg(reinterpret_cast<const uint32_t *>(tile + mx_code_offset(r, b) + 4 * (lane & 3)));
        const float s = mx_scale(__ldg(tile + mx_scale_offset(r, b >> 2) + (b & 3)));
        float v[8];
        #pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = e2m1_value(code >> (4 * i)) * s;
        store8(out + row * K + k, v);
    }
}

__global__ void mx_pack_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                               uint8_t *__restrict__ W, int64_t R, int64_t K, int64_t kt) {
    const int lane = threadIdx.x & 31;
    const int64_t warp0 = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5;
    const int64_t warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    for (int64_t u = warp0; u < R * kt; u += warps) {
        const int64_t row = u / kt, t = u - row * kt, k = t * 256 + 8 * lane;
        const bool live = k < K;
        const uint32_t code = live ? __ldcs(reinterpret_cast<const uint32_t *>(codes + (row * K + k) / 2)) : 0u;
        const uint32_t word = mx_scale_word(live ? scales[(row * K + k) / 32] : 0u, lane);
        uint8_t *tile = W + ((row >> 7) * kt + t) * kMxTileBytes;
        const int r = static_cast<int>(row & 127);
        *reinterpret_cast<uint32_t *>(tile + mx_code_offset(r, lane >> 2) + 4 * (lane & 3)) = code;
        if ((lane & 15) == 0) *reinterpret_cast<uint32_t *>(tile + mx_scale_offset(r, lane >> 4)) = word;
    }
}

int grid_for(int64_t warps_needed, int sm_count) {
    const int64_t ctas = (warps_needed + 7) / 8;
    const int64_t cap = static_cast<int64_t>(sm_count) * 16;
    return static_cast<int>(ctas < 1 ? 1 : (ctas < cap ? ctas : cap));
}

}  // namespace

namespace q4 {

cudaError_t launch_mx_quantize(const void *X, int type, uint8_t *W, int64_t R, int64_t K, const DeviceInfo &dev,
                               cudaStream_t s) {
    const int64_t kt = mx_k_tiles(K);
    const int grid = grid_for(R * kt, dev.sm_count);
    if (type == Q4_TYPE_F32)
        mx_quantize_kernel<<<grid, 256, 0, s>>>(static_cast<const float *>(X), W, R, K, kt);
    else if (type == Q4_TYPE_BF16)
        mx_quantize_kernel<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16 *>(X), W, R, K, kt);
    else
        mx_quantize_kernel<<<grid, 256, 0, s>>>(static_cast<const __half *>(X), W, R, K, kt);
    return cudaGetLastError();
}

cudaError_t launch_mx_dequant(const uint8_t *W, void *out, int type, int64_t R, int64_t K, const DeviceInfo &dev,
                              cudaStream_t s) {
    const int64_t kt = mx_k_tiles(K);
    const int grid = grid_for(R * kt, dev.sm_count);
    if (type == Q4_TYPE_F32)
        mx_dequant_kernel<<<grid, 256, 0, s>>>(W, static_cast<float *>(out), R, K, kt);
    else if (type == Q4_TYPE_BF16)
        mx_dequant_kernel<<<grid, 256, 0, s>>>(W, static_cast<__nv_bfloat16 *>(out), R, K, kt);
    else
        mx_dequant_kernel<<<grid, 256, 0, s>>>(W, static_cast<__half *>(out), R, K, kt);
    return cudaGetLastError();
}

cudaError_t launch_mx_pack(const uint8_t *codes, const uint8_t *scales, uint8_t *W, int64_t R, int64_t K,
                           const DeviceInfo &dev, cudaStream_t s) {
    const int64_t kt = mx_k_tiles(K);
    mx_pack_kernel<<<grid_for(R * kt, dev.sm_count), 256, 0, s>>>(codes, scales, W, R, K, kt);
    return cudaGetLastError();
}

}  // namespace q4
