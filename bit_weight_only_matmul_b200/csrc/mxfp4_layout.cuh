// mxfp4_layout.cuh -- the MXFP4 matrix in memory, and the conversion of
// values to it, shared by the kernels that write it (quantize, pack, block
// norm) and those that read it (dequant, product).
//
// An MXFP4 matrix of R rows by K values is cut into tiles of 128 rows x 256
// k, kept one after the other (k fastest).  A tile is 17408 bytes:
//   * 128 rows of 128 bytes of codes, two to a byte with the lower k in the
//     low bits; the 16-byte chunk of block b (32 values) of row r lies at
//     chunk b ^ (r & 7) of the row, the 128-byte swizzle in which the tensor
//     cores read a K-major operand from shared memory;
//   * two times 512 scale bytes (128 k each): the scale of row r, block b at
//     512 * (b / 4) + 16 * (r % 32) + 4 * (r / 32) + b % 4, the order in
//     which a copy from shared memory lays scales into tensor memory.
// So one contiguous copy brings a tile in the form the tensor cores take it
// in: the product of few rows needs no tensor map, and a stream of weights
// reads memory front to back.  Blocks past K in the last tile hold zero codes
// and a zero scale byte.  Rows past R are never written; the product copies
// some of them or all with the tile, and the rows and columns of the
// accumulator that they reach are never stored.
#pragma once

#include <cstdint>

#include "q4_0_internal.cuh"

namespace q4 {

constexpr int kMxTileRows = 128;
constexpr int kMxTileK = 256;
constexpr int kMxCodeBytes = kMxTileRows * kMxTileK / 2;      // 16384
constexpr int kMxTileBytes = kMxCodeBytes + 1024;             // 17408

constexpr int64_t mx_k_tiles(int64_t K) { return (K + kMxTileK - 1) / kMxTileK; }
constexpr int64_t mx_row_tiles(int64_t R) { return (R + kMxTileRows - 1) / kMxTileRows; }

}  // namespace q4

#ifdef __CUDACC__
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace q4dev {

// Byte offset in its tile of the codes of block b (0..7) of row r (0..127).
__device__ __forceinline__ int mx_code_offset(int r, int b) { return r * 128 + ((b ^ (r & 7)) << 4); }

// Byte offset in its tile of the scales of blocks 4g .. 4g+3 of row r.
__device__ __forceinline__ int mx_scale_offset(int r, int g) {
    return q4::kMxCodeBytes + 512 * g + 16 * (r & 31) + 4 * (r >> 5);
}

// Of a block whose largest magnitude has the bits `amax` (sign bit clear): its
// scale byte, E + 127 with E = floor(log2 amax) - 2, at least 0; 255 (NaN) with
// an infinity or a NaN.  The exponent field of amax is floor(log2 amax) + 127
// (0 for a subnormal, whose E is below the range).
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
    const uint32_t e = amax >> 23;
    return e == 255u ? 255u : max(e, 2u) - 2u;
}
// And 2^-E (for a block that is NaN any number).
__device__ __forceinline__ float mx_inverse_scale(uint32_t amax) { return __uint_as_float((256u - max(amax >> 23, 2u)) << 23); }

// 2^E of a scale byte; NaN for 255.
__device__ __forceinline__ float mx_scale(uint32_t byte) {
    return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23);
}

// Eight scaled values as E2M1 codes, value i in bits 4i .. 4i+3: to nearest,
// ties to the even code, magnitudes above 6 to 6.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n .reg .b8 b0, b1, b2, b3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
        " mov.b32 %0, {b0, b1, b2, b3};\n}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Four of them.
__device__ __forceinline__ uint32_t e2m1x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n .reg .b8 b0, b1;\n .reg .b16 h;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        " mov.b16 h, {b0, b1};\n"
        " cvt.u32.u16 %0, h;\n}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// The largest of three magnitudes; NaN if one is NaN.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// The bits of a magnitude, NaN among them above all numbers.
__device__ __forceinline__ uint32_t magnitude_bits(float a) { return __float_as_uint(a) & 0x7FFFFFFFu; }

// Four consecutive lanes hold a block, eight values each (lane & 3 the part):
// the lane's code word; `byte` is the block's scale byte in all four lanes.
// All 32 lanes of the warp take part.  Multiplying by a power of two is exact
// (what underflows is far below the smallest code's half), so the only
// rounding is the one to E2M1.
__device__ __forceinline__ uint32_t mx_encode8(const float (&v)[8], uint32_t &byte) {
    uint32_t a = magnitude_bits(max_abs(max_abs(v[0], v[1], v[2]), max_abs(v[3], v[4], v[5]), max_abs(v[6], v[7], v[7])));
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
    byte = mx_scale_byte(a);
    const float inv = mx_inverse_scale(a);
    float s[8];
    #pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = v[i] * inv;
    return e2m1x8(s);
}

// Eight values as they lie in memory.
template <class T> struct Raw8;
template <> struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const void *p, int64_t at) {
        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
        a = __ldcs(q);
        b = __ldcs(q + 1);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};
template <> struct Raw8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const void *p, int64_t at) {
        a = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + at));
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};
template <> struct Raw8<__half> {
    uint4 a;
    __device__ __forceinline__ void load(const void *p, int64_t at) {
        a = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const __half *>(p) + at));
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
};

}  // namespace q4dev
#endif
