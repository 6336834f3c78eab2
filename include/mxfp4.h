/*
 * mxfp4.h -- C ABI of the MXFP4 operators of libq4_0_b200.so: the microscaled
 * 4-bit floating-point format, quantized to, packed, dequantized and
 * multiplied on the block-scaled tensor cores of sm_100a.  Conventions (device
 * pointers, streams, checks, status codes, devices) are those of q4_0.h.
 *
 * The format (OCP microscaling, MXFP4).  A row is cut into blocks of 32 values
 * along K.  A value is an E2M1 number c (0, 0.5, 1, 1.5, 2, 3, 4 or 6 and a
 * sign; codes 0..7, sign in bit 3) times its block's scale 2^E, kept as the
 * byte E + 127 (E8M0); byte 255 makes the whole block NaN.
 *
 * An MXFP4 matrix of R rows by K values is one buffer of mxfp4_bytes(R, K)
 * bytes, in tiles of 128 rows x 256 k, k fastest; a tile is 17408 bytes:
 *   - 128 rows of 128 bytes of codes, two to a byte, the lower k in the low
 *     bits; block b (0..7) of row r at byte 128*r + 16*(b ^ (r & 7));
 *   - from byte 16384 the scales: block b of row r at byte
 *     16384 + 512*(b/4) + 16*(r%32) + 4*(r/32) + b%4.
 * Blocks past K in the last tile hold zero codes and zero scale bytes (every
 * function here writes them so, and mxfp4_gemm relies on it).  Rows past R are
 * never written and may hold anything, no result depends on them; but
 * mxfp4_gemm copies whole tiles and reads them too, so that all mxfp4_bytes()
 * bytes have to be there.
 */
#ifndef MXFP4_B200_H
#define MXFP4_B200_H

#include "q4_0.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of an MXFP4 matrix of R rows by K values; -1 for invalid sizes
 * (negative, above Q4_0_MAX_DIM, K % 32 != 0). */
Q4_0_API int64_t mxfp4_bytes(int64_t R, int64_t K);

/* X [R,K] (row-major; fp32, bf16 or fp16: x_type) to MXFP4: per block
 * E = floor(log2 a) - 2 for the largest magnitude a, at least -127 (a block
 * of zeros: -127); codes x * 2^-E to the nearest E2M1 number, ties to the
 * even code, magnitudes above 6 to 6.  A block that holds an infinity or a
 * NaN gets scale byte 255.  Deterministic and bit-exact.  X and W 16-byte
 * aligned and not overlapping, K % 32 == 0; R == 0 or K == 0 writes nothing. */
Q4_0_API int mxfp4_quantize(const void *X, int x_type, void *W, int64_t R, int64_t K, q4_0_stream_t stream);

/* The values an MXFP4 matrix stands for, out [R,K] row-major in fp32, bf16 or
 * fp16 (out_type).  Exact in fp32 and bf16 (a code has two significant bits
 * and the exponents fit, but for codes from 2 on at the largest scales, above
 * the type's range: infinity); rounded once, to nearest even, in fp16.
 * W and out 16-byte aligned and not overlapping. */
Q4_0_API int mxfp4_dequant(const void *W, void *out, int out_type, int64_t R, int64_t K, q4_0_stream_t stream);

/* Codes and scales as checkpoints hold them into the layout above (bit-exact):
 *   codes  [R,K/2] uint8 row-major, two codes to a byte, the lower k in the
 *          low bits;
 *   scales [R,K/32] uint8 row-major, E + 127 (255: NaN).
 * All pointers 16-byte aligned, W overlapping neither of the others; R == 0 or
 * K == 0 writes nothing. */
Q4_0_API int mxfp4_pack(const uint8_t *codes, const uint8_t *scales, void *W, int64_t R, int64_t K, q4_0_stream_t stream);

/* Y[M,N] = X[M,K] * W[N,K]^T of two MXFP4 matrices, Y row-major in fp32 or
 * bf16 (y_type), overwritten.  Products are exact within fp32's normal range
 * and sums fp32; a bf16 Y is rounded once.  The same inputs give the same
 * bits.  W, X, Y 16-byte aligned, Y not overlapping W or X; K % 32 == 0.
 * M == 0 or N == 0 does nothing; K == 0 fills Y with zeros.  A NaN block makes
 * its row (of X) or column (of W) of Y NaN. */
Q4_0_API int mxfp4_gemm(const void *W, const void *X, void *Y, int y_type, int64_t M, int64_t N, int64_t K,
                        q4_0_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_B200_H */
