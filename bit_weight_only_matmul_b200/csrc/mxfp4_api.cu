// mxfp4_api.cu -- the C ABI of the MXFP4 operators (include/mxfp4.h) and of
// the block norm (include/q4_0.h): argument checks, then one launch.
#include <cmath>

#include "../../include/mxfp4.h"
#include "mxfp4_layout.cuh"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_dims(int64_t R, int64_t K) {
    if (R < 0 || K < 0 || R > Q4_0_MAX_DIM || K > Q4_0_MAX_DIM || K % 32 != 0) return Q4_ERR_INVALID_ARG;
    return Q4_OK;
}

bool value_type(int t) { return t == Q4_TYPE_F32 || t == Q4_TYPE_BF16 || t == Q4_TYPE_F16; }

int done(cudaError_t e) { return e == cudaSuccess ? Q4_OK : q4::api_cuda_fail(e); }

}  // namespace

extern "C" {

int64_t mxfp4_bytes(int64_t R, int64_t K) {
    if (check_dims(R, K) != Q4_OK) return -1;
    return q4::mx_row_tiles(R) * q4::mx_k_tiles(K) * q4::kMxTileBytes;
}

int mxfp4_quantize(const void *X, int x_type, void *W, int64_t R, int64_t K, q4_0_stream_t stream) {
    int st = check_dims(R, K);
    if (st != Q4_OK) return st;
    if (!value_type(x_type)) return Q4_ERR_INVALID_ARG;
    if (R == 0 || K == 0) return Q4_OK;
    if (!X || !W) return Q4_ERR_INVALID_ARG;
    if (!aligned16(X) || !aligned16(W)) return Q4_ERR_MISALIGNED;
    const q4::DeviceInfo *dev = nullptr;
    st = q4::api_device(&dev);
    if (st != Q4_OK) return st;
    return done(q4::launch_mx_quantize(X, x_type, static_cast<uint8_t *>(W), R, K, *dev,
                                       reinterpret_cast<cudaStream_t>(stream)));
}

int mxfp4_dequant(const void *W, void *out, int out_type, int64_t R, int64_t K, q4_0_stream_t stream) {
    int st = check_dims(R, K);
    if (st != Q4_OK) return st;
    if (!value_type(out_type)) return Q4_ERR_INVALID_ARG;
    if (R == 0 || K == 0) return Q4_OK;
    if (!W || !out) return Q4_ERR_INVALID_ARG;
    if (!aligned16(W) || !aligned16(out)) return Q4_ERR_MISALIGNED;
    const q4::DeviceInfo *dev = nullptr;
    st = q4::api_device(&dev);
    if (st != Q4_OK) return st;
    return done(q4::launch_mx_dequant(static_cast<const uint8_t *>(W), out, out_type, R, K, *dev,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

int mxfp4_pack(const uint8_t *codes, const uint8_t *scales, void *W, int64_t R, int64_t K, q4_0_stream_t stream) {
    int st = check_dims(R, K);
    if (st != Q4_OK) return st;
    if (R == 0 || K == 0) return Q4_OK;
    if (!codes || !scales || !W) return Q4_ERR_INVALID_ARG;
    if (!aligned16(codes) || !aligned16(scales) || !aligned16(W)) return Q4_ERR_MISALIGNED;
    const q4::DeviceInfo *dev = nullptr;
    st = q4::api_device(&dev);
    if (st != Q4_OK) return st;
    return done(q4::launch_mx_pack(codes, scales, static_cast<uint8_t *>(W), R, K,
                                   reinterpret_cast<cudaStream_t>(stream)));
}

int mxfp4_gemm(const void *W, const void *X, void *Y, int y_type, int64_t M, int64_t N, int64_t K, q4_0_stream_t stream) {
    if (M < 0 || M > Q4_0_MAX_DIM) return Q4_ERR_INVALID_ARG;
    int st = check_dims(N, K);
    if (st != Q4_OK) return st;
    if (y_type != Q4_TYPE_F32 && y_type != Q4_TYPE_BF16) return Q4_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return Q4_OK;
    if (!Y) return Q4_ERR_INVALID_ARG;
    if (!aligned16(Y)) return Q4_ERR_MISALIGNED;
    if (K != 0) {
        if (!W || !X) return Q4_ERR_INVALID_ARG;
        if (!aligned16(W) || !aligned16(X)) return Q4_ERR_MISALIGNED;
    }
    const q4::DeviceInfo *dev = nullptr;
    st = q4::api_device(&dev);
    if (st != Q4_OK) return st;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (K == 0) return done(cudaMemsetAsync(Y, 0, static_cast<size_t>(M) * N * (y_type == Q4_TYPE_F32 ? 4 : 2), s));
    return done(q4::launch_mx_gemm(static_cast<const uint8_t *>(W), static_cast<const uint8_t *>(X), Y, y_type, M, N, K,
                                   *dev, s));
}

int q4_0_block_norm(const q4_0_block *b, q4_0_stream_t stream) {
    if (!b) return Q4_ERR_INVALID_ARG;
    if (b->M < 0 || b->M > Q4_0_MAX_DIM || b->D < 0 || b->D > Q4_0_MAX_NORM_DIM || b->D % 32 != 0) return Q4_ERR_INVALID_ARG;
    if (b->r_type != Q4_TYPE_F32 && b->r_type != Q4_TYPE_BF16) return Q4_ERR_INVALID_ARG;
    if (b->y && b->y_type != Q4_TYPE_F32 && b->y_type != Q4_TYPE_BF16) return Q4_ERR_INVALID_ARG;
    if (b->x && b->x_type != Q4_TYPE_F32 && b->x_type != Q4_TYPE_BF16 && b->x_type != Q4_TYPE_MXFP4) return Q4_ERR_INVALID_ARG;
    if (!(b->eps >= 0.0f) || std::isinf(b->eps) || b->gate_span < 0) return Q4_ERR_INVALID_ARG;
    if (!b->y && (b->post_weight || b->gate)) return Q4_ERR_INVALID_ARG;
    if (!b->x && b->pre_weight) return Q4_ERR_INVALID_ARG;
    if (b->M == 0 || b->D == 0) return Q4_OK;
    if (!b->r || (!b->x && !b->r_out)) return Q4_ERR_INVALID_ARG;
    const void *all[] = {b->y, b->r, b->r_out, b->x, b->post_weight, b->gate, b->pre_weight};
    for (const void *p : all)
        if (!aligned16(p)) return Q4_ERR_MISALIGNED;
    const q4::DeviceInfo *dev = nullptr;
    const int st = q4::api_device(&dev);
    if (st != Q4_OK) return st;
    return done(q4::launch_block_norm(*b, *dev, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
