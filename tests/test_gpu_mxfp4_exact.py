"""The MXFP4 product where it is exact: any misplaced code, scale, row, column
or part of K shows as another number, on every way the product works."""
import numpy as np
import pytest
import torch

from tests import mxfp4_exact as exact
from tests import mxfp4_reference as ref
from tests.gpu_helpers import no_device_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q4():
    import bit_weight_only_matmul_b200 as q4
    return q4


def _matrix(q4, codes, scales):
    """The MXFP4 matrix, NaN scales and codes in the rows behind the last."""
    W = torch.full((q4.mxfp4_bytes(*codes.shape),), 0xFF, dtype=torch.uint8, device="cuda")
    q4.mxfp4_pack(*exact.on_gpu(codes, scales), W, *codes.shape)
    return W


@pytest.mark.parametrize("M,N,K,what", exact.CASES)
def test_product_is_exact(q4, M, N, K, what):
    w, x, want = exact.case(M, N, K)
    W, X = _matrix(q4, *w), _matrix(q4, *x)
    for t in (torch.float32, torch.bfloat16):
        Y = torch.full((M * N + 64,), 7.0, dtype=t, device="cuda")
        q4.mxfp4_gemm(W, X, Y, M, N, K)
        assert exact.same(Y[:M * N].view(M, N), want), (what, t)
        assert (Y[M * N:] == 7.0).all()
    no_device_error(q4)


@pytest.mark.parametrize("M,N,K,what", [c for c in exact.CASES if c[0] > 1 and c[1] > 1])
def test_nan_blocks_mark_their_rows_and_columns_only(q4, M, N, K, what):
    w, x, want = exact.case(M, N, K, nan=True)
    W, X = _matrix(q4, *w), _matrix(q4, *x)
    Y = torch.empty((M, N), device="cuda")
    q4.mxfp4_gemm(W, X, Y, M, N, K)
    assert exact.same(Y, want), what


@pytest.mark.parametrize("M,N,K", [(2, 130, 3104), (30, 100, 2080), (20, 2500, 1056), (300, 77, 1056), (1850, 1100, 288)])
def test_scales_far_apart_in_a_row(q4, M, N, K):
    """Blocks of one row 2^50 apart: each of the K products is aligned to the
    largest of its sum, and so off by 2^-23 of that at most, and each of the
    partial sums joined, fewer than K / 32 of them, by 2^-23 of itself."""
    rng = np.random.default_rng(M + N)
    mats = []
    for R in (N, M):
        codes = rng.integers(0, 16, (R, K), dtype=np.uint8)
        scales = rng.integers(102, 153, (R, K // 32), dtype=np.uint8)
        mats.append((_matrix(q4, codes, scales), ref.values(codes, scales)))
    (W, w), (X, x) = mats
    Y = torch.empty((M, N), device="cuda")
    q4.mxfp4_gemm(W, X, Y, M, N, K)
    assert np.all(np.abs(Y.double().cpu().numpy() - x @ w.T) <= (K + K / 32) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T))
