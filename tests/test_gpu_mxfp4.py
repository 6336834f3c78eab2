"""MXFP4 quantisation, packing, dequantisation (bit for bit) and the product
(against the 64-bit product of the same values) on the GPU."""
import numpy as np
import pytest
import torch

from tests import mxfp4_reference as ref
from tests.gpu_helpers import no_device_error

pytestmark = pytest.mark.gpu
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def q4():
    import bit_weight_only_matmul_b200 as q4
    return q4


def _matrix(q4, R, K):
    """Room for an MXFP4 matrix, filled with a pattern that shows what was written."""
    return torch.full((q4.mxfp4_bytes(R, K),), 0xA5, dtype=torch.uint8, device="cuda")


def _check_bytes(W, codes, scales):
    want, known = ref.layout(codes, scales)
    got = W.cpu().numpy()
    assert np.array_equal(got[known], want[known])
    assert (got[~known] == 0xA5).all()      # rows past the last are left as they were


def _hard(rng, R, K):
    x = rng.standard_normal((R, K)) * np.exp2(rng.integers(-12, 12, (R, K // 32)).repeat(32, 1))
    q = np.exp2(np.floor(np.log2(np.abs(x).reshape(R, -1, 32).max(-1))) - 2).repeat(32, 1)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.5, 0.0])
    tie = rng.random((R, K)) < 0.3          # exact ties, zeros and values above 6
    x = np.where(tie & (np.arange(K) % 32 != 0), np.sign(x) * mids[rng.integers(0, 9, (R, K))] * q, x)
    x[:, 0] = np.where(rng.random(R) < 0.5, 0.0, x[:, 0])
    if R > 4:
        x[1, :32] = 0.0
        x[2, :32] = -0.0
        x[3, :32] *= 1e-30
        x[4, K - 32:] = 2.0 ** -140
    return x


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("R,K", [(1, 32), (1, 5120), (5, 288), (127, 256), (128, 512), (129, 800), (300, 1056)])
def test_quantize_bit_exact(q4, t, R, K):
    rng = np.random.default_rng(R * 31 + K)
    x = torch.from_numpy(_hard(rng, R, K)).to(DTYPES[t]).cuda()
    W = _matrix(q4, R, K)
    q4.mxfp4_quantize(x, W, R, K)
    codes, scales = ref.quantize(x.double().cpu().numpy())
    _check_bytes(W, codes, scales)
    for o in DTYPES.values():
        out = torch.full((R, K), float("nan"), dtype=o, device="cuda")
        q4.mxfp4_dequant(W, out, R, K)
        want = torch.from_numpy(ref.values(codes, scales)).to(o)
        assert torch.equal(out.cpu().view(torch.int16 if o != torch.float32 else torch.int32),
                           want.view(torch.int16 if o != torch.float32 else torch.int32))


def test_quantize_ends_of_the_range(q4):
    f = np.float32
    rows = [f(3.4028234663852886e38), f(2.0 ** 127), f(2.0 ** -126), f(2.0 ** -149), f(2.0 ** -125), f(1.1754942e-38)]
    x = np.zeros((len(rows) + 3, 64), f)
    for i, v in enumerate(rows):
        x[i, 7], x[i, 40] = v, -v
    x[-3, 3], x[-2, 3], x[-1, 3] = np.inf, -np.inf, np.nan     # the other block of these rows stays finite
    x[-3:, 5], x[-3:, 40] = 1.0, 1.0
    W = _matrix(q4, *x.shape)
    q4.mxfp4_quantize(torch.from_numpy(x).cuda(), W, *x.shape)
    codes, scales = ref.quantize(x)
    out = torch.empty(x.shape, device="cuda")
    q4.mxfp4_dequant(W, out, *x.shape)
    assert np.array_equal(out.cpu().numpy().astype(np.float64), ref.values(codes, scales), equal_nan=True)
    assert torch.isnan(out[-3:, :32]).all() and torch.isfinite(out[-3:, 32:]).all()


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16, torch.float16])
def test_dequant_of_every_code_and_scale(q4, t):
    codes = np.tile(np.arange(32, dtype=np.uint8) % 16, (256, 1))
    scales = np.arange(256, dtype=np.uint8)[:, None]
    W, out = _matrix(q4, 256, 32), torch.empty((256, 32), dtype=t, device="cuda")
    q4.mxfp4_pack(torch.from_numpy(ref.packed(codes)).cuda(), torch.from_numpy(scales).cuda(), W, 256, 32)
    q4.mxfp4_dequant(W, out, 256, 32)
    want = torch.from_numpy(ref.values(codes, scales)).to(t)
    got = out.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.isnan(got[255]).all()
    assert torch.equal(got[:255], want[:255])


@pytest.mark.parametrize("R,K", [(1, 32), (7, 96), (130, 288), (256, 512)])
def test_pack_bit_exact(q4, R, K):
    rng = np.random.default_rng(R + K)
    codes = rng.integers(0, 16, (R, K), dtype=np.uint8)
    scales = rng.integers(0, 256, (R, K // 32), dtype=np.uint8)
    W = _matrix(q4, R, K)
    q4.mxfp4_pack(torch.from_numpy(ref.packed(codes)).cuda(), torch.from_numpy(scales).cuda(), W, R, K)
    _check_bytes(W, codes, scales)


def _random_matrix(q4, rng, R, K, spread=6):
    codes = rng.integers(0, 16, (R, K), dtype=np.uint8)
    scales = rng.integers(127 - spread, 128 + spread, (R, K // 32), dtype=np.uint8)
    W = _matrix(q4, R, K)
    q4.mxfp4_pack(torch.from_numpy(ref.packed(codes)).cuda(), torch.from_numpy(scales).cuda(), W, R, K)
    return ref.values(codes, scales), W


def _check_product(Y, X, W, K, what=""):
    """The products are exact, so only the K - 1 additions round: each at most
    by 2^-23 of its partial sum (2^-24 for a rounding to nearest; a tensor core
    may truncate), and the partial sums are at most sum |x w|.  A bf16 result
    adds its own rounding, 2^-8 of the value at most."""
    exact, mag = X @ W.T, np.abs(X) @ np.abs(W).T
    bound = K * 2.0 ** -23 * mag
    got = Y.double().cpu().numpy()
    if Y.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (np.abs(exact) + bound)
    bad = ~(np.abs(got - exact) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[0], got[bad][0], exact[bad][0])


SHAPES = [(1, 1, 32), (1, 128, 256), (1, 5120, 1024), (2, 129, 288), (7, 300, 544), (8, 1000, 2048), (9, 128, 96),
          (31, 257, 1280), (32, 640, 4096), (33, 200, 512), (64, 128, 3200), (100, 391, 608), (127, 130, 256),
          (128, 256, 1056), (129, 256, 512), (200, 1024, 768), (255, 129, 352), (256, 512, 2304), (257, 300, 1024),
          (300, 77, 4128), (513, 1290, 640), (3, 16400, 512), (17, 128, 8192), (65, 700, 2560), (128, 1024, 4096),
          (16, 40000, 288), (90, 20000, 320), (1000, 2050, 1056), (2500, 2600, 320),
          (385, 5000, 2080), (1100, 2304, 512), (33, 1, 32), (48, 5200, 1024), (20, 2048, 8192),
          (127, 1000, 5120), (64, 5120, 5120), (72, 130, 8192), (113, 20000, 1056), (121, 257, 4096), (44, 5003, 8160),
          (33, 2304, 8192), (128, 2048, 5120), (3, 2100, 8192), (50, 300, 2048), (1, 4096, 4096), (2, 1000, 5120)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_gemm(q4, M, N, K, out):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    x, X = _random_matrix(q4, rng, M, K)
    w, W = _random_matrix(q4, rng, N, K)
    Y = torch.full((M * N + 64,), 7.0, dtype=DTYPES[out], device="cuda")
    q4.mxfp4_gemm(W, X, Y, M, N, K)
    _check_product(Y[:M * N].view(M, N), x, w, K, (M, N, K, out))
    assert (Y[M * N:] == 7.0).all()
    no_device_error(q4)


def test_gemm_every_row_and_block_has_its_own_scale(q4):
    """One non-zero weight and one non-zero activation at a time pick out each
    (row, block): a misplaced scale or code shows as a wrong power of two."""
    for M, N, K in ((256, 256, 512), (8, 128, 512)):
        cw = np.full((N, K), 2, np.uint8)           # all ones
        cx = np.zeros((M, K), np.uint8)
        m = np.arange(M)
        cx[m, (m * 37) % K] = 2                     # a one at a place of its own in each row
        sw = (100 + (np.arange(N)[:, None] * 5 + np.arange(K // 32)[None] * 3) % 50).astype(np.uint8)
        sx = (100 + (np.arange(M)[:, None] * 7 + np.arange(K // 32)[None] * 11) % 50).astype(np.uint8)
        mats = []
        for c, s in ((cw, sw), (cx, sx)):
            B = _matrix(q4, *c.shape)
            q4.mxfp4_pack(torch.from_numpy(ref.packed(c)).cuda(), torch.from_numpy(s).cuda(), B, *c.shape)
            mats.append(B)
        Y = torch.empty((M, N), device="cuda")
        q4.mxfp4_gemm(mats[0], mats[1], Y, M, N, K)
        want = ref.values(cx, sx) @ ref.values(cw, sw).T
        assert np.array_equal(Y.cpu().numpy().astype(np.float64), want)


def test_gemm_nan_block_marks_its_row_and_column_only(q4):
    rng = np.random.default_rng(5)
    M, N, K = 40, 200, 768
    mats = []
    for R, bad in ((N, 150), (M, 11)):
        codes = rng.integers(0, 16, (R, K), dtype=np.uint8)
        scales = rng.integers(120, 134, (R, K // 32), dtype=np.uint8)
        scales[bad, 5] = 255
        B = _matrix(q4, R, K)
        q4.mxfp4_pack(torch.from_numpy(ref.packed(codes)).cuda(), torch.from_numpy(scales).cuda(), B, R, K)
        mats.append(B)
    Y = torch.empty((M, N), device="cuda")
    q4.mxfp4_gemm(mats[0], mats[1], Y, M, N, K)
    nan = torch.isnan(Y).cpu().numpy()
    want = np.zeros((M, N), bool)
    want[11], want[:, 150] = True, True
    assert np.array_equal(nan, want)


@pytest.mark.parametrize("M", [17, 40, 255])
@pytest.mark.parametrize("cx,cw", [(1, 1), (1, 7), (7, 2)])
def test_gemm_over_the_whole_range_of_scales(q4, M, cx, cw):
    """One product a sum, of all pairs of scales 2^-127 .. 2^127: exact wherever
    fp32 has the number as a normal one, infinite above."""
    K, w_exp = 64, np.arange(255)
    x_exp = w_exp[:: 255 // M][:M]

    def matrix(exps, code):
        codes = np.zeros((len(exps), K), np.uint8)
        scales = np.full((len(exps), 2), 127, np.uint8)
        codes[:, 5], scales[:, 0] = code, exps
        B = _matrix(q4, len(exps), K)
        q4.mxfp4_pack(torch.from_numpy(ref.packed(codes)).cuda(), torch.from_numpy(scales).cuda(), B, len(exps), K)
        return B
    W, X = matrix(w_exp, cw), matrix(x_exp, cx)
    Y = torch.empty((M, 255), device="cuda")
    q4.mxfp4_gemm(W, X, Y, M, 255, K)
    value = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    want = value[cx] * value[cw] * np.exp2(x_exp[:, None] - 127.0) * np.exp2(w_exp[None, :] - 127.0)
    got = Y.double().cpu().numpy()
    normal, above = (want >= 2.0 ** -126) & (want < 2.0 ** 128), want >= 2.0 ** 128
    assert np.array_equal(got[normal], want[normal])
    assert np.isposinf(got[above]).all()
    assert (got[want < 2.0 ** -126] < 2.0 ** -126).all()


@pytest.mark.parametrize("M,N,K", [(3, 70, 288), (33, 200, 544), (130, 300, 1056), (300, 40, 288)])
def test_gemm_does_not_look_at_rows_past_the_last(q4, M, N, K):
    """Memory behind the last rows may hold anything: NaN scales here, and no
    row or column of the result knows of them."""
    rng = np.random.default_rng(M)
    mats = []
    for R in (N, M):
        codes = rng.integers(0, 16, (R, K), dtype=np.uint8)
        scales = rng.integers(121, 133, (R, K // 32), dtype=np.uint8)
        B = torch.full((q4.mxfp4_bytes(R, K),), 0xFF, dtype=torch.uint8, device="cuda")
        q4.mxfp4_pack(torch.from_numpy(ref.packed(codes)).cuda(), torch.from_numpy(scales).cuda(), B, R, K)
        mats.append((ref.values(codes, scales), B))
    Y = torch.empty((M, N), device="cuda")
    q4.mxfp4_gemm(mats[0][1], mats[1][1], Y, M, N, K)
    _check_product(Y, mats[1][0], mats[0][0], K)


def test_gemm_on_the_first_rows_of_a_larger_matrix(q4):
    rng = np.random.default_rng(8)
    x, X = _random_matrix(q4, rng, 300, 512)
    w, W = _random_matrix(q4, rng, 200, 512)
    for M, N in ((1, 200), (130, 129), (299, 1)):
        Y = torch.empty((M, N), device="cuda")
        q4.mxfp4_gemm(W, X, Y, M, N, 512)
        _check_product(Y, x[:M], w[:N], 512)


def test_gemm_of_nothing(q4):
    W = torch.empty(0, dtype=torch.uint8, device="cuda")
    Y = torch.full((3, 5), 7.0, device="cuda")
    q4.mxfp4_gemm(W, W, Y, 3, 5, 0)
    assert (Y == 0).all()
    q4.mxfp4_gemm(W, W, Y, 0, 5, 0)


def test_binding_refusals(q4):
    R, K = 4, 64
    x = torch.zeros((R, K), device="cuda")
    W = _matrix(q4, R, K)
    with pytest.raises(ValueError, match="dtype"):
        q4.mxfp4_quantize(x.double(), W, R, K)
    with pytest.raises(ValueError, match="elements"):
        q4.mxfp4_quantize(x, W, R + 1, K)
    with pytest.raises(ValueError, match="elements"):
        q4.mxfp4_quantize(x, W[:100], R, K)
    with pytest.raises(ValueError, match="contiguous"):
        q4.mxfp4_quantize(torch.zeros((R, 2 * K), device="cuda")[:, :K], W, R, K)
    with pytest.raises(ValueError, match="dtype"):
        q4.mxfp4_gemm(W, W, x.half(), R, R, K)
    with pytest.raises(q4.Q4Error):
        q4.mxfp4_quantize(x, W, 2, 40)
    with pytest.raises(ValueError, match="dtype"):
        q4.q4_0_block_norm(x, R, K, r_out=x.bfloat16())


def test_binding_refuses_tensors_without_plain_storage(q4):
    from torch._subclasses.fake_tensor import FakeTensorMode
    R, K = 4, 64
    x = torch.ones((R, K), device="cuda")
    W = _matrix(q4, R, K)
    with FakeTensorMode():
        fake = torch.empty((R, K), device="cuda")
    for bad in (x.to_sparse(), torch.nested.nested_tensor([x, x]), fake):
        for call in (lambda: q4.mxfp4_quantize(bad, W, R, K), lambda: q4.mxfp4_dequant(W, bad, R, K),
                     lambda: q4.mxfp4_gemm(W, W, bad, R, R, K), lambda: q4.q4_0_block_norm(bad, R, K, x=x),
                     lambda: q4.q4_0_block_norm(x, R, K, x=bad)):
            with pytest.raises((ValueError, RuntimeError)):
                call()
    assert torch.equal(x, torch.ones_like(x))
