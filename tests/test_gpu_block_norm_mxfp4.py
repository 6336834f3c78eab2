"""The block norm's MXFP4 output from every instance of its two kernels: equal
to the quantized fp32 output, and nothing written behind the matrix."""
import numpy as np
import pytest
import torch

from tests import mxfp4_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q4():
    import bit_weight_only_matmul_b200 as q4
    return q4


# many rows with one, two and four groups a thread, of 256 and of 512 threads, and rows of
# which the last turn of the warps has something to do for some only; few rows alike
@pytest.mark.parametrize("M,D", [(200, 96), (300, 1024), (150, 1056), (200, 6176), (200, 6432), (200, 8192), (200, 8224), (149, 9504),
                                 (200, 16384), (160, 16416), (3, 4096), (2, 6432), (5, 8224), (129, 16160), (2, 20000)])
@pytest.mark.parametrize("y", [torch.float32, torch.bfloat16, None])
def test_every_instance(q4, M, D, y):
    g = torch.Generator(device="cuda").manual_seed(M * 3 + D)
    r, pre = torch.randn((M, D), generator=g, device="cuda"), torch.randn((D,), generator=g, device="cuda")
    kw = dict(pre_weight=pre)
    if y is not None:
        kw.update(y=torch.randn((M, D), generator=g, device="cuda").to(y), post_weight=pre.flip(0).contiguous(), scale=0.5)
    x = torch.empty((M, D), device="cuda")
    n = q4.mxfp4_bytes(M, D)
    matrix = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    q4.q4_0_block_norm(r, M, D, x=x, **kw)
    q4.q4_0_block_norm(r, M, D, x=matrix[:n], **kw)
    want, known = ref.layout(*ref.quantize(x.double().cpu().numpy()))
    got = matrix.cpu().numpy()
    assert np.array_equal(got[:n][known], want[known])
    assert (got[:n][~known] == 0xA5).all() and (got[n:] == 0xA5).all()
    _, wx = ref.block_norm(r.double().cpu().numpy(), None if y is None else kw["y"].double().cpu().numpy(),
                           None if y is None else kw["post_weight"].double().cpu().numpy(), scale=0.5, pre=pre.double().cpu().numpy())
    # a sum of D <= 32768 squares within 69 * 2^-24 of itself (32 + 5 + 5 steps one after another,
    # each lane's and each line's), its root half of that, twice; ten roundings more: under 2^-17
    # of the larger of the value and what cancelled in it
    size = np.abs(wx) + 8.0 * np.abs(pre.double().cpu().numpy())
    assert np.all(np.abs(x.double().cpu().numpy() - wx) <= 2.0 ** -17 * size)


@pytest.mark.parametrize("M", [2, 200])
def test_squares_that_fp32_does_not_hold(q4, M):
    """As the header says: sums of squares above 3.4e38 give a norm of zeros,
    and with eps == 0 squares below 7e-46 = 2^-150 one of infinities."""
    D = 512
    big, small = torch.full((M, D), 1e18, device="cuda"), torch.full((M, D), 2.0 ** -76, device="cuda")
    for r, eps, want in ((big, 1e-6, 0.0), (big, 0.0, 0.0), (small, 0.0, float("inf")), (0.5 * big, 1e-6, 1.0)):
        x = torch.full((M, D), float("nan"), device="cuda")
        q4.q4_0_block_norm(r, M, D, x=x, eps=eps)
        assert torch.allclose(x, torch.full_like(x, want), rtol=2.0 ** -20, atol=0), (eps, want, x[0, :4])
