"""The block norm on the GPU against its formula in 64 bits."""
import numpy as np
import pytest
import torch

from tests import mxfp4_reference as ref

pytestmark = pytest.mark.gpu
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def q4():
    import bit_weight_only_matmul_b200 as q4
    return q4


def _close(got, want, size, rounded):
    """`size`: the sum of the magnitudes that were added; fp32 arithmetic is
    within 2^-18 of it: a sum of D <= 32768 squares, added in at most 32 + 5 +
    5 steps one after another, is under 69 * 2^-24 off, its root half of that, and
    the products around it under ten roundings of 2^-24 more (two sums in x:
    under 2^-17.6 in all, so 2^-17).  bf16 adds half a step, 2^-8."""
    tol = 2.0 ** -17 * size
    if rounded:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= tol + 1e-37)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0], got[bad][0], want[bad][0])


def _run(q4, M, D, y="f32", r="f32", x="bf16", post=True, gate=True, span=0, pre=True, scale=0.75, eps=1e-6, in_place=False,
         seed=0, amplitude=1.0):
    g = np.random.default_rng(seed + M * 5 + D)
    t = lambda a, k="f32": torch.from_numpy(np.ascontiguousarray(a)).to(DTYPES[k]).cuda()  # noqa: E731
    yd = t(amplitude * g.standard_normal((M, D)) * np.exp(g.standard_normal((M, 1))), y) if y else None
    rd = t(3 * g.standard_normal((M, D)), r)
    pd = t(1 + 0.2 * g.standard_normal(D)) if post else None
    gd = t(g.standard_normal((-(-M // span) if span else 1, D))) if gate else None
    wd = t(1 + 0.2 * g.standard_normal(D)) if pre else None
    host = lambda a: None if a is None else a.double().cpu().numpy()  # noqa: E731
    wr, wx = ref.block_norm(host(rd), host(yd), host(pd), host(gd), span, scale, host(wd), eps)
    size_h = np.abs(wr - host(rd)) + np.abs(host(rd))
    size_x = np.abs(wx) / np.maximum(np.abs(wr), 1e-300) * size_h + np.abs(wx)
    out = rd if in_place else torch.full_like(rd, float("nan"))
    xd = torch.full((M, D), float("nan"), dtype=DTYPES[x], device="cuda") if x else None
    q4.q4_0_block_norm(rd, M, D, y=yd, post_weight=pd, gate=gd, gate_span=span, scale=scale, pre_weight=wd, x=xd, r_out=out,
                       eps=eps)
    _close(out, wr, size_h, r == "bf16")
    if x:
        _close(xd, wx, size_x, x == "bf16")


@pytest.mark.parametrize("M,D", [(1, 32), (1, 5120), (2, 256), (3, 288), (5, 4128), (17, 8192), (3, 8224), (2, 16384),
                                 (3, 16416), (2, 32768), (300, 1024), (2000, 512), (10000, 96), (400, 4128),
                                 (450, 8192), (1200, 2080), (320, 16384)])
@pytest.mark.parametrize("y,r,x", [("f32", "f32", "bf16"), ("bf16", "bf16", "f32"), ("bf16", "f32", "bf16")])
def test_block_norm(q4, M, D, y, r, x):
    _run(q4, M, D, y, r, x)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate,span", [(False, 0), (True, 0), (True, 1), (True, 7), (True, 1000)])
@pytest.mark.parametrize("pre,x", [(True, "bf16"), (False, "f32"), (False, None)])
@pytest.mark.parametrize("M,D", [(20, 544), (700, 544), (400, 2336)])
def test_block_norm_parts(q4, post, gate, span, pre, x, M, D):
    _run(q4, M, D, post=post, gate=gate, span=span, pre=pre, x=x)


def test_block_norm_without_y_in_place_and_extremes(q4):
    _run(q4, 9, 1024, y=None, post=False, gate=False)
    _run(q4, 900, 1024, y=None, post=False, gate=False, r="bf16")
    _run(q4, 500, 4096, in_place=True, r="bf16", y="bf16")
    _run(q4, 300, 2048, in_place=True)
    _run(q4, 4, 512, in_place=True, r="bf16")
    _run(q4, 4, 512, scale=0.0)
    _run(q4, 4, 512, scale=-2.0, eps=0.0)
    _run(q4, 4, 512, amplitude=1e-15)
    _run(q4, 4, 512, amplitude=1e15)


def test_block_norm_zero_rows(q4):
    z = torch.zeros((3, 64), device="cuda")
    x = torch.full((3, 64), float("nan"), device="cuda")
    r2 = torch.full((3, 64), float("nan"), device="cuda")
    w = torch.ones(64, device="cuda")
    q4.q4_0_block_norm(z, 3, 64, y=z, post_weight=w, pre_weight=w, x=x, r_out=r2)
    assert (x == 0).all() and (r2 == 0).all()


def test_block_norm_keeps_bad_rows_to_themselves(q4):
    M, D = 5, 256
    y = torch.randn((M, D), device="cuda")
    r = torch.randn((M, D), device="cuda")
    y[2, 17] = float("nan")
    r[4, 3] = float("inf")
    x, r2 = torch.empty_like(r), torch.empty_like(r)
    w = torch.ones(D, device="cuda")
    q4.q4_0_block_norm(r, M, D, y=y, post_weight=w, pre_weight=w, x=x, r_out=r2)
    assert torch.isnan(x[2]).all() and torch.isnan(x[4, 3])
    assert torch.isfinite(x[[0, 1, 3]]).all() and torch.isfinite(r2[[0, 1, 3]]).all()


@pytest.mark.parametrize("M,D", [(1, 32), (1, 5120), (3, 288), (130, 1056), (500, 1056), (333, 5120), (2, 9000 // 32 * 32), (3, 16416), (2, 32768)])
def test_block_norm_to_mxfp4_is_the_quantized_fp32_norm(q4, M, D):
    """The MXFP4 output equals mxfp4_quantize of the fp32 output, bit for bit,
    and rows past M are left alone."""
    g = torch.Generator(device="cuda").manual_seed(M + D)
    y, r = (torch.randn((M, D), generator=g, device="cuda") for _ in range(2))
    post, pre, gate = (torch.randn((D,), generator=g, device="cuda") for _ in range(3))
    kw = dict(y=y, post_weight=post, gate=gate, pre_weight=pre, scale=0.5)
    x = torch.empty((M, D), device="cuda")
    a, b = (torch.full((q4.mxfp4_bytes(M, D),), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(2))
    q4.q4_0_block_norm(r, M, D, x=x, **kw)
    q4.mxfp4_quantize(x, a, M, D)
    q4.q4_0_block_norm(r, M, D, x=b, **kw)
    assert torch.equal(a, b)
    codes, scales = ref.quantize(x.double().cpu().numpy())
    want, known = ref.layout(codes, scales)
    assert np.array_equal(b.cpu().numpy()[known], want[known])
