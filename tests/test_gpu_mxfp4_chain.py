"""The MXFP4 operators and the block norm as a decoder uses them: one after the
other, on the Q4_0 product too, captured and replayed, on several streams and
threads, and over sizes whose offsets pass 32 bits."""
import threading

import numpy as np
import pytest
import torch

import oracle
import workloads
from tests import mxfp4_reference as ref
from tests.gpu_helpers import check_gemm, dev, no_device_error, pack_on_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q4():
    import bit_weight_only_matmul_b200 as q4
    return q4


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


class Block:
    """A residual block around one MXFP4 product: norm -> product -> norm / gate / residual -> next norm."""

    def __init__(self, q4, M, D, seed=0):
        g = _gen(seed)
        self.q4, self.M, self.D = q4, M, D
        self.r, self.pre, self.post, self.next = _randn(g, M, D), *(1 + 0.1 * _randn(g, D) for _ in range(3))
        self.gate = _randn(g, 1, D)
        self.W = torch.empty(q4.mxfp4_bytes(D, D), dtype=torch.uint8, device="cuda")
        q4.mxfp4_quantize(0.05 * _randn(g, D, D), self.W, D, D)
        self.X = torch.empty(q4.mxfp4_bytes(M, D), dtype=torch.uint8, device="cuda")
        self.Y = torch.empty((M, D), dtype=torch.bfloat16, device="cuda")
        self.r2, self.x2 = torch.empty((M, D), device="cuda"), torch.empty((M, D), dtype=torch.bfloat16, device="cuda")

    def run(self, stream=None):
        q4, M, D = self.q4, self.M, self.D
        q4.q4_0_block_norm(self.r, M, D, pre_weight=self.pre, x=self.X, stream=stream)
        q4.mxfp4_gemm(self.W, self.X, self.Y, M, D, D, stream=stream)
        q4.q4_0_block_norm(self.r, M, D, y=self.Y, post_weight=self.post, gate=self.gate, scale=0.5, pre_weight=self.next,
                           x=self.x2, r_out=self.r2, stream=stream)

    def out(self):
        return [t.clone() for t in (self.X, self.Y, self.r2, self.x2)]


@pytest.mark.parametrize("M,D", [(1, 1024), (5, 800), (32, 2048), (150, 1056), (700, 2048)])
def test_block(q4, M, D):
    """Each step against 64 bits, on what the step before it gave on the GPU."""
    b = Block(q4, M, D, seed=M)
    b.X.zero_()
    b.run()
    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    x, w = torch.empty((M, D), device="cuda"), torch.empty((D, D), device="cuda")
    q4.mxfp4_dequant(b.X, x, M, D)
    q4.mxfp4_dequant(b.W, w, D, D)
    _, wx = ref.block_norm(host(b.r), pre=host(b.pre))
    # a value lies within half a code's step of what it stands for: a quarter of
    # the value or of the block's unit, or up to the clamp from 8 to 6 units,
    # and the fp32 norm may round to the other side of a border
    unit = np.exp2(np.floor(np.log2(np.abs(wx).reshape(M, -1, 32).max(-1) * (1 + 2.0 ** -17))) - 2).repeat(32, 1)
    assert np.all(np.abs(host(x) - wx) <= np.maximum(2.0 * unit, 0.25 * np.abs(wx)) * (1 + 2.0 ** -16))
    exact, mag = host(x) @ host(w).T, np.abs(host(x)) @ np.abs(host(w)).T
    bound = D * 2.0 ** -23 * mag
    assert np.all(np.abs(host(b.Y) - exact) <= bound + 2.0 ** -8 * (np.abs(exact) + bound))
    r2, x2 = ref.block_norm(host(b.r), host(b.Y), host(b.post), host(b.gate), 0, 0.5, host(b.next))
    size = np.abs(r2 - host(b.r)) + np.abs(host(b.r))
    assert np.all(np.abs(host(b.r2) - r2) <= 2.0 ** -17 * size)
    size = np.abs(x2) * (1 + size / np.maximum(np.abs(r2), 1e-300))
    assert np.all(np.abs(host(b.x2) - x2) <= 2.0 ** -17 * size + 2.0 ** -8 * np.abs(x2) * (1 + 2.0 ** -7))
    no_device_error(q4)


def test_norm_feeds_the_q4_0_product(q4):
    M, K, N = 3, 1024, 300
    rng = np.random.default_rng(4)
    codes = rng.integers(0, 16, size=(N, K), dtype=np.uint8)
    scales = (np.abs(rng.standard_normal((N, K // 32))) * 0.002 + 1e-4).astype(np.float16).view(np.uint16)
    W = pack_on_gpu(q4, codes, scales)
    r, w = dev(rng.standard_normal((M, K)).astype(np.float32)), torch.ones(K, device="cuda")
    x, Y = torch.empty((M, K), dtype=torch.bfloat16, device="cuda"), torch.empty((M, N), device="cuda")
    q4.q4_0_block_norm(r, M, K, pre_weight=w, x=x)
    q4.q4_0_gemm(W, x, Y, M, N, K)
    y2, x2 = torch.empty((M, N), device="cuda"), torch.empty((M, 288), device="cuda")
    q4.q4_0_block_norm(Y[:, :288].contiguous(), M, 288, x=x2)       # the product's fp32 Y as a stream
    bits = workloads.fp32_to_bf16_bits(x.float().cpu().numpy())
    Y_or, B_or = oracle.get().gemm(oracle.get().pack(codes, scales), bits, M, N, K)
    check_gemm(Y.cpu().numpy(), Y_or, B_or, "norm then q4_0_gemm")
    _, want = ref.block_norm(Y[:, :288].double().cpu().numpy())
    assert np.abs(x2.double().cpu().numpy() - want).max() <= 2.0 ** -16 * np.abs(want).max()
    del y2


@pytest.mark.parametrize("M", [1, 40, 400])
def test_captured_and_replayed_on_new_inputs(q4, M):
    a, b = Block(q4, M, 1024, seed=1), Block(q4, M, 1024, seed=2)
    b.run()
    want = b.out()
    a.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run()
    for name in ("r", "pre", "post", "next", "gate", "W"):
        getattr(a, name).copy_(getattr(b, name))
    a.X.copy_(b.X)
    for _ in range(3):
        g.replay()
    for got, w in zip(a.out(), want):
        assert torch.equal(got, w)


def test_graphs_of_two_streams_at_once(q4):
    """Large and small products of two graphs share nothing but the GPU."""
    blocks = [Block(q4, M, D, seed=M) for M, D in ((300, 2048), (2, 2048), (1, 1024), (64, 1024))]
    want = []
    for b in blocks:
        b.run()
        want.append(b.out())
    torch.cuda.synchronize()
    graphs, streams = [], [torch.cuda.Stream() for _ in blocks]
    for b, s in zip(blocks, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(4):
                b.run()
        graphs.append(g)
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for b, w in zip(blocks, want):
        for got, x in zip(b.out(), w):
            assert torch.equal(got, x)
    no_device_error(q4)


def test_products_of_five_streams_at_once(q4):
    """Clusters of every size and pairs of CTAs, waiting for each other's SMs."""
    calls, want = [], []
    for M, N, K in ((64, 1024, 5120), (128, 1024, 5120), (16, 1024, 8192), (2, 5120, 4096), (300, 2048, 1024)):
        g = _gen(M)
        W = torch.empty(q4.mxfp4_bytes(N, K), dtype=torch.uint8, device="cuda")
        X = torch.empty(q4.mxfp4_bytes(M, K), dtype=torch.uint8, device="cuda")
        Y = torch.empty((M, N), device="cuda")
        q4.mxfp4_quantize(_randn(g, N, K), W, N, K)
        q4.mxfp4_quantize(_randn(g, M, K), X, M, K)
        q4.mxfp4_gemm(W, X, Y, M, N, K)
        want.append(Y.clone())
        Y.fill_(float("nan"))
        calls.append((W, X, Y, M, N, K, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(50):
        for c in calls:
            q4.mxfp4_gemm(*c)
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        assert torch.equal(c[2], w)
    no_device_error(q4)


def test_stream_arguments(q4):
    """A stream object, its handle and the current stream mean the same; the
    call waits for what is before it on that stream."""
    b = Block(q4, 6, 1024, seed=3)
    b.run()
    want = b.out()
    s = torch.cuda.Stream()
    for how in ("object", "handle", "current"):
        src = b.r.clone()
        b.r.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
            b.r.copy_(src)
            if how == "current":
                b.run()
        if how != "current":
            b.run(s if how == "object" else s.cuda_stream)
        s.synchronize()
        for got, w in zip(b.out(), want):
            assert torch.equal(got, w), how


def test_two_threads(q4):
    blocks = [Block(q4, M, 1024, seed=M) for M in (1, 300)]
    want = []
    for b in blocks:
        b.run()
        want.append(b.out())
    torch.cuda.synchronize()
    errors = []

    def work(b, w):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(50):
                    b.run()
                got = b.out()
            s.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(got, w))
        except BaseException as e:  # noqa: B902
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(blocks, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


@pytest.mark.parametrize("M,N,K", [(1, 5120, 8192), (32, 16384, 1024), (7, 2048, 8192), (128, 5120, 2048), (700, 4096, 2048),
                                   (2048, 4096, 1024)])
def test_repeated_runs_are_bit_identical(q4, M, N, K):
    g = _gen(M)
    W = torch.empty(q4.mxfp4_bytes(N, K), dtype=torch.uint8, device="cuda")
    X = torch.empty(q4.mxfp4_bytes(M, K), dtype=torch.uint8, device="cuda")
    q4.mxfp4_quantize(_randn(g, N, K), W, N, K)
    q4.mxfp4_quantize(_randn(g, M, K), X, M, K)
    first = torch.empty((M, N), device="cuda")
    q4.mxfp4_gemm(W, X, first, M, N, K)
    Y = torch.empty_like(first)
    for _ in range(20):
        Y.fill_(float("nan"))
        q4.mxfp4_gemm(W, X, Y, M, N, K)
        assert torch.equal(Y, first)
    no_device_error(q4)


def test_misaligned_views_are_refused(q4):
    flat = torch.zeros(4096, device="cuda")
    W = torch.empty(q4.mxfp4_bytes(4, 64), dtype=torch.uint8, device="cuda")
    big = torch.empty(q4.mxfp4_bytes(4, 64) + 16, dtype=torch.uint8, device="cuda")
    for call in (lambda: q4.mxfp4_quantize(flat[1:], W, 4, 64), lambda: q4.mxfp4_quantize(flat, big[8:], 4, 64),
                 lambda: q4.mxfp4_dequant(W, flat[2:], 4, 64), lambda: q4.mxfp4_gemm(W, W, flat[3:], 4, 4, 64),
                 lambda: q4.q4_0_block_norm(flat[1:], 4, 64, x=flat[64:])):
        with pytest.raises(q4.Q4Error, match="MISALIGNED"):
            call()


def test_quantize_and_dequant_past_32_bit_offsets(q4):
    R, K = 530_000, 8192                                       # 4.3e9 values, 8.7 GB of bf16
    X = torch.zeros((R, K), dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1, 262_143, 262_144, 524_287, 524_288, R - 1], device="cuda")
    X[at] = _randn(_gen(0), len(at), K).bfloat16()
    W = torch.empty(q4.mxfp4_bytes(R, K), dtype=torch.uint8, device="cuda")
    q4.mxfp4_quantize(X, W, R, K)
    X.fill_(float("nan"))
    q4.mxfp4_dequant(W, X, R, K)
    want = _randn(_gen(0), len(at), K).bfloat16().double().cpu().numpy()
    assert np.array_equal(X[at].double().cpu().numpy(), ref.values(*ref.quantize(want)))
    rest = torch.ones(R, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert not X[rest][::1009].any()
    del X, W
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M,N,K,out", [(9, 262_272, 32768, torch.float32), (300, 262_272, 32768, torch.bfloat16),
                                       (16500, 262_272, 256, torch.bfloat16)])
def test_gemm_past_32_bit_offsets(q4, M, N, K, out):
    """A weight of 4.5 GB, and an output of 4.3e9 values: the corners of the
    product against 64 bits."""
    g = _gen(M)
    W = torch.empty(q4.mxfp4_bytes(N, K), dtype=torch.uint8, device="cuda")
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device="cuda")
    scales = torch.randint(120, 134, (N, K // 32), generator=g, dtype=torch.uint8, device="cuda")
    q4.mxfp4_pack(codes, scales, W, N, K)
    X = torch.empty(q4.mxfp4_bytes(M, K), dtype=torch.uint8, device="cuda")
    x = _randn(g, M, K)
    q4.mxfp4_quantize(x, X, M, K)
    Y = torch.empty((M, N), dtype=out, device="cuda")
    q4.mxfp4_gemm(W, X, Y, M, N, K)
    ns = torch.tensor([0, 127, 128, 131_071, 131_072, 200_001, N - 1], device="cuda")
    ms = torch.tensor(sorted({0, M // 2, M - 1}), device="cuda")
    c = codes[ns].cpu().numpy()
    c = np.stack((c & 15, c >> 4), -1).reshape(len(ns), K)
    w = ref.values(c, scales[ns].cpu().numpy())
    xv = ref.values(*ref.quantize(x[ms].double().cpu().numpy()))
    exact, mag = xv @ w.T, np.abs(xv) @ np.abs(w).T
    bound = K * 2.0 ** -23 * mag
    if out == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (np.abs(exact) + bound)
    got = Y[ms][:, ns].double().cpu().numpy()
    assert np.all(np.abs(got - exact) <= bound)
    del W, codes, scales, X, Y
    torch.cuda.empty_cache()
    no_device_error(q4)


def test_block_norm_past_32_bit_offsets(q4):
    M, D = 270_000, 8192
    r = torch.ones((M, D), dtype=torch.bfloat16, device="cuda")
    r[M - 1] = torch.arange(D, device="cuda").bfloat16()
    x = torch.empty_like(r)
    w = torch.full((D,), 2.0, device="cuda")
    q4.q4_0_block_norm(r, M, D, pre_weight=w, x=x, eps=0.0)
    assert (x[:M - 1:997] == 2.0).all()
    want = ref.block_norm(r[M - 1:].double().cpu().numpy(), pre=w.double().cpu().numpy(), eps=0.0)[1]
    assert np.all(np.abs(x[M - 1:].double().cpu().numpy() - want) <= 2.0 ** -8 * (1 + 2.0 ** -8) * np.abs(want))
    del r, x
    torch.cuda.empty_cache()
