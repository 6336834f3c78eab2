"""The MXFP4 operators and the block norm where what they read is written by
another stream, or only just before: forks and joins, eager and captured, and
weights written in the same chain of launches."""
import pytest
import torch

from tests.gpu_helpers import no_device_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q4():
    import bit_weight_only_matmul_b200 as q4
    return q4


def _randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


class Chain:
    """Weights quantized, rows normed and their product, from fp32 buffers that change from run to run."""

    def __init__(self, q4, M, N, K):
        self.q4, self.sizes = q4, (M, N, K)
        self.w, self.r = torch.empty((N, K), device="cuda"), torch.empty((M, K), device="cuda")
        self.W, self.X = (torch.zeros(q4.mxfp4_bytes(R, K), dtype=torch.uint8, device="cuda") for R in (N, M))
        self.Y = torch.empty((M, N), device="cuda")

    def fill(self, seed):
        M, N, K = self.sizes
        self.w.copy_(_randn(2 * seed, N, K))
        self.r.copy_(_randn(2 * seed + 1, M, K))

    def weights(self):
        self.q4.mxfp4_quantize(self.w, self.W, self.sizes[1], self.sizes[2])

    def rows(self):
        self.q4.q4_0_block_norm(self.r, self.sizes[0], self.sizes[2], x=self.X)

    def product(self):
        self.q4.mxfp4_gemm(self.W, self.X, self.Y, *self.sizes)

    def apart(self, seed):
        """The product of seed's inputs, every launch waited for."""
        self.fill(seed)
        for f in (self.weights, self.rows, self.product):
            f()
            torch.cuda.synchronize()
        return self.Y.clone()


SIZES = [(2, 5120, 4096), (1, 256, 8192), (32, 16384, 1024), (100, 1000, 2048), (300, 5003, 1056), (1500, 5120, 512)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("captured", [False, True])
def test_weights_written_in_the_same_chain(q4, M, N, K, captured):
    """The product asks for weight tiles while the launches before it, which
    write them, still run: what it multiplies is what they wrote."""
    c = Chain(q4, M, N, K)
    want = [c.apart(seed) for seed in range(4)]

    def run():
        c.weights()
        c.rows()
        c.product()
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        run = g.replay
    for i in range(40):
        c.fill(i % 4)
        run()
        assert torch.equal(c.Y, want[i % 4]), i
    no_device_error(q4)


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("captured", [False, True])
def test_fork_and_join(q4, M, N, K, captured):
    """Weights on one stream, rows on another, the product after both."""
    c = Chain(q4, M, N, K)
    want = [c.apart(seed) for seed in range(2)]
    other = torch.cuda.Stream()

    def run():
        here = torch.cuda.current_stream()
        other.wait_stream(here)
        with torch.cuda.stream(other):
            c.weights()
        c.rows()
        here.wait_stream(other)
        c.product()
        other.wait_stream(here)
        with torch.cuda.stream(other):
            c.rows()                       # reads and writes what the product has just read
        here.wait_stream(other)
        c.product()
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        run = g.replay
    for i in range(20):
        c.fill(i % 2)
        run()
        assert torch.equal(c.Y, want[i % 2]), i
    no_device_error(q4)
