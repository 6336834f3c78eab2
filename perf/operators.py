"""Cases and plain forms of the MXFP4 operators and of the fused block norm.

MXFP4: rows cut into blocks of 32 values along K; a value is an E2M1 number (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign) times its
block's power of two, E = floor(log2(largest magnitude)) - 2, held as the byte E + 127.

Kinds of cases: "quantize" (values to MXFP4 and back to the values they stand for), "gemm" (activations to MXFP4, then their product
with an MXFP4 weight), "norm" (a block's output into the residual stream, and the next product's input), "step" (norm straight to
MXFP4, then the product: the run of them in a decoder)."""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # activations of one token, as a decode step quantises them before each product
        {"name": "quantize one token", "kind": "quantize", "rows": 1, "K": 5120, "type": "bf16"},
        # activations of a prompt, with an odd number of rows and a K that ends inside a tile
        {"name": "quantize a ragged prompt", "kind": "quantize", "rows": 1003, "K": 4128, "type": "f16"},
        # a weight matrix of a feed-forward block, quantised when a model is loaded
        {"name": "quantize a weight", "kind": "quantize", "rows": 16384, "K": 5120, "type": "f32"},
        # decode of one sequence: the feed-forward block's down projection
        {"name": "gemm one token", "kind": "gemm", "M": 1, "N": 5120, "K": 8192, "out": "f32"},
        # 32 concurrent sequences through the gate/up projection
        {"name": "gemm 32 tokens", "kind": "gemm", "M": 32, "N": 16384, "K": 5120, "out": "f32"},
        # a short prompt with odd sizes
        {"name": "gemm ragged", "kind": "gemm", "M": 333, "N": 5003, "K": 4128, "out": "bf16"},
        # a long prompt through the gate/up projection
        {"name": "gemm prompt", "kind": "gemm", "M": 4096, "N": 16384, "K": 5120, "out": "bf16"},
        # after a block of one token: one gate for all rows
        {"name": "norm one token", "kind": "norm", "M": 1, "D": 5120, "y": "f32", "r": "f32", "x": "bf16", "span": 0},
        # a batch of sequences of 77 rows, each with a gate of its own, on a bf16 residual stream
        {"name": "norm gates by sequence", "kind": "norm", "M": 1001, "D": 4128, "y": "bf16", "r": "bf16", "x": "bf16", "span": 77},
        # a long prompt on an fp32 residual stream
        {"name": "norm prompt", "kind": "norm", "M": 4096, "D": 8192, "y": "f32", "r": "f32", "x": "bf16", "span": 0},
        # decode of two sequences: norm, then the fused query/key/value projection
        {"name": "step two tokens", "kind": "step", "M": 2, "N": 5120, "K": 4096, "y": "f32", "r": "f32", "span": 1},
        # a prompt: norm, then the projection
        {"name": "step prompt", "kind": "step", "M": 1500, "N": 5120, "K": 4096, "y": "bf16", "r": "f32", "span": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _k(rng, lo, hi):
    return max(lo, _log(rng, lo, hi) // 32 * 32)


def draw(rng):
    kind = rng.choice(["quantize", "gemm", "gemm", "norm", "step"])
    if kind == "quantize":
        return {"kind": kind, "rows": _log(rng, 1, 8192), "K": _k(rng, 256, 8192), "type": rng.choice(["f32", "bf16", "f16"])}
    if kind == "gemm":
        return {"kind": kind, "M": _log(rng, 1, 4096), "N": _log(rng, 256, 16384), "K": _k(rng, 256, 5120),
                "out": rng.choice(["f32", "bf16"])}
    M, span = _log(rng, 1, 4096), rng.choice([0, 0, 1, 19, 256])
    if kind == "norm":
        return {"kind": kind, "M": M, "D": _k(rng, 256, 8192), "y": rng.choice(["f32", "bf16"]), "r": rng.choice(["f32", "bf16"]),
                "x": "bf16", "span": span}
    return {"kind": kind, "M": M, "N": _log(rng, 256, 16384), "K": _k(rng, 256, 5120), "y": rng.choice(["f32", "bf16"]),
            "r": "f32", "span": span}


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, rows, K):
    """Rows of different loudness, a few channels much larger than the others."""
    x = _randn(g, rows, K)
    x.mul_(torch.exp(0.5 * _randn(g, rows, 1)))
    return x.mul_(torch.where(torch.rand((1, K), generator=g, device="cuda") < 0.01, 12.0, 1.0))


def _weight(s, g, N, K):
    """An MXFP4 weight as a checkpoint holds it: codes two to a byte (the lower k in the low bits), one scale byte a block."""
    e, mag, sign = _codes(_randn(g, N, K).mul_(0.02))
    code = torch.zeros_like(mag, dtype=torch.uint8)
    for i, v in enumerate(GRID):
        code.masked_fill_(mag == v, i)
    code = (code + 8 * sign.to(torch.uint8)).view(N, K // 2, 2)
    s["codes"] = (code[..., 0] + 16 * code[..., 1]).contiguous()
    s["scales"] = (e + 127).to(torch.uint8).view(N, K // 32)
    if own:  # laid out once, when the weights are loaded
        import bit_weight_only_matmul_b200 as q4
        s["W"] = torch.empty(q4.mxfp4_bytes(N, K), dtype=torch.uint8, device="cuda")
        q4.mxfp4_pack(s["codes"], s["scales"], s["W"], N, K)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    kind = case["kind"]
    if kind == "quantize":
        R, K = case["rows"], case["K"]
        x = _activations(g, R, K) if case["type"] != "f32" else _randn(g, R, K).mul_(0.02)
        s["X"] = x.to(DTYPES[case["type"]])
        s["out"] = torch.empty((R, K), dtype=torch.bfloat16, device="cuda")
        rows = R
    elif kind == "gemm":
        rows, K = case["M"], case["K"]
        s["X"] = _activations(g, rows, K).to(torch.bfloat16)
        _weight(s, g, case["N"], K)
        s["Y"] = torch.empty((rows, case["N"]), dtype=DTYPES[case["out"]], device="cuda")
    else:
        rows, K = case["M"], case["D"] if kind == "norm" else case["K"]
        s["y"] = (0.7 * _activations(g, rows, K)).to(DTYPES[case["y"]])
        s["r"] = (3.0 * _activations(g, rows, K)).to(DTYPES[case["r"]])
        s["r_out"] = torch.empty_like(s["r"])
        s["post"], s["pre"] = 1 + 0.1 * _randn(g, K), 1 + 0.1 * _randn(g, K)
        s["gate"] = 0.5 * _randn(g, 1 if not case["span"] else -(-rows // case["span"]), K)
        s["scale"] = 0.75
        if kind == "norm":
            s["x"] = torch.empty((rows, K), dtype=DTYPES[case["x"]], device="cuda")
        else:
            _weight(s, g, case["N"], K)
            s["Y"] = torch.empty((rows, case["N"]), dtype=torch.bfloat16, device="cuda")
    if own and kind != "norm":  # room for the quantised rows
        import bit_weight_only_matmul_b200 as q4
        s["Xq"] = torch.empty(q4.mxfp4_bytes(rows, K), dtype=torch.uint8, device="cuda")
    return s


def _codes(x):
    """The exponents [rows, K/32, 1], E2M1 magnitudes and signs [rows, K/32, 32] of fp32 x."""
    b = x.view(x.shape[0], -1, 32)
    a = b.abs().amax(-1, keepdim=True)
    e = torch.where(a == 0, -127, (torch.frexp(a).exponent - 3).clamp(-127, 125))
    m = torch.ldexp(b.abs(), -e)
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    return e, (torch.round(m / step) * step).clamp_(max=6.0), torch.signbit(b)


def _quantized(x):
    """The values that fp32 x stands for in MXFP4."""
    e, mag, sign = _codes(x)
    return torch.ldexp(torch.where(sign, -mag, mag), e).view_as(x)


def _decoded(s):
    """The weight's values, from its codes and scale bytes."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device="cuda")
    c = s["codes"].int()
    w = grid[torch.stack((c & 15, c >> 4), dim=-1)].view(*s["scales"].shape, 32)
    return torch.ldexp(w, s["scales"].int().unsqueeze(-1) - 127).view(c.shape[0], -1)


def _norm(s):
    y, r = s["y"].float(), s["r"].float()
    h = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * s["post"]
    gate = s["gate"].repeat_interleave(s["span"], 0)[: y.shape[0]] if s["span"] else s["gate"]
    r = r + s["scale"] * gate * h
    return r, r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * s["pre"]


def _run_own(s):
    import bit_weight_only_matmul_b200 as q4
    kind = s["kind"]
    if kind == "quantize":
        q4.mxfp4_quantize(s["X"], s["Xq"], s["rows"], s["K"])
        q4.mxfp4_dequant(s["Xq"], s["out"], s["rows"], s["K"])
        return s["out"]
    if kind == "gemm":
        q4.mxfp4_quantize(s["X"], s["Xq"], s["M"], s["K"])
        q4.mxfp4_gemm(s["W"], s["Xq"], s["Y"], s["M"], s["N"], s["K"])
        return s["Y"]
    q4.q4_0_block_norm(s["r"], s["M"], s["r"].shape[1], y=s["y"], post_weight=s["post"], gate=s["gate"], gate_span=s["span"],
                       scale=s["scale"], pre_weight=s["pre"], x=s["x"] if kind == "norm" else s["Xq"], r_out=s["r_out"], eps=EPS)
    if kind == "norm":
        return s["r_out"], s["x"]
    q4.mxfp4_gemm(s["W"], s["Xq"], s["Y"], s["M"], s["N"], s["K"])
    return s["r_out"], s["Y"]


def run(s):
    if own:
        return _run_own(s)
    kind = s["kind"]
    if kind == "quantize":
        return _quantized(s["X"].float()).to(torch.bfloat16)
    if kind == "gemm":
        return (_quantized(s["X"].float()) @ _decoded(s).T).to(DTYPES[s["out"]])
    r, x = _norm(s)
    if kind == "norm":
        return r.to(s["r"].dtype), x.to(s["x"].dtype)
    return r, (_quantized(x) @ _decoded(s).T).to(torch.bfloat16)


def work(case):
    kind = case["kind"]
    if kind == "quantize":
        n = case["rows"] * case["K"]
        return {"bytes": n * (SIZE[case["type"]] + 17 / 32 + 2), "flops": 4 * n}
    if kind == "norm":
        n, D = case["M"] * case["D"], case["D"]
        gates = 1 if not case["span"] else -(-case["M"] // case["span"])
        return {"bytes": n * (SIZE[case["y"]] + 2 * SIZE[case["r"]] + SIZE[case["x"]]) + 4 * D * (2 + gates), "flops": 12 * n}
    M, N, K = case["M"], case["N"], case["K"]
    w = {"bytes": N * K * 17 / 32, "flops": 2 * M * N * K}
    if kind == "gemm":
        w["bytes"] += 2 * M * K + SIZE[case["out"]] * M * N
    else:
        gates = 1 if not case["span"] else -(-M // case["span"])
        w["bytes"] += M * K * (SIZE[case["y"]] + 2 * SIZE[case["r"]]) + 4 * K * (2 + gates) + 2 * M * N
    return w


def _nearest(x):
    """MXFP4 values of x in 64 bits: the nearest number of the grid, of two equally near ones that with the even code."""
    x = x.double()
    b = x.reshape(x.shape[0], -1, 32)
    a = b.abs().amax(-1, keepdim=True)
    k = torch.floor(torch.log2(a))
    k = k + (torch.exp2(k + 1) <= a).double() - (torch.exp2(k) > a).double()  # a logarithm next to a whole number may be rounded to either side
    unit = torch.exp2(k.sub(2).clamp(-127, 125))
    m = b.abs() / unit
    best, far = torch.zeros_like(m), m.clone()
    for i in (2, 4, 6, 1, 3, 5, 7):  # even codes first: an odd one has to be nearer
        d = (m - GRID[i]).abs()
        best = torch.where(d < far, GRID[i], best)
        far = torch.minimum(d, far)
    return (torch.copysign(best, b) * unit).reshape(x.shape)


def _weight64(s):
    c = s["codes"].long()
    grid = torch.tensor(GRID, dtype=torch.float64, device="cuda")
    w = torch.empty((c.shape[0], 2 * c.shape[1]), dtype=torch.float64, device="cuda")
    for half, part in ((0, c % 16), (1, c // 16)):
        w[:, half::2] = grid[part % 8] * (1 - 2 * (part // 8))
    return w * torch.exp2(s["scales"].double() - 127).repeat_interleave(32, 1)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "quantize":
        return _nearest(s["X"])
    if kind == "gemm":
        return torch.matmul(_nearest(s["X"]), _weight64(s).t())
    y, r = s["y"].double(), s["r"].double()
    rows = torch.arange(y.shape[0], device="cuda")
    gate = s["gate"].double()[rows // case["span"] if case["span"] else torch.zeros_like(rows)]
    h = y / torch.sqrt((y * y).sum(1, keepdim=True) / y.shape[1] + EPS) * s["post"].double()
    r = torch.addcmul(r, gate, h, value=s["scale"])
    x = r / torch.sqrt((r * r).sum(1, keepdim=True) / r.shape[1] + EPS) * s["pre"].double()
    if kind == "norm":
        return r, x
    return r, torch.matmul(_nearest(x), _weight64(s).t())
