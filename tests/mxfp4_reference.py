"""Plain MXFP4 and block-norm arithmetic in numpy's 64-bit floats, written from
the format's definition, for the tests of the MXFP4 operators and of the block
norm."""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TILE_BYTES, CODE_BYTES = 17408, 16384


def bf16(x: np.ndarray) -> np.ndarray:
    """x rounded to bf16 (nearest even), as float32; NaN stays NaN."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), np.float32(np.nan), r)


def quantize(x: np.ndarray):
    """Codes [R, K] (0..15) and scale bytes [R, K/32] of x [R, K]."""
    b = np.asarray(x, np.float64).reshape(x.shape[0], -1, 32)
    with np.errstate(invalid="ignore", over="ignore"):
        a = np.abs(b).max(-1)
        bad = ~np.isfinite(b).all(-1)
        _, e = np.frexp(np.where(bad | (a == 0), 1.0, a))       # a = m * 2^e with m in [0.5, 1)
        E = np.clip(np.where(a == 0, -127, e - 3), -127, 125)
        m = np.abs(np.where(bad[..., None], 0.0, b)) * np.exp2(-E.astype(np.float64))[..., None]
        mid = (GRID[:-1] + GRID[1:]) / 2
        code = np.searchsorted(mid, m, side="left")             # a value on a midpoint goes down ...
        on = np.isin(m, mid) & (code % 2 == 1)
        code = code + on                                        # ... unless the code below it is odd
    code = np.where(np.signbit(b), code + 8, code).astype(np.uint8)
    scale = np.where(bad, 255, E + 127).astype(np.uint8)
    return code.reshape(x.shape), scale


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """The values [R, K] (float64) of codes and scale bytes."""
    v = np.where(codes & 8, -1.0, 1.0) * GRID[codes & 7]
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(s, 32, axis=1)


def packed(codes: np.ndarray) -> np.ndarray:
    """Codes [R, K] as [R, K/2] bytes, the lower k in the low bits."""
    return np.ascontiguousarray(codes[:, 0::2] | (codes[:, 1::2] << 4))


def layout(codes: np.ndarray, scales: np.ndarray):
    """The matrix's bytes, and a mask of those that are defined (rows past R are not)."""
    R, K = codes.shape
    rt, kt = -(-R // 128), -(-K // 256)
    out = np.zeros((rt, kt, TILE_BYTES), np.uint8)
    known = np.zeros(out.shape, bool)
    c = np.zeros((R, kt * 256), np.uint8)
    c[:, :K] = codes
    s = np.zeros((R, kt * 8), np.uint8)
    s[:, :K // 32] = scales
    p = packed(c).reshape(R, kt, 8, 16)
    for row in range(R):
        t, r = divmod(row, 128)
        for b in range(8):
            at = 128 * r + 16 * (b ^ (r & 7))
            out[t, :, at:at + 16] = p[row, :, b]
            known[t, :, at:at + 16] = True
            at = CODE_BYTES + 512 * (b // 4) + 16 * (r % 32) + 4 * (r // 32) + b % 4
            out[t, :, at] = s[row].reshape(kt, 8)[:, b]
            known[t, :, at] = True
    return out.reshape(-1), known.reshape(-1)


def block_norm(r, y=None, post=None, gate=None, span=0, scale=1.0, pre=None, eps=1e-6):
    """(r', x) in 64 bits."""
    r = np.asarray(r, np.float64)
    if y is not None:
        h = np.asarray(y, np.float64)
        if post is not None:
            h = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * np.asarray(post, np.float64)
        if gate is not None:
            g = np.asarray(gate, np.float64).reshape(-1, r.shape[1])
            h = h * g[np.arange(r.shape[0]) // span if span else np.zeros(r.shape[0], int)]
        r = r + scale * h
    x = r / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    return r, x if pre is None else x * np.asarray(pre, np.float64)
