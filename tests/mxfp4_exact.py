"""MXFP4 products whose every partial sum fp32 holds exactly, in whatever order
it is taken, and the shapes that reach each way the product works."""
from __future__ import annotations

import numpy as np
import torch

from tests import mxfp4_reference as ref

# What each group reaches on 148 SMs: the number of CTAs that share K, for one
# or two rows and for more, rows that fill no group of four or eight; and the
# tiles of 128 and of 256 activation rows, with odd numbers of 128-row tiles of
# W, of X and of both, one step of K, and a last band of one tile.
SHAPES = {
    "whole K": [(1, 1, 32), (7, 20000, 288), (33, 200, 512), (100, 391, 608), (20, 20000, 3104), (113, 8000, 4128)],
    "2 parts": [(1, 6400, 2560), (2, 6400, 3104), (5, 6400, 3104), (30, 6400, 4128), (48, 7168, 7168), (127, 6400, 8160)],
    "3 parts": [(2, 2816, 2080), (13, 2304, 2080), (33, 5120, 4128), (98, 3300, 5152)],
    "4 parts": [(1, 3300, 2560), (31, 2816, 3104), (45, 2304, 3104), (127, 2816, 6176)],
    "6 parts": [(1, 100, 1312), (3, 130, 1312), (30, 100, 2080), (66, 130, 2560), (98, 100, 4128), (16, 896, 4352),
                (64, 2816, 5376)],
    "8 parts": [(2, 100, 3104), (5, 130, 3104), (45, 300, 3104), (121, 257, 8160), (128, 513, 8192)],
    "128-row tiles": [(129, 130, 288), (300, 77, 4128), (333, 1000, 1056), (1000, 200, 32)],
    "256-row tiles": [(1850, 1100, 544), (300, 6200, 800), (130, 9500, 288), (4200, 600, 288), (1850, 1100, 32),
                      (513, 5000, 4128)],
}
CASES = [(*s, what) for what, shapes in SHAPES.items() for s in shapes]


def operand(rng, R, K, nan=()):
    """Codes, scale bytes and values of R rows of K: any codes, blocks of one or
    two times a power of two that the row has for itself.  The products of a
    sum are then multiples of a quarter, at most 144 of the rows' powers, so
    that K <= 8192 of them stay below 2^24 quarters wherever the sum is
    interrupted.  `nan`: (row, block) places that get the scale byte of NaN."""
    assert K <= 8192
    codes = rng.integers(0, 16, (R, K), dtype=np.uint8)
    scales = (127 + rng.integers(-20, 21, (R, 1)) + rng.integers(0, 2, (R, K // 32))).astype(np.uint8)
    for place in nan:
        scales[place] = 255
    return codes, scales, ref.values(codes, scales)


def product(x, w):
    """X W^T in 64 bits: NaN where a row of X or of W holds one."""
    xn, wn = np.isnan(x).any(1), np.isnan(w).any(1)
    y = np.nan_to_num(x) @ np.nan_to_num(w).T
    y[xn], y[:, wn] = np.nan, np.nan
    return y


def case(M, N, K, nan=False):
    """((codes, scales) of W, of X, the product)."""
    rng = np.random.default_rng(M * 11 + N * 5 + K)
    places = [[(R - 1, K // 32 - 1), (R // 2, int(rng.integers(K // 32)))] if nan else [] for R in (N, M)]
    cw, sw, w = operand(rng, N, K, places[0])
    cx, sx, x = operand(rng, M, K, places[1])
    return (cw, sw), (cx, sx), product(x, w)


def on_gpu(codes, scales):
    """The two arrays as mxfp4_pack takes them."""
    return torch.from_numpy(ref.packed(codes)).cuda(), torch.from_numpy(scales).cuda()


def same(Y, want):
    """Y equals the exact product, rounded once to Y's type."""
    got, want = Y.cpu(), torch.from_numpy(want).to(Y.dtype)
    return torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
