"""The MXFP4 entry points and the block norm on the CPU: what the library
exports, the host-side argument checks (before any CUDA call), the binding's
refusals, and the reference the GPU tests compare with."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

from tests import mxfp4_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20   # a fake, 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def q4():
    import bit_weight_only_matmul_b200 as q4
    return q4


def test_every_declared_symbol_is_exported(q4):
    text = open(os.path.join(ROOT, "include", "mxfp4.h")).read()
    names = sorted(set(re.findall(r"Q4_0_API\s+[\w\s\*]*?\b(mxfp4_\w+)\s*\(", text)))
    assert names == sorted(q4.MXFP4_EXPORTS)
    lib = ctypes.CDLL(q4.LIB_PATH)
    assert all(hasattr(lib, n) for n in names)


def test_bytes(q4):
    assert q4.mxfp4_bytes(1, 32) == 17408
    assert q4.mxfp4_bytes(128, 256) == 17408
    assert q4.mxfp4_bytes(129, 257 + 31) == 4 * 17408
    assert q4.mxfp4_bytes(0, 64) == 0 and q4.mxfp4_bytes(64, 0) == 0
    assert q4.mxfp4_bytes(4, 33) == -1 and q4.mxfp4_bytes(-1, 32) == -1 and q4.mxfp4_bytes(1, 1 << 31) == -1


def test_quantize_dequant_pack_checks(q4):
    bad, mis = q4.Q4_ERR_INVALID_ARG, q4.Q4_ERR_MISALIGNED
    qz, dq, pk = q4.lib.mxfp4_quantize, q4.lib.mxfp4_dequant, q4.lib.mxfp4_pack
    for f in (lambda x, w, r, k, t=1: qz(x, t, w, r, k, None), lambda x, w, r, k, t=1: dq(w, x, t, r, k, None)):
        assert f(A, A, 4, 48) == bad                  # K % 32
        assert f(A, A, -1, 64) == bad
        assert f(A, A, 4, 64, 3) == bad               # MXFP4 is no value type
        assert f(A, A, 4, 64, -1) == bad
        assert f(None, A, 4, 64) == bad and f(A, None, 4, 64) == bad
        assert f(A + 8, A, 4, 64) == mis and f(A, A + 4, 4, 64) == mis
        assert f(None, None, 0, 64) == q4.Q4_OK and f(None, None, 4, 0) == q4.Q4_OK
    assert pk(A, A, A, 4, 40, None) == bad
    assert pk(None, A, A, 4, 64, None) == bad and pk(A, None, A, 4, 64, None) == bad and pk(A, A, None, 4, 64, None) == bad
    assert pk(A + 1, A, A, 4, 64, None) == mis and pk(A, A + 2, A, 4, 64, None) == mis and pk(A, A, A + 8, 4, 64, None) == mis
    assert pk(None, None, None, 0, 64, None) == q4.Q4_OK


def test_gemm_checks(q4):
    bad, mis, g = q4.Q4_ERR_INVALID_ARG, q4.Q4_ERR_MISALIGNED, q4.lib.mxfp4_gemm
    assert g(A, A, A, 0, 1, 8, 48, None) == bad
    assert g(A, A, A, 0, -1, 8, 64, None) == bad and g(A, A, A, 0, 1, -8, 64, None) == bad
    assert g(A, A, A, 0, 1 << 31, 8, 64, None) == bad
    assert g(A, A, A, 2, 1, 8, 64, None) == bad and g(A, A, A, 3, 1, 8, 64, None) == bad    # Y is fp32 or bf16
    assert g(None, A, A, 0, 1, 8, 64, None) == bad and g(A, None, A, 0, 1, 8, 64, None) == bad
    assert g(A, A, None, 0, 1, 8, 64, None) == bad and g(A, A, None, 0, 1, 8, 0, None) == bad
    assert g(A + 2, A, A, 0, 1, 8, 64, None) == mis and g(A, A + 8, A, 0, 1, 8, 64, None) == mis
    assert g(A, A, A + 4, 1, 1, 8, 64, None) == mis
    assert g(None, None, None, 0, 0, 8, 64, None) == q4.Q4_OK and g(None, None, None, 0, 4, 0, 64, None) == q4.Q4_OK


def test_block_norm_checks(q4):
    bad, mis = q4.Q4_ERR_INVALID_ARG, q4.Q4_ERR_MISALIGNED

    def f(**k):
        b = q4.q4_0_block(**{**dict(y=A, r=A, r_out=A, x=A, post_weight=A, gate=A, pre_weight=A, M=4, D=64, gate_span=0,
                                    scale=1.0, eps=1e-6, y_type=0, r_type=0, x_type=1), **k})
        return q4.lib.q4_0_block_norm(ctypes.byref(b), None)

    assert f(D=48) == bad and f(D=-32) == bad and f(M=-1) == bad and f(D=q4.Q4_0_MAX_NORM_DIM + 32) == bad
    assert f(y_type=2) == bad and f(r_type=2) == bad and f(r_type=3) == bad and f(x_type=2) == bad and f(x_type=4) == bad
    assert f(eps=-1.0) == bad and f(eps=float("nan")) == bad and f(eps=float("inf")) == bad
    assert f(gate_span=-1) == bad
    assert f(r=None) == bad and f(r_out=None, x=None, pre_weight=None) == bad
    assert f(y=None) == bad and f(y=None, gate=None) == bad           # a weight or gate of nothing
    assert f(x=None) == bad                                           # a second weight without a second norm
    for name in ("y", "r", "r_out", "x", "post_weight", "gate", "pre_weight"):
        assert f(**{name: A + 8}) == mis, name
    assert f(M=0) == q4.Q4_OK and f(D=0) == q4.Q4_OK
    assert q4.lib.q4_0_block_norm(None, None) == bad


def test_binding_refuses_host_tensors(q4):
    x = torch.zeros(4, 64)
    w = torch.zeros(q4.mxfp4_bytes(4, 64), dtype=torch.uint8)
    for call in (lambda: q4.mxfp4_quantize(x, w, 4, 64), lambda: q4.mxfp4_dequant(w, x, 4, 64),
                 lambda: q4.mxfp4_gemm(w, w, x, 4, 4, 64), lambda: q4.q4_0_block_norm(x, 4, 64, x=x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_block_struct_matches_the_header(q4, tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    fields = [n for n, _ in q4.q4_0_block._fields_]
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "mxfp4.h"', "int main(void) {",
             '    printf("size %zu\\n", sizeof(q4_0_block));']
    lines += [f'    printf("{n} %zu\\n", offsetof(q4_0_block, {n}));' for n in fields] + ["    return 0;", "}"]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines) + "\n")
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", f"-I{os.path.join(ROOT, 'include')}", str(src),
                    "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split("\n")
    got = dict(l.split() for l in out if l.strip())
    assert int(got["size"]) == ctypes.sizeof(q4.q4_0_block)
    for n in fields:
        assert int(got[n]) == getattr(q4.q4_0_block, n).offset, n


def test_reference_quantizes_by_the_definition():
    """Every E2M1 number, every midpoint (to the even code) and the ends of the
    scale's range, from hand-derived values."""
    x = np.zeros((1, 32))
    x[0, :16] = [0, 0.5, 1, 1.5, 2, 3, 4, 6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 7.9]
    x[0, 16:] = -x[0, :16]
    c, s = ref.quantize(x)
    assert s[0, 0] == 127                                       # largest magnitude 7.9: floor(log2) - 2 = 0
    assert list(c[0, :16]) == [0, 1, 2, 3, 4, 5, 6, 7, 0, 2, 2, 4, 4, 6, 6, 7]
    assert list(c[0, 17:32]) == [int(v) + 8 for v in c[0, 1:16]]
    for a, byte in ((0.0, 0), (2.0 ** -149, 0), (2.0 ** -125, 0), (2.0 ** -124, 1), (1.0, 125), (2.0 ** 127, 252),
                    (3.4028234663852886e38, 252), (np.inf, 255), (np.nan, 255)):
        assert ref.quantize(np.full((1, 32), a))[1][0, 0] == byte, a
    v = ref.values(*ref.quantize(x))
    assert np.abs(v - x)[0, :15].max() == 1.0 and v[0, 15] == 6.0    # 5 is one away from 4
