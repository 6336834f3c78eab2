"""The MXFP4 product in the debug build (Q4_DEBUG: index checks of its copies,
its tensor-memory columns and the places it sends its sums to): no check fires
on any way the product works, and the result is exact."""
import ctypes
import importlib.util
import os

import pytest
import torch

from tests import mxfp4_exact as exact

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def dlib():
    spec = importlib.util.spec_from_file_location("q4_0_b200_build", os.path.join(ROOT, "bit_weight_only_matmul_b200", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    lib = ctypes.CDLL(mod.build(debug=True))
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.mxfp4_bytes.restype, lib.mxfp4_bytes.argtypes = i64, [i64, i64]
    lib.mxfp4_pack.argtypes = [vp, vp, vp, i64, i64, vp]
    lib.mxfp4_gemm.argtypes = [vp, vp, vp, i32, i64, i64, i64, vp]
    lib.q4_0_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint32), i32]
    return lib


def _flags(lib):
    f = ctypes.c_uint32(0)
    assert lib.q4_0_device_error(ctypes.byref(f), 1) == 0
    return f.value


@pytest.mark.parametrize("M,N,K,what", exact.CASES)
def test_no_check_fires(dlib, M, N, K, what):
    w, x, want = exact.case(M, N, K)
    s = torch.cuda.current_stream().cuda_stream
    mats = []
    for codes, scales in (w, x):
        W = torch.zeros(dlib.mxfp4_bytes(*codes.shape), dtype=torch.uint8, device="cuda")
        c, e = exact.on_gpu(codes, scales)
        assert dlib.mxfp4_pack(c.data_ptr(), e.data_ptr(), W.data_ptr(), *codes.shape, s) == 0
        mats.append(W)
    _flags(dlib)
    Y = torch.full((M, N), float("nan"), device="cuda")
    assert dlib.mxfp4_gemm(mats[0].data_ptr(), mats[1].data_ptr(), Y.data_ptr(), 0, M, N, K, s) == 0
    torch.cuda.synchronize()
    assert _flags(dlib) == 0, what
    assert exact.same(Y, want), what
