"""What the operators that stand on their own refuse before any device work (CPU)."""
import ctypes

import pytest

import attention_qkv_gemm_gb300 as pkg
from attention_qkv_gemm_gb300 import build as libbuild


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return pkg.load()


@pytest.mark.parametrize("args,code", [
    ((0, 2, 2, 2, 1e-5), pkg.TFL_ERR_INVALID_ARG),
    (((1 << 24) + 1, 2, 2, 2, 1e-5), pkg.TFL_ERR_INVALID_ARG),
    ((64, 2, 2, 2, -1.0), pkg.TFL_ERR_INVALID_ARG),
    ((64, 2, 2, 2, float("nan")), pkg.TFL_ERR_INVALID_ARG),
    ((64, 2, 2, 2, float("inf")), pkg.TFL_ERR_INVALID_ARG),
    ((64, 3, 0, 2, 1e-5), pkg.TFL_ERR_UNSUPPORTED),   # e4m3 x
    ((64, 4, 4, 4, 1e-5), pkg.TFL_ERR_UNSUPPORTED),   # no such type
    ((64, 2, 1, 2, 1e-5), pkg.TFL_ERR_UNSUPPORTED),   # bf16 x with an fp16 residual
    ((64, 0, 2, 0, 1e-5), pkg.TFL_ERR_UNSUPPORTED),   # fp32 x with a bf16 residual
    ((64, 2, 2, 0, 1e-5), pkg.TFL_ERR_UNSUPPORTED),   # bf16 x with an fp32 y
    ((64, 1, 1, 2, 1e-5), pkg.TFL_ERR_UNSUPPORTED),   # fp16 x with a bf16 y
])
def test_rmsnorm_create_refuses(lib, args, code):
    h = ctypes.c_void_p()
    assert lib.tfl_rmsnorm_create(*args, ctypes.byref(h)) == code
    assert h.value is None and pkg.tfl_last_error() != ""


@pytest.mark.parametrize("args,code", [
    ((0, 64, 2, 2, 0, 0), pkg.TFL_ERR_INVALID_ARG),
    ((64, -8, 2, 2, 0, 0), pkg.TFL_ERR_INVALID_ARG),
    ((64, 64, 2, 2, 2, 0), pkg.TFL_ERR_INVALID_ARG),        # no such activation
    ((64, 64, 2, 2, 0, -1), pkg.TFL_ERR_INVALID_ARG),
    ((64, 64, 2, 2, 0, 1 << 31), pkg.TFL_ERR_INVALID_ARG),
    ((64, 64, 0, 0, 0, 0), pkg.TFL_ERR_UNSUPPORTED),        # fp32
    ((64, 64, 1, 2, 0, 0), pkg.TFL_ERR_UNSUPPORTED),        # fp16 operands, bf16 output
    ((64, 64, 3, 3, 0, 0), pkg.TFL_ERR_UNSUPPORTED),        # an e4m3 output
    ((64, 64, 3, 2, 0, 8), pkg.TFL_ERR_UNSUPPORTED),        # a backward of e4m3 operands
    ((68, 64, 2, 2, 0, 0), pkg.TFL_ERR_UNSUPPORTED),
    ((64, 60, 2, 2, 0, 0), pkg.TFL_ERR_UNSUPPORTED),
    ((72, 64, 3, 2, 0, 0), pkg.TFL_ERR_UNSUPPORTED),        # 16 for e4m3
    (((1 << 24) + 8, 64, 2, 2, 0, 0), pkg.TFL_ERR_UNSUPPORTED),
])
def test_glu_create_refuses(lib, args, code):
    h = ctypes.c_void_p()
    assert lib.tfl_glu_create(*args, ctypes.byref(h)) == code
    assert h.value is None and pkg.tfl_last_error() != ""


def test_null_handles_are_refused(lib):
    assert lib.tfl_glu_create(64, 64, 2, 2, 0, 0, None) == pkg.TFL_ERR_INVALID_ARG
    assert lib.tfl_glu_forward(None, 1, *[None] * 8) == pkg.TFL_ERR_INVALID_ARG
    assert lib.tfl_glu_backward(None, 1, *[None] * 8) == pkg.TFL_ERR_INVALID_ARG
    assert lib.tfl_glu_status(None, None) == pkg.TFL_ERR_INVALID_ARG
    lib.tfl_glu_destroy(None)  # no-op
    assert lib.tfl_rmsnorm_create(64, 2, 2, 2, 1e-5, None) == pkg.TFL_ERR_INVALID_ARG
    assert lib.tfl_rmsnorm_forward(None, 1, *[None] * 7) == pkg.TFL_ERR_INVALID_ARG
    assert lib.tfl_rmsnorm_backward(None, 1, *[None] * 8) == pkg.TFL_ERR_INVALID_ARG
    lib.tfl_rmsnorm_destroy(None)  # no-op
