"""The root-mean-square norm at the ends of its range, against float64 (oracle/ops.py) on the same
inputs: rows and eps so small that a power of r = 1 / sqrt(mean(s^2) + eps) leaves fp32's range while
the result does not.  Bounds as in test_gpu_rmsnorm.py, whose helpers these are."""
import numpy as np
import pytest

from oracle import ops
from tests.test_gpu_rmsnorm import E, _code, _close, _n, _np, _pkg, _randn, _stream, _type, _u

pytestmark = pytest.mark.gpu


# eps, size of the rows: r = 1e15 and 4e18; r = 1e10 and 1e15 from eps alone, over rows of zeros
# and rows far below it.  Widths of each of the kernels: vectors, single values, two passes.
@pytest.mark.parametrize("eps,size", [(0.0, 1e-15), (0.0, 2.5e-19), (1e-20, 0.0), (1e-30, 0.0), (1e-30, 1e-18)])
@pytest.mark.parametrize("rows,d", [(5, 8), (700, 1024), (3, 4096), (5, 16384), (40, 103), (5, 5001), (3, 8193)])
@pytest.mark.parametrize("xt,rt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_backward_of_tiny_rows(rows, d, xt, rt, eps, size):
    import torch
    pkg = _pkg()
    gen = torch.Generator(device="cuda").manual_seed(rows + d)
    s = (torch.randn((rows, d), generator=gen, device="cuda") * size).to(_type(rt))
    s[:, 0] = size  # no row of zeros where eps is 0, which has no norm
    dy, dres, gamma = _randn(gen, (rows, d), xt), _randn(gen, (rows, d), rt), 1 + _randn(gen, (d,), "f32", 0.2)
    dx, dsum = torch.empty((rows, d), dtype=_type(xt), device="cuda"), torch.empty((rows, d), dtype=_type(rt), device="cuda")
    dgamma = torch.empty(d, device="cuda")
    h = pkg.tfl_rmsnorm_create(d, _code(xt), _code(rt), _code(xt), eps)
    pkg.tfl_rmsnorm_backward(h, rows, s.data_ptr(), gamma.data_ptr(), dy.data_ptr(), dres.data_ptr(), dx.data_ptr(),
                             dsum.data_ptr(), dgamma.data_ptr(), _stream())
    torch.cuda.synchronize()
    pkg.tfl_rmsnorm_destroy(h)
    eps = float(np.float32(eps))
    s, dy, dres, gamma = _np(s), _np(dy), _np(dres), _np(gamma)
    ds, dg = ops.rms_norm_backward(s, gamma, dy, dres, eps)
    r = 1 / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps)
    a = dy * gamma
    m = np.abs(dres) + r * np.abs(a) + np.abs(s) * r ** 3 * np.mean(np.abs(a * s), axis=1, keepdims=True)
    # squares of rows of size 2.5e-19 (6e-38) are good to fp32's least value: 2^-149 / 6e-38 < 2^-24 each
    own = (3.5 * _n(d) + 24) * E * m
    _close(_np(dx), ds, own + _u(xt) * np.abs(ds), "dx")
    _close(_np(dsum), ds, own + _u(rt) * np.abs(ds), "dsum")
    _close(_np(dgamma), dg, (rows / 304 + 64 + _n(d) + 12) * E * np.sum(np.abs(dy * s * r), axis=0) + 1e-30, "dgamma")


# rows of zeros and rows whose y lies below the least maximum a scale is taken from (2^-100 = 7.9e-31),
# beside ordinary ones: r up to 1e6 and 1e15, times 448 / 2^-100 = 5.7e32
@pytest.mark.parametrize("eps,tiny", [(1e-12, 2.0 ** -126), (1e-14, 2.0 ** -126), (1e-30, 2.0 ** -130)])
@pytest.mark.parametrize("rows,d", [(6, 8), (700, 1024), (6, 103), (6, 5001), (6, 8193), (6, 16384)])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_e4m3_of_rows_of_zeros_and_of_almost_nothing(rows, d, xt, eps, tiny):
    import torch
    pkg = _pkg()
    gen = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn((rows, d), generator=gen, device="cuda")
    x[1::6] = 0
    x[2::6] = tiny * torch.randint(-3, 4, x[2::6].shape, generator=gen, device="cuda")
    x, gamma = x.to(_type(xt)), torch.ones(d, device="cuda")
    y, scale = torch.zeros((rows, d), device="cuda").to(_type("e4m3")), torch.zeros(rows, device="cuda")
    h = pkg.tfl_rmsnorm_create(d, _code(xt), _code(xt), _code("e4m3"), eps)
    pkg.tfl_rmsnorm_forward(h, rows, x.data_ptr(), None, gamma.data_ptr(), None, y.data_ptr(), scale.data_ptr(), _stream())
    torch.cuda.synchronize()
    pkg.tfl_rmsnorm_destroy(h)
    _, ref = ops.rms_norm(_np(x), None, _np(gamma), float(np.float32(eps)))
    rs = ops.row_scale(ref)
    own = (_n(d) / 2 + 10) * E * np.abs(ref)
    _close(_np(scale), rs, (_n(d) / 2 + 14) * E * rs, "scale")
    assert (_np(y)[1::6] == 0).all() and (_np(y)[2::6] != 0).any()
    # as in test_gpu_rmsnorm.py, in units of the scale (products with it leave no room for subnormals)
    _close(_np(y), ref / rs[:, None], 2.0 ** -4 * np.abs(ref / rs[:, None]) + 2.0 ** -10 + 2 * own / rs[:, None], "y")
