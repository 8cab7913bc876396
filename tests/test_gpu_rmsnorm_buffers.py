"""The root-mean-square norm's backward on buffers aligned only to their elements, and the kernels of
wide rows over more rows than they have blocks.  Bounds and helpers of test_gpu_rmsnorm.py."""
import pytest

from tests.test_gpu_rmsnorm import (EPS, _backward, _check_backward, _check_forward, _code, _forward, _pkg, _randn, _stream,
                                    _type)

pytestmark = pytest.mark.gpu

BUFFERS = ("sum", "gamma", "dy", "dres", "dx", "dsum", "dgamma")


# each buffer alone one element past its alignment, then all; every class of widths
@pytest.mark.parametrize("which", [(b,) for b in BUFFERS] + [BUFFERS])
@pytest.mark.parametrize("rows,d", [(3, 8), (700, 256), (333, 1024), (40, 2048), (40, 8192), (700, 16384)])
@pytest.mark.parametrize("xt,rt", [("bf16", "f32"), ("f16", "f16")])
def test_backward_of_unaligned_buffers(rows, d, xt, rt, which):
    import torch
    pkg = _pkg()
    gen = torch.Generator(device="cuda").manual_seed(rows + d)
    room = {}

    def place(name, t):
        at = 1 if name in which else 0
        flat = torch.full((t.numel() + 2,), 7.0, dtype=t.dtype, device="cuda")
        v = flat[at:at + t.numel()].view(t.shape)
        v.copy_(t)
        room[name] = (flat, at, t.numel())
        return v

    s, dy = place("sum", _randn(gen, (rows, d), rt, 2.0)), place("dy", _randn(gen, (rows, d), xt))
    dres, gamma = place("dres", _randn(gen, (rows, d), rt)), place("gamma", 1 + _randn(gen, (d,), "f32", 0.2))
    dx = place("dx", torch.zeros((rows, d), dtype=_type(xt), device="cuda"))
    dsum = place("dsum", torch.zeros((rows, d), dtype=_type(rt), device="cuda"))
    dgamma = place("dgamma", torch.zeros(d, device="cuda"))
    h = pkg.tfl_rmsnorm_create(d, _code(xt), _code(rt), _code(xt), EPS)
    pkg.tfl_rmsnorm_backward(h, rows, s.data_ptr(), gamma.data_ptr(), dy.data_ptr(), dres.data_ptr(), dx.data_ptr(),
                             dsum.data_ptr(), dgamma.data_ptr(), _stream())
    torch.cuda.synchronize()
    pkg.tfl_rmsnorm_destroy(h)
    _check_backward(rows, d, xt, rt, (s, dy, dres, gamma, dx, dsum, dgamma))
    for flat, at, n in room.values():  # nothing around the buffers is touched
        assert (flat[:at] == 7).all() and (flat[at + n:] == 7).all()


# more rows than the 8 blocks an SM of the forward and the 4 of the backward (on 152 SMs 1216 and 608);
# the last row's partial sums do not fit for that many blocks (64 MiB hold 41 rows of them)
@pytest.mark.parametrize("rows,d", [(2500, 8193), (1300, 32776), (100, 400001)])
@pytest.mark.parametrize("xt,rt,yt", [("bf16", "f32", "e4m3"), ("f16", "f16", "f16")])
def test_wide_rows_over_several_turns(rows, d, xt, rt, yt):
    _check_forward(rows, d, xt, rt, yt, _forward(rows, d, xt, rt, yt, seed=d))
    _check_backward(rows, d, xt, rt, _backward(rows, d, xt, rt, seed=d))
