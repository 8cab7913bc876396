"""Layer norm and the linear layer at the ends of their range: buffers whose offsets pass 32 bits, and a
program whose very first call is captured into a graph.  Helpers of test_gpu_ops_range.py."""
import subprocess
import sys

import numpy as np
import pytest

from oracle import ops
from tests.test_gpu_ops_range import EPS, ROOT, _big, _close, _np, _rows

pytestmark = pytest.mark.gpu


def _st():
    import torch
    return torch.cuda.current_stream().cuda_stream


def test_layer_norm_of_more_than_two_to_the_32_values():
    import torch
    import attention_qkv_gemm_gb300 as pkg
    rows, d = 140_000, 32768  # 4.6e9 values
    gen = torch.Generator(device="cuda").manual_seed(0)
    x, gamma, beta = _big((rows, d), gen), 1 + 0.1 * torch.randn(d, generator=gen, device="cuda"), torch.ones(d, device="cuda")
    y, scale = torch.empty(rows, d, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(rows, device="cuda")
    h = pkg.tfl_layernorm_create(d, pkg.TFL_BF16, pkg.TFL_BF16, pkg.TFL_E4M3, EPS)
    pkg.tfl_layernorm_forward(h, rows, x.data_ptr(), None, gamma.data_ptr(), beta.data_ptr(), None, y.data_ptr(),
                              scale.data_ptr(), None, _st())
    torch.cuda.synchronize()
    pkg.tfl_layernorm_destroy(h)
    for i in _rows(rows):
        r = ops.layer_norm(_np(x[i:i + 1]), None, _np(gamma), _np(beta), EPS)[1]
        got = _np(y[i:i + 1]) * float(scale[i])
        assert (np.abs(got - r) <= 2.0 ** -4 * np.abs(r) + 2.0 ** -9 * float(scale[i])).all()


@pytest.mark.parametrize("rows,d", [(150_001, 16384), (1_100_003, 2001)])  # 2.5e9 and 2.2e9 values
def test_layer_norm_backward_of_more_than_two_to_the_31_values(rows, d):
    import torch
    import attention_qkv_gemm_gb300 as pkg
    gen = torch.Generator(device="cuda").manual_seed(1)
    s, dy = _big((rows, d), gen), _big((rows, d), gen)
    gamma, dgamma, dbeta = torch.ones(d, device="cuda"), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    stats = torch.empty(rows, 2, device="cuda")
    for i in range(0, rows, 20_000):
        var, m = torch.var_mean(s[i:i + 20_000].float(), dim=1, correction=0)
        stats[i:i + 20_000, 0], stats[i:i + 20_000, 1] = m, torch.rsqrt(var + EPS)
    dx = torch.empty_like(s)
    h = pkg.tfl_layernorm_create(d, pkg.TFL_BF16, pkg.TFL_BF16, pkg.TFL_BF16, EPS)
    pkg.tfl_layernorm_backward(h, rows, s.data_ptr(), stats.data_ptr(), gamma.data_ptr(), dy.data_ptr(), None, dx.data_ptr(), None,
                               dgamma.data_ptr(), dbeta.data_ptr(), _st())
    torch.cuda.synchronize()
    pkg.tfl_layernorm_destroy(h)
    for i in _rows(rows):
        st = _np(stats[i:i + 1])
        r = ops.layer_norm_backward(_np(s[i:i + 1]), st[:, 0], st[:, 1], _np(gamma), _np(dy[i:i + 1]), None)[0]
        _close(_np(dx[i:i + 1]), r, 2.0 ** -8)
    ref = torch.zeros(2, 64, dtype=torch.float64, device="cuda")
    for i in range(0, rows, 20_000):
        b = dy[i:i + 20_000, :64].double()
        t = (s[i:i + 20_000, :64].double() - stats[i:i + 20_000, :1].double()) * stats[i:i + 20_000, 1:].double()
        ref += torch.stack([(t * b).sum(0), b.sum(0)])
    # fp32 sums of up to 1.1e6 terms of size about 1, a thread's rows / 152 of them in a row: far below 0.5 of a
    # spread of 390 to 1050
    assert (dgamma[:64].double() - ref[0]).abs().max() < 0.5 and (dbeta[:64].double() - ref[1]).abs().max() < 0.5


def test_linear_of_more_than_two_to_the_32_outputs():
    import torch
    import attention_qkv_gemm_gb300 as pkg
    tokens, k, n = 140_000, 64, 32768  # y, z and the residual: 4.6e9 values
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, w, bias = _big((tokens, k), gen), _big((n, k), gen, 0.125), torch.randn(n, generator=gen, device="cuda")
    y, z, res = (torch.empty(tokens, n, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    for i, part in enumerate(res.split(1000)):
        part.fill_(float(i % 7))
    op = pkg.tfl_linear_create(k, n, pkg.TFL_BF16, pkg.TFL_BF16, pkg.TFL_ACT_SILU)
    pkg.tfl_linear_forward(op, tokens, x.data_ptr(), None, w.data_ptr(), None, bias.data_ptr(), res.data_ptr(), z.data_ptr(),
                           y.data_ptr(), _st())
    assert pkg.tfl_linear_status(op, _st()) == 0
    pkg.tfl_linear_destroy(op)
    for i in _rows(tokens):
        r, rz = ops.linear(_np(x[i:i + 1]), _np(w), _np(bias), _np(res[i:i + 1]), "silu")
        _close(_np(y[i:i + 1]), r, 2.0 ** -8)
        _close(_np(z[i:i + 1]), rz, 2.0 ** -8)


def test_linear_backward_of_more_than_two_to_the_31_slopes():
    import torch
    import attention_qkv_gemm_gb300 as pkg
    tokens, k, n = 70_000, 64, 32768  # dz: 2.3e9 values
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, w, z, dy = _big((tokens, k), gen), _big((n, k), gen, 0.125), _big((tokens, n), gen), _big((tokens, n), gen, 0.01)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(n, device="cuda")
    op = pkg.tfl_linear_create(k, n, pkg.TFL_BF16, pkg.TFL_BF16, pkg.TFL_ACT_SILU, pkg.TFL_BF16, tokens)
    pkg.tfl_linear_backward(op, tokens, x.data_ptr(), w.data_ptr(), z.data_ptr(), dy.data_ptr(), dx.data_ptr(), dw.data_ptr(),
                            db.data_ptr(), _st())
    assert pkg.tfl_linear_status(op, _st()) == 0
    pkg.tfl_linear_destroy(op)
    for i in _rows(tokens):
        r = ops.linear_backward(_np(x[i:i + 1]), _np(w), _np(z[i:i + 1]), _np(dy[i:i + 1]), "silu")[0]
        # dz and dx rounded to bf16: relative 2-norm at most 1.2 * 2^-8 over these 64 sums of 32768
        assert np.linalg.norm(_np(dx[i:i + 1]) - r) <= 1.5 * 2.0 ** -8 * np.linalg.norm(r)
    for at in (0, n - 64):
        sl = slice(at, at + 64)
        p = torch.sigmoid(z[:, sl].double())
        dz = dy[:, sl].double() * (p + z[:, sl].double() * p * (1 - p))
        r = dz.t() @ x.double()
        assert float((dw[sl].double() - r).norm() / r.norm()) <= 1.5 * 2.0 ** -8
        assert float((db[sl].double() - dz.sum(0)).abs().max() / dz.abs().sum(0).max()) <= 2.0 ** -18


FIRST_CALL = """
import sys, torch
sys.path.insert(0, {root!r})
import attention_qkv_gemm_gb300 as pkg
x = torch.randn(9, 256, device="cuda").bfloat16()
w = torch.randn(64, 256, device="cuda").bfloat16()
g, b = torch.ones(256, device="cuda"), torch.zeros(64, device="cuda")
y, h, z, dx = torch.empty_like(x), torch.zeros(9, 64, device="cuda").bfloat16(), torch.zeros(9, 64, device="cuda").bfloat16(), torch.zeros_like(x)
st1, dg, dbe, dw, db = torch.zeros(9, 2, device="cuda"), torch.zeros_like(g), torch.zeros_like(g), torch.zeros_like(w), torch.zeros_like(b)
n = pkg.tfl_layernorm_create(256, 2, 2, 2)
f = pkg.tfl_linear_create(256, 64, 2, 2, pkg.TFL_ACT_GELU, 2, 9)
P = lambda t: t.data_ptr()
def step(st):
    pkg.tfl_layernorm_forward(n, 9, P(x), None, P(g), None, None, P(y), None, P(st1), st)
    pkg.tfl_linear_forward(f, 9, P(y), None, P(w), None, P(b), None, P(z), P(h), st)
    pkg.tfl_linear_backward(f, 9, P(y), P(w), P(z), P(h), P(dx), P(dw), P(db), st)
    pkg.tfl_layernorm_backward(n, 9, P(x), P(st1), P(g), P(dx), None, P(dx), None, P(dg), P(dbe), st)
graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
torch.cuda.synchronize()
with torch.cuda.graph(graph, stream=st):
    step(st.cuda_stream)
graph.replay()
torch.cuda.synchronize()
first = [t.clone() for t in (h, z, dx, dg, dbe, dw, db)]
step(torch.cuda.current_stream().cuda_stream)
torch.cuda.synchronize()
assert all(torch.equal(a, b) and a.abs().sum() > 0 for a, b in zip(first, (h, z, dx, dg, dbe, dw, db)))
print("same")
"""


def test_the_first_call_of_a_program_may_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.format(root=ROOT)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr
