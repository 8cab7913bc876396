"""The operators that stand on their own at the ends of their range: buffers whose offsets pass 32
bits, and a program whose very first call is captured into a graph."""
import os
import subprocess
import sys

import numpy as np
import pytest

from oracle import ops

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EPS = 1e-5


def _np(t):
    return t.double().cpu().numpy()


def _big(shape, gen, std=1.0):
    """bf16 values without a full-size fp32 copy."""
    import torch
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for part in out.split(max(1, (1 << 28) // shape[1])):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda") * std)
    return out


def _rows(n):
    return [0, 1, n // 2, n - 2, n - 1]


def _close(u, r, rel):
    """Every element to rel |r| plus the fp32 noise of its row (2^-16 of the row's largest)."""
    assert np.isfinite(u).all()
    assert (np.abs(u - r) <= rel * np.abs(r) + 2.0 ** -16 * np.abs(r).max(axis=-1, keepdims=True)).all()


def test_norm_of_more_than_two_to_the_32_values():
    import torch
    import attention_qkv_gemm_gb300 as pkg
    rows, d = 140_000, 32768  # 4.6e9 values
    gen = torch.Generator(device="cuda").manual_seed(0)
    x, gamma = _big((rows, d), gen), 1 + 0.1 * torch.randn(d, generator=gen, device="cuda")
    y, scale = torch.empty(rows, d, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(rows, device="cuda")
    h = pkg.tfl_rmsnorm_create(d, pkg.TFL_BF16, pkg.TFL_BF16, pkg.TFL_E4M3, EPS)
    pkg.tfl_rmsnorm_forward(h, rows, x.data_ptr(), None, gamma.data_ptr(), None, y.data_ptr(), scale.data_ptr(),
                            torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    pkg.tfl_rmsnorm_destroy(h)
    for i in _rows(rows):
        r = ops.rms_norm(_np(x[i:i + 1]), None, _np(gamma), EPS)[1]
        got = _np(y[i:i + 1]) * float(scale[i])
        assert (np.abs(got - r) <= 2.0 ** -4 * np.abs(r) + 2.0 ** -9 * float(scale[i])).all()


def test_norm_backward_of_more_than_two_to_the_31_values():
    import torch
    import attention_qkv_gemm_gb300 as pkg
    rows, d = 150_001, 16384  # 2.5e9 values
    gen = torch.Generator(device="cuda").manual_seed(1)
    s, dy = _big((rows, d), gen), _big((rows, d), gen)
    gamma, dgamma = torch.ones(d, device="cuda"), torch.empty(d, device="cuda")
    dx = torch.empty_like(s)
    h = pkg.tfl_rmsnorm_create(d, pkg.TFL_BF16, pkg.TFL_BF16, pkg.TFL_BF16, EPS)
    pkg.tfl_rmsnorm_backward(h, rows, s.data_ptr(), gamma.data_ptr(), dy.data_ptr(), None, dx.data_ptr(), None,
                             dgamma.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    pkg.tfl_rmsnorm_destroy(h)
    for i in _rows(rows):
        r = ops.rms_norm_backward(_np(s[i:i + 1]), _np(gamma), _np(dy[i:i + 1]), None, EPS)[0]
        _close(_np(dx[i:i + 1]), r, 2.0 ** -8)
    ref = torch.zeros(64, dtype=torch.float64, device="cuda")
    for i in range(0, rows, 20_000):
        a, b = s[i:i + 20_000], dy[i:i + 20_000, :64].double()
        r = torch.rsqrt(torch.linalg.vector_norm(a, dim=1, dtype=torch.float32).double() ** 2 / d + EPS)
        ref += (a[:, :64].double() * b * r[:, None]).sum(0)
    # sums of 150001 terms of size about 1, in fp32, r good to 1e-6: far below 0.1 of their spread, 387
    assert (dgamma[:64].double() - ref).abs().max() < 0.1


def test_feed_forward_of_more_than_two_to_the_32_outputs():
    import torch
    import attention_qkv_gemm_gb300 as pkg
    tokens, d, f = 140_000, 64, 32768  # h: 4.6e9 values
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, wg, wu = _big((tokens, d), gen), _big((f, d), gen, 0.125), _big((f, d), gen, 0.125)
    h = torch.empty(tokens, f, dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    op = pkg.tfl_glu_create(d, f, pkg.TFL_BF16, pkg.TFL_BF16, pkg.TFL_ACT_SILU)
    pkg.tfl_glu_forward(op, tokens, x.data_ptr(), None, wg.data_ptr(), None, wu.data_ptr(), None, h.data_ptr(), st)
    assert pkg.tfl_glu_status(op, st) == 0
    pkg.tfl_glu_destroy(op)
    for i in _rows(tokens):
        _close(_np(h[i:i + 1]), ops.glu(_np(x[i:i + 1]), _np(wg), _np(wu), "silu"), 2.0 ** -8)


def test_feed_forward_backward_of_more_than_two_to_the_31_slopes():
    import torch
    import attention_qkv_gemm_gb300 as pkg
    tokens, d, f = 70_000, 64, 32768  # dg, du: 2.3e9 values
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, wg, wu = _big((tokens, d), gen), _big((f, d), gen, 0.125), _big((f, d), gen, 0.125)
    dh = _big((tokens, f), gen, 0.01)
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    st = torch.cuda.current_stream().cuda_stream
    op = pkg.tfl_glu_create(d, f, pkg.TFL_BF16, pkg.TFL_BF16, pkg.TFL_ACT_SILU, tokens)
    pkg.tfl_glu_backward(op, tokens, x.data_ptr(), wg.data_ptr(), wu.data_ptr(), dh.data_ptr(), dx.data_ptr(),
                         dwg.data_ptr(), dwu.data_ptr(), st)
    assert pkg.tfl_glu_status(op, st) == 0
    pkg.tfl_glu_destroy(op)
    for i in _rows(tokens):
        r = ops.glu_backward(_np(x[i:i + 1]), _np(wg), _np(wu), _np(dh[i:i + 1]), "silu")[0]
        # dg, du and dx rounded to bf16: relative 2-norm at most 1.2 * 2^-8 over these 64 sums of 65536
        assert np.linalg.norm(_np(dx[i:i + 1]) - r) <= 1.5 * 2.0 ** -8 * np.linalg.norm(r)
    # the weights' gradients of 64 rows at each end of d_ff, over all tokens
    for at in (0, f - 64):
        sl = slice(at, at + 64)
        g, u, e = x.float() @ wg[sl].float().t(), x.float() @ wu[sl].float().t(), dh[:, sl].float()
        p = torch.sigmoid(g)
        for got, slope in ((dwg, e * u * p * (1 + g * (1 - p))), (dwu, e * g * p)):
            r = slope.double().t() @ x.double()
            assert float((got[sl].double() - r).norm() / r.norm()) <= 1.5 * 2.0 ** -8


FIRST_CALL = """
import sys, torch
sys.path.insert(0, {root!r})
import attention_qkv_gemm_gb300 as pkg
x = torch.randn(9, 256, device="cuda").bfloat16()
w = torch.randn(64, 256, device="cuda").bfloat16()
g = torch.ones(256, device="cuda")
y, h, dx, dg = torch.empty_like(x), torch.zeros(9, 64, device="cuda").bfloat16(), torch.zeros_like(x), torch.zeros_like(g)
dwg, dwu = torch.zeros_like(w), torch.zeros_like(w)
n = pkg.tfl_rmsnorm_create(256, 2, 2, 2)
f = pkg.tfl_glu_create(256, 64, 2, 2, 0, 9)
P = lambda t: t.data_ptr()
def step(st):
    pkg.tfl_rmsnorm_forward(n, 9, P(x), None, P(g), None, P(y), None, st)
    pkg.tfl_glu_forward(f, 9, P(y), None, P(w), None, P(w), None, P(h), st)
    pkg.tfl_glu_backward(f, 9, P(y), P(w), P(w), P(h), P(dx), P(dwg), P(dwu), st)
    pkg.tfl_rmsnorm_backward(n, 9, P(x), P(g), P(dx), None, P(dx), None, P(dg), st)
graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
torch.cuda.synchronize()
with torch.cuda.graph(graph, stream=st):
    step(st.cuda_stream)
graph.replay()
torch.cuda.synchronize()
first = [t.clone() for t in (h, dx, dg, dwg, dwu)]
step(torch.cuda.current_stream().cuda_stream)
torch.cuda.synchronize()
assert all(torch.equal(a, b) and a.abs().sum() > 0 for a, b in zip(first, (h, dx, dg, dwg, dwu)))
print("same")
"""


def test_the_first_call_of_a_program_may_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.format(root=ROOT)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr
