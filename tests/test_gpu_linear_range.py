"""The linear layer's activations at the ends of z's range, in every form of its forward."""
import pytest

import attention_qkv_gemm_gb300 as pkg
from tests.test_gpu_linear import P, _code, _stream, _type

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
# z, act(z): -inf is -inf times 0, no number, as in the gated feed-forward; past 1e4 the activation is 0 or z to
# the last bit, and 2^60 and 2^100 are numbers of bf16 and fp32 alike
Z = [INF, -INF, NAN, 2.0 ** 60, -2.0 ** 60, 2.0 ** 100, -2.0 ** 100, 0.0]
Y = [INF, NAN, NAN, 2.0 ** 60, 0.0, 2.0 ** 100, 0.0, 0.0]

# the few-token kernel, lone CTAs, CTAs that share a sum, pairs of narrow and of wide tiles
FORMS = [((3, 64, 64), pkg.TFL_GLU_FORM_FEW), ((40, 64, 64), pkg.TFL_GLU_FORM_LONE), ((40, 4096, 64), pkg.TFL_GLU_FORM_SHARED),
         ((2600, 1024, 2064), pkg.TFL_GLU_FORM_PAIR), ((5860, 272, 1472), pkg.TFL_GLU_FORM_WIDE)]


def test_the_sizes_take_these_forms():
    for kind in (pkg.TFL_BF16, pkg.TFL_E4M3):
        for (tokens, k, n), form in FORMS:
            assert pkg.tfl_selftest_linear_plan(k, n, kind, 0, tokens)[0] == form, (kind, tokens, k, n)


@pytest.mark.parametrize("tokens,k,n", [size for size, _ in FORMS])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("kind,out,res,train", [("bf16", "f32", False, False), ("bf16", "f32", True, True),
                                                ("bf16", "bf16", True, False), ("bf16", "bf16", False, True),
                                                ("e4m3", "f32", False, False)])
def test_infinite_and_large_z(tokens, k, n, act, kind, out, res, train):
    """x is zero, so z is the bias, exactly."""
    import torch
    x, w = torch.zeros(tokens, k, device="cuda"), torch.ones(n, k, device="cuda")
    xs = ws = None
    if kind == "e4m3":
        x, w = x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn)
        xs, ws = torch.ones(tokens, device="cuda"), torch.ones(n, device="cuda")
    else:
        x, w = x.bfloat16(), w.bfloat16()
    bias = torch.tensor(Z, device="cuda").repeat(n // 8)
    want = bias if act == "none" else torch.tensor(Y, device="cuda").repeat(n // 8)
    y = torch.full((tokens, n), 7.0, device="cuda").to(_type(out))
    r = torch.zeros_like(y) if res else None
    z = torch.full((tokens, n), 7.0, device="cuda").bfloat16() if train and act != "none" else None
    op = pkg.tfl_linear_create(k, n, _code(kind), _code(out), _code(act))
    pkg.tfl_linear_forward(op, tokens, P(x), P(xs), P(w), P(ws), P(bias), P(r), P(z), P(y), _stream())
    assert pkg.tfl_linear_status(op, _stream()) == 0
    pkg.tfl_linear_destroy(op)
    same = lambda a, b: bool(((a.float() == b) | (a.isnan() & b.isnan())).all())  # noqa: E731
    assert same(y, want.expand(tokens, n)), y[0, :8].tolist()
    assert z is None or same(z, bias.expand(tokens, n)), z[0, :8].tolist()
