"""Layer norm in every kernel: rows that begin inside a 16-byte vector above all, at sizes chosen by the dispatch's
rule (bounds as in test_gpu_layernorm.py)."""
import pytest

from tests import layernorm_forms as forms
from tests.test_gpu_layernorm import _backward, _check_backward, _check_forward, _forward
from tests.test_gpu_rmsnorm import _code, _pkg, _stream
from tests.test_layernorm_plan import every_size

pytestmark = pytest.mark.gpu

EPS = 1e-5
P = lambda t: None if t is None else t.data_ptr()  # noqa: E731


def test_the_sizes_reach_every_kernel_on_this_gpu():
    pkg = _pkg()
    for part, sizes in ((0, forms.FORWARD), (1, forms.BACKWARD)):
        assert forms.kinds(part, sizes) == forms.kinds(part, every_size())
    for rows, d in forms.STRADDLE:
        assert pkg.tfl_selftest_layernorm_plan(d, pkg.TFL_F32, 1, rows)[0] == pkg.TFL_LN_FORM_STRADDLE


@pytest.mark.parametrize("rows,d", forms.FORWARD)
@pytest.mark.parametrize("xt,rt,yt", [("bf16", "f32", "e4m3"), ("f16", "f16", "f16"), ("bf16", "bf16", "e4m3"), ("f32", "f32", "bf16"),
                                      ("f16", "f32", "f16")])
def test_forward_in_every_kernel(rows, d, xt, rt, yt):
    _check_forward(rows, d, xt, rt, yt, _forward(rows, d, xt, rt, yt, seed=rows + d))


@pytest.mark.parametrize("rows,d", forms.BACKWARD)
@pytest.mark.parametrize("xt,rt", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
def test_backward_in_every_kernel(rows, d, xt, rt):
    _check_backward(rows, d, xt, rt, _backward(rows, d, xt, rt, seed=rows + d))


@pytest.mark.parametrize("rows,d", forms.STRADDLE)
@pytest.mark.parametrize("xt,rt", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
def test_backward_of_many_rows_that_begin_inside_a_vector(rows, d, xt, rt):
    _check_backward(rows, d, xt, rt, _backward(rows, d, xt, rt, seed=rows + d))


@pytest.mark.parametrize("rows,d", [(250001, 9), (20000, 103), (6000, 516), (2003, 4099)])
@pytest.mark.parametrize("xt,rt", [("f16", "f32"), ("bf16", "bf16")])
def test_backward_without_what_may_be_left_out(rows, d, xt, rt):
    _check_backward(rows, d, xt, rt, _backward(rows, d, xt, rt, with_dres=False, both=False, with_beta=False, seed=d))


@pytest.mark.parametrize("rows,d", [(250001, 9), (120001, 18), (45001, 50), (20000, 103), (10001, 242), (6000, 513), (6000, 516),
                                    (4001, 514), (1500, 2034), (1001, 4082), (2003, 4099), (1000, 8177)])
@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_backward_in_place_of_rows_that_share_vectors(rows, d, t):
    """Neighbouring rows' groups read and write the same 16 bytes: each its own values of them."""
    import torch
    pkg = _pkg()
    s, stats, dy, dres, gamma, dx, _, dgamma, dbeta = _backward(rows, d, t, t, both=False, seed=4)
    h = pkg.tfl_layernorm_create(d, _code(t), _code(t), _code(t), EPS)
    for first, second in (("dy", None), ("dres", None), ("sum", None), ("dy", "sum"), ("sum", "dres")):
        for _ in range(3):
            b = {"sum": s.clone(), "dy": dy.clone(), "dres": dres.clone(), None: None}
            g2, b2 = torch.empty_like(dgamma), torch.empty_like(dbeta)
            pkg.tfl_layernorm_backward(h, rows, P(b["sum"]), P(stats), P(gamma), P(b["dy"]), P(b["dres"]), P(b[first]), P(b[second]),
                                       P(g2), P(b2), _stream())
            assert torch.equal(b[first], dx) and torch.equal(g2, dgamma) and torch.equal(b2, dbeta), (first, second)
            assert second is None or torch.equal(b[second], dx), (first, second)
    pkg.tfl_layernorm_destroy(h)


@pytest.mark.parametrize("rows,d", [(40009, 9), (40009, 18), (20000, 103), (6007, 250), (2600, 2034), (601, 4099), (601, 8177)])
@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_forward_in_place_of_rows_that_share_vectors(rows, d, t):
    import torch
    pkg = _pkg()
    x, res, gamma, beta, out, y, _, stats = _forward(rows, d, t, t, t, seed=3)
    h = pkg.tfl_layernorm_create(d, _code(t), _code(t), _code(t), EPS)
    for _ in range(3):
        x2, r2, st = x.clone(), res.clone(), torch.empty_like(stats)
        pkg.tfl_layernorm_forward(h, rows, P(x2), P(r2), P(gamma), P(beta), P(r2), P(x2), None, P(st), _stream())
        assert torch.equal(r2, out) and torch.equal(x2, y) and torch.equal(st, stats)
        x3, y3 = x.clone(), torch.empty_like(y)
        pkg.tfl_layernorm_forward(h, rows, P(x3), P(res), P(gamma), P(beta), P(x3), P(y3), None, None, _stream())
        assert torch.equal(x3, out) and torch.equal(y3, y)
    pkg.tfl_layernorm_destroy(h)


@pytest.mark.parametrize("rows,d", [(250001, 9), (120001, 17), (45001, 51), (20000, 103), (8000, 255), (1001, 4081)])
@pytest.mark.parametrize("xt,rt", [("bf16", "f32"), ("f16", "f16")])
def test_backward_keeps_rows_without_numbers_to_themselves(rows, d, xt, rt):
    import torch
    pkg = _pkg()
    s, stats, dy, dres, gamma, dx, dsum, _, _ = _backward(rows, d, xt, rt, seed=2)
    bad = sorted({1, rows // 2, rows - 2})
    s2, dy2, dres2 = s.clone(), dy.clone(), dres.clone()
    s2[bad[0]], dy2[bad[1]], dres2[bad[2]] = float("nan"), float("inf"), float("nan")
    dx2, g, b = torch.empty_like(dx), torch.empty_like(gamma), torch.empty_like(gamma)
    h = pkg.tfl_layernorm_create(d, _code(xt), _code(rt), _code(xt), EPS)
    pkg.tfl_layernorm_backward(h, rows, P(s2), P(stats), P(gamma), P(dy2), P(dres2), P(dx2), None, P(g), P(b), _stream())
    torch.cuda.synchronize()
    pkg.tfl_layernorm_destroy(h)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[bad] = False
    assert torch.equal(dx2[keep], dx[keep]) and not dx2[bad].isfinite().all(dim=1).any()


@pytest.mark.parametrize("rows,d", [(250001, 9), (20000, 103), (6000, 513), (2011, 1021)])
def test_buffers_around_rows_that_begin_inside_a_vector_stay_as_they_were(rows, d):
    import torch
    pkg = _pkg()
    s, stats, dy, dres, gamma, dx, *_ = _backward(rows, d, "bf16", "bf16", both=False, seed=7)
    n = rows * d
    h = pkg.tfl_layernorm_create(d, _code("bf16"), _code("bf16"), _code("bf16"), EPS)
    flat = torch.full((n + 64,), 7.0, device="cuda").bfloat16()
    g = torch.full((d + 8,), 7.0, device="cuda")
    b = torch.full((d + 8,), 7.0, device="cuda")
    pkg.tfl_layernorm_backward(h, rows, P(s), P(stats), P(gamma), P(dy), P(dres), P(flat), None, P(g), P(b), _stream())
    assert torch.equal(flat[:n].view(rows, d), dx) and (flat[n:] == 7).all() and (g[d:] == 7).all() and (b[d:] == 7).all()
    flat.fill_(7)
    pkg.tfl_layernorm_forward(h, rows, P(s), None, P(gamma), None, None, P(flat), None, None, _stream())
    assert (flat[n:] == 7).all()
    pkg.tfl_layernorm_destroy(h)
