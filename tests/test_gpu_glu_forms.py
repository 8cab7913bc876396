"""Every form of the gated feed-forward's kernels in every mode, against float64 on the GPU.

The bounds are those of test_gpu_glu.py, element by element and on the 2-norm.
"""
import pytest

from tests import glu_forms
from tests.test_gpu_glu import ACC, TINY, U, _backward, _codes, _forward, _pkg, _rows8, _stream, _type

pytestmark = pytest.mark.gpu


def _activation(g, kind):
    import torch
    if kind == "silu":
        p = torch.sigmoid(g)
        return g * p, p + g * p * (1 - p)
    cdf = 0.5 * (1 + torch.special.erf(g * 0.5 ** 0.5))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * 0.3989422804014327


def _eval(g):
    return 4e-7 * (1 + g.abs())


def _close(u, r, bound, limit, what):
    u = u.double()
    assert u.isfinite().all(), f"{what}: non-finite"
    over = (u - r).abs() / bound
    assert bool((over <= 1).all()), f"{what}: {int((over > 1).sum())} of {u.numel()} outside, worst {float(over.max()):.3f} of the bound"
    rel = float((u - r).norm() / r.norm())
    assert rel <= limit, f"{what}: relative 2-norm {rel:.2e} over {limit:.2e}"


def _check_forward(x, wg, wu, h, act, t, extra=0.0):
    g, u = x @ wg.t(), x @ wu.t()
    k = (x.shape[1] / 16 + 16) * ACC + extra
    dg, du = k * (x.abs() @ wg.abs().t()), k * (x.abs() @ wu.abs().t())
    a, _ = _activation(g, act)
    bound = (1.13 * u.abs() * dg + a.abs() * du + 1.13 * dg * du + (2.0 ** -20 * a.abs() + _eval(g)) * u.abs()
             + U[t] * (a * u).abs() + TINY[t])
    _close(h, a * u, bound, 0.8 * U[t], "h")


KINDS = [("bf16", "silu"), ("f16", "gelu")]


def test_the_sizes_reach_every_form_on_this_gpu():
    assert glu_forms.reached() == glu_forms.WANTED


@pytest.mark.parametrize("tokens,d,f", glu_forms.FORWARD)
@pytest.mark.parametrize("t,act", KINDS)
def test_forward(tokens, d, f, t, act):
    x, wg, wu, h = _forward(tokens, d, f, t, act, seed=tokens + d)
    _check_forward(x.double(), wg.double(), wu.double(), h, act, t)


@pytest.mark.parametrize("tokens,d,f", glu_forms.E4M3)
@pytest.mark.parametrize("t,act", KINDS)
def test_forward_of_e4m3_operands(tokens, d, f, t, act):
    import torch
    pkg = _pkg()
    gen = torch.Generator(device="cuda").manual_seed(tokens + d)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    ops8 = [_rows8(rnd(tokens, d) * 2.0 ** torch.randint(-8, 6, (tokens, 1), generator=gen, device="cuda")),
            _rows8(rnd(f, d) * d ** -0.5), _rows8(rnd(f, d) * d ** -0.5)]
    h = torch.full((tokens + 3, f), 7.0, dtype=_type(t), device="cuda")
    code, a = _codes(t, act)
    g = pkg.tfl_glu_create(d, f, pkg.TFL_E4M3, code, a)
    try:
        pkg.tfl_glu_forward(g, tokens, *(v.data_ptr() for pair in ops8 for v in pair), h.data_ptr(), _stream())
        assert pkg.tfl_glu_status(g, _stream()) == 0, pkg.tfl_last_error()
    finally:
        pkg.tfl_glu_destroy(g)
    assert (h[tokens:] == 7).all()
    _check_forward(*(v.double() * s.double()[:, None] for v, s in ops8), h[:tokens], act, t, extra=2.0 ** -22)


@pytest.mark.parametrize("tokens,d,f", glu_forms.BACKWARD)
@pytest.mark.parametrize("t,act", KINDS)
def test_backward(tokens, d, f, t, act):
    import torch
    got = _backward(tokens, d, f, t, act, seed=tokens + f)
    x, wg, wu, dh = (v.double() for v in got[:4])
    g, u = x @ wg.t(), x @ wu.t()
    a, slope = _activation(g, act)
    dg, du = dh * u * slope, dh * a
    k = (d / 16 + 16) * ACC
    eg, eu = k * (x.abs() @ wg.abs().t()), k * (x.abs() @ wu.abs().t())
    edg = dh.abs() * (slope.abs() * eu + 0.8 * (u.abs() + eu) * eg + (2.0 ** -19 * slope.abs() + _eval(g)) * u.abs())
    edu = dh.abs() * (1.13 * eg + 2.0 ** -20 * a.abs() + _eval(g))
    edg, edu = edg + U[t] * dg.abs() + TINY[t], edu + U[t] * du.abs() + TINY[t]
    dx = dg @ wg + du @ wu
    bx = edg @ wg.abs() + edu @ wu.abs() + (f / 8 + 16) * ACC * (dg.abs() @ wg.abs() + du.abs() @ wu.abs())
    _close(got[4], dx, 1.01 * bx + U[t] * dx.abs() + TINY[t], 1.2 * U[t], "dx")
    for out, e, v, what in ((got[5], edg, dg, "dwg"), (got[6], edu, du, "dwu")):
        r = v.t() @ x
        bound = e.t() @ x.abs() + (tokens / 16 + 16) * ACC * (v.abs().t() @ x.abs())
        _close(out, r, 1.01 * bound + U[t] * r.abs() + TINY[t], 1.2 * U[t], what)
    del eg, eu, edg, edu
    torch.cuda.empty_cache()


@pytest.mark.parametrize("tokens,d,f", sorted(set(glu_forms.FORWARD + glu_forms.BACKWARD)))
def test_rows_do_not_affect_one_another(tokens, d, f):
    """Rows with no numbers and infinities at the ends of tiles: the other rows keep their bits, forward and dx."""
    import torch
    from tests.test_gpu_glu import _inputs
    pkg = _pkg()
    x, wg, wu, dh = _inputs(tokens, d, f, "bf16", 4)
    bad = sorted({1, min(127, tokens - 1), tokens // 2, tokens - 2})
    code, a = _codes("bf16", "silu")
    op = pkg.tfl_glu_create(d, f, code, code, a, tokens)
    out = []
    for dirty in (False, True):
        if dirty:
            x[bad, 3] = float("nan")
            x[bad[0], 5] = float("inf")
        h, dx, dwg, dwu = torch.empty_like(dh), torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
        P = lambda t: t.data_ptr()  # noqa: E731
        pkg.tfl_glu_forward(op, tokens, P(x), None, P(wg), None, P(wu), None, P(h), _stream())
        pkg.tfl_glu_backward(op, tokens, P(x), P(wg), P(wu), P(dh), P(dx), P(dwg), P(dwu), _stream())
        out.append((h, dx))
    assert pkg.tfl_glu_status(op, _stream()) == 0
    pkg.tfl_glu_destroy(op)
    keep = torch.ones(tokens, dtype=torch.bool, device="cuda")
    keep[bad] = False
    for clean, dirty in zip(*out):
        assert torch.equal(clean[keep], dirty[keep]) and clean.isfinite().all() and dirty[bad].isnan().all()


@pytest.mark.parametrize("tokens,d,f", glu_forms.BACKWARD)
def test_same_bits_every_time_and_in_a_graph(tokens, d, f):
    """Forward and backward one behind the other, twice, and captured and replayed on another stream."""
    import torch
    from tests.test_gpu_glu import _inputs
    pkg = _pkg()
    x, wg, wu, dh = _inputs(tokens, d, f, "f16", 5)
    code, a = _codes("f16", "gelu")
    op = pkg.tfl_glu_create(d, f, code, code, a, tokens)
    out = torch.empty_like(dh), torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    P = lambda t: t.data_ptr()  # noqa: E731

    def step(st):
        pkg.tfl_glu_forward(op, tokens, P(x), None, P(wg), None, P(wu), None, P(out[0]), st)
        pkg.tfl_glu_backward(op, tokens, P(x), P(wg), P(wu), P(dh), P(out[1]), P(out[2]), P(out[3]), st)

    step(_stream())
    ref = [v.clone() for v in out]
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=st):
        step(st.cuda_stream)
    for again in (lambda: step(_stream()), graph.replay, graph.replay):
        for v in out:
            v.zero_()
        again()
        torch.cuda.synchronize()
        assert all(torch.equal(v, r) for v, r in zip(out, ref))
    assert pkg.tfl_glu_status(op, _stream()) == 0
    pkg.tfl_glu_destroy(op)
