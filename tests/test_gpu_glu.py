"""The gated feed-forward on the GPU against float64 (oracle/ops.py) on the same inputs.

Bounds per element.  u = eps / 2 of the 16-bit type; products of the operands are exact in
fp32 and a sum over K takes K / 16 + 16 accumulation steps, each off by at most a = 2^-22 of
the absolute sum (the tensor cores' accumulation need not round to nearest):
  g, u     dg = (D / 16 + 16) a |x||Wg|^T, du alike; e4m3 scales: 2 more fp32 roundings
  act      |act'| <= 1.13, |act''| <= 0.8; evaluating it: 2^-20 relative plus 4e-7 (1 + |g|)
           (Abramowitz & Stegun 7.1.26 is good to 1.5e-7 absolute)
  h        1.13 |u| dg + |act| du + 1.13 dg du + the evaluation times |u|, plus u|h|
  dg, du   the same for dh u act' and dh act, plus one rounding of each to the operands' type
  dx, dW   those through the products, their own accumulation, plus u|.|
and half a step at the type's smallest value.  Worst-case sums are wide for long sums, so the
2-norm is held as well: independent roundings of relative size at most u have an rms of at
most u / sqrt 3, two of them (dg or du, and the output) 0.82 u, so 1.2 u with the fp32 terms.
"""
import numpy as np
import pytest

from oracle import ops

pytestmark = pytest.mark.gpu

ACC = 2.0 ** -22
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def _pkg():
    import attention_qkv_gemm_gb300 as pkg
    return pkg


def _type(name):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16}[name]


def _codes(name, act):
    pkg = _pkg()
    return {"f16": pkg.TFL_F16, "bf16": pkg.TFL_BF16}[name], {"silu": pkg.TFL_ACT_SILU, "gelu": pkg.TFL_ACT_GELU}[act]


def _np(t):
    return t.double().cpu().numpy()


def _stream():
    import torch
    return torch.cuda.current_stream().cuda_stream


def _close(u, r, bound, what):
    assert np.isfinite(u).all(), f"{what}: non-finite"
    over = np.abs(u - r) / bound
    assert (over <= 1).all(), (f"{what}: {int((over > 1).sum())} of {u.size} outside, worst {over.max():.3f} of the "
                               f"bound, first at {np.argwhere(over > 1)[:3].tolist()}")


def _norm_close(u, r, limit, what):
    if r.size >= 1000:
        rel = np.linalg.norm(u - r) / np.linalg.norm(r)
        assert rel <= limit, f"{what}: relative 2-norm {rel:.2e} over {limit:.2e}"


def _inputs(tokens, d, f, t, seed):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device="cuda") * std).to(_type(t))  # noqa: E731
    return rnd(tokens, d), rnd(f, d, std=d ** -0.5), rnd(f, d, std=d ** -0.5), rnd(tokens, f)


def _eval(g):
    return 4e-7 * (1 + np.abs(g))


def _forward_bound(x, wg, wu, act, t, extra=0.0):
    g, u = x @ wg.T, x @ wu.T
    k = (x.shape[1] / 16 + 16) * ACC + extra
    dg, du = k * (np.abs(x) @ np.abs(wg).T), k * (np.abs(x) @ np.abs(wu).T)
    a, _ = ops.activation(g, act)
    h = a * u
    return h, (1.13 * np.abs(u) * dg + np.abs(a) * du + 1.13 * dg * du + (2.0 ** -20 * np.abs(a) + _eval(g)) * np.abs(u)
               + U[t] * np.abs(h) + TINY[t])


def _forward(tokens, d, f, t, act, seed=0):
    import torch
    pkg = _pkg()
    x, wg, wu, _ = _inputs(tokens, d, f, t, seed)
    h = torch.full((tokens + 3, f), 7.0, dtype=_type(t), device="cuda")
    code, a = _codes(t, act)
    g = pkg.tfl_glu_create(d, f, code, code, a)
    try:
        pkg.tfl_glu_forward(g, tokens, x.data_ptr(), None, wg.data_ptr(), None, wu.data_ptr(), None, h.data_ptr(),
                            _stream())
        assert pkg.tfl_glu_status(g, _stream()) == 0, pkg.tfl_last_error()
    finally:
        pkg.tfl_glu_destroy(g)
    assert (h[tokens:] == 7).all()  # rows behind the last stay as they were
    return x, wg, wu, h[:tokens]


# one token and few, one value of width, k and columns that no tile divides, tile edges, more
# tiles than the GPU holds at a time
SIZES = [(1, 8, 8), (1, 1024, 520), (3, 72, 16), (8, 264, 40), (9, 1000, 136), (16, 512, 24), (17, 64, 256),
         (33, 136, 1000), (64, 2056, 128), (65, 64, 136), (127, 72, 136), (128, 64, 128), (129, 200, 264),
         (300, 1160, 712), (513, 64, 1000), (4100, 72, 1032),
         # few tiles of long rows: several CTAs share a tile's sum
         (20, 4104, 72), (100, 2056, 520), (128, 1096, 4096), (300, 4096, 264)]


@pytest.mark.parametrize("tokens,d,f", SIZES)
@pytest.mark.parametrize("t,act", [("bf16", "silu"), ("f16", "gelu")])
def test_forward(tokens, d, f, t, act):
    x, wg, wu, h = _forward(tokens, d, f, t, act, seed=tokens + d)
    r, bound = _forward_bound(_np(x), _np(wg), _np(wu), act, t)
    _close(_np(h), r, bound, "h")
    _norm_close(_np(h), r, 0.8 * U[t], "h")


@pytest.mark.parametrize("t,act", [("bf16", "gelu"), ("f16", "silu")])
def test_forward_of_the_other_pairs(t, act):
    for tokens, d, f in ((5, 88, 72), (200, 88, 200)):
        x, wg, wu, h = _forward(tokens, d, f, t, act)
        r, bound = _forward_bound(_np(x), _np(wg), _np(wu), act, t)
        _close(_np(h), r, bound, "h")


@pytest.mark.parametrize("d,f", [(1032, 40), (1160, 72), (1400, 1200), (2048, 5120), (2056, 48), (2600, 64), (4056, 56),
                                 (4096, 1032), (8192, 16), (8200, 16)])
@pytest.mark.parametrize("tokens", [1, 8])
def test_forward_of_a_few_tokens_and_long_rows(tokens, d, f):
    """Rows read in one round of a block's warps, in several, and in several with little in the last."""
    x, wg, wu, h = _forward(tokens, d, f, "bf16", "silu")
    r, bound = _forward_bound(_np(x), _np(wg), _np(wu), "silu", "bf16")
    _close(_np(h), r, bound, "h")


def _rows8(t):
    import torch
    scale = t.abs().amax(dim=1).clamp_min(2.0 ** -100) / 448
    return (t / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn), scale


@pytest.mark.parametrize("tokens,d,f", [(1, 16, 16), (1, 2064, 528), (7, 144, 32), (16, 1024, 48), (33, 144, 272),
                                        (100, 4112, 144), (30, 8192, 544), (200, 1024, 512), (4100, 144, 1040)])
@pytest.mark.parametrize("t,act", [("bf16", "silu"), ("f16", "gelu")])
def test_forward_of_e4m3_operands(tokens, d, f, t, act):
    import torch
    pkg = _pkg()
    gen = torch.Generator(device="cuda").manual_seed(tokens + d)
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=gen, device="cuda") * std  # noqa: E731
    (x, sx), (wg, sg), (wu, su) = _rows8(rnd(tokens, d)), _rows8(rnd(f, d, std=d ** -0.5)), _rows8(rnd(f, d, std=d ** -0.5))
    h = torch.full((tokens + 3, f), 7.0, dtype=_type(t), device="cuda")
    code, a = _codes(t, act)
    g = pkg.tfl_glu_create(d, f, pkg.TFL_E4M3, code, a)
    try:
        pkg.tfl_glu_forward(g, tokens, x.data_ptr(), sx.data_ptr(), wg.data_ptr(), sg.data_ptr(), wu.data_ptr(),
                            su.data_ptr(), h.data_ptr(), _stream())
        assert pkg.tfl_glu_status(g, _stream()) == 0, pkg.tfl_last_error()
    finally:
        pkg.tfl_glu_destroy(g)
    assert (h[tokens:] == 7).all()
    real = [_np(v) * _np(s)[:, None] for v, s in ((x, sx), (wg, sg), (wu, su))]
    r, bound = _forward_bound(*real, act, t, extra=2.0 ** -22)
    _close(_np(h[:tokens]), r, bound, "h")
    _norm_close(_np(h[:tokens]), r, 0.8 * U[t], "h")


def _backward(tokens, d, f, t, act, seed=0, room=5):
    import torch
    pkg = _pkg()
    x, wg, wu, dh = _inputs(tokens, d, f, t, seed)
    dx = torch.full((tokens + 3, d), 7.0, dtype=_type(t), device="cuda")
    dwg, dwu = torch.full_like(wg, 7.0), torch.full_like(wu, 7.0)
    code, a = _codes(t, act)
    g = pkg.tfl_glu_create(d, f, code, code, a, tokens + room)
    try:
        pkg.tfl_glu_backward(g, tokens, x.data_ptr(), wg.data_ptr(), wu.data_ptr(), dh.data_ptr(), dx.data_ptr(),
                             dwg.data_ptr(), dwu.data_ptr(), _stream())
        assert pkg.tfl_glu_status(g, _stream()) == 0, pkg.tfl_last_error()
    finally:
        pkg.tfl_glu_destroy(g)
    assert (dx[tokens:] == 7).all()
    return x, wg, wu, dh, dx[:tokens], dwg, dwu


@pytest.mark.parametrize("tokens,d,f", [(1, 8, 8), (1, 264, 72), (3, 72, 16), (65, 64, 136), (128, 256, 64),
                                        (129, 200, 264), (300, 1160, 712), (1000, 72, 328), (70, 1000, 2568),
                                        (5000, 2056, 72), (20, 520, 2056), (5, 2056, 1032), (200, 264, 4104),
                                        (6000, 136, 200)])
@pytest.mark.parametrize("t,act", [("bf16", "silu"), ("f16", "gelu")])
def test_backward(tokens, d, f, t, act):
    got = _backward(tokens, d, f, t, act, seed=tokens + f)
    x, wg, wu, dh = (_np(v) for v in got[:4])
    dx, dwg, dwu, g, u, dg, du = ops.glu_backward(x, wg, wu, dh, act, return_intermediates=True)
    k = (d / 16 + 16) * ACC
    eg, eu = k * (np.abs(x) @ np.abs(wg).T), k * (np.abs(x) @ np.abs(wu).T)
    a, slope = ops.activation(g, act)
    edg = np.abs(dh) * (np.abs(slope) * eu + 0.8 * (np.abs(u) + eu) * eg + (2.0 ** -19 * np.abs(slope) + _eval(g)) * np.abs(u))
    edu = np.abs(dh) * (1.13 * eg + 2.0 ** -20 * np.abs(a) + _eval(g))
    edg, edu = edg + U[t] * np.abs(dg) + TINY[t], edu + U[t] * np.abs(du) + TINY[t]
    bx = edg @ np.abs(wg) + edu @ np.abs(wu) + (f / 8 + 16) * ACC * (np.abs(dg) @ np.abs(wg) + np.abs(du) @ np.abs(wu))
    _close(_np(got[4]), dx, 1.01 * bx + U[t] * np.abs(dx) + TINY[t], "dx")
    _norm_close(_np(got[4]), dx, 1.2 * U[t], "dx")
    for u16, r, e, v, what in ((got[5], dwg, edg, dg, "dwg"), (got[6], dwu, edu, du, "dwu")):
        bound = e.T @ np.abs(x) + (tokens / 16 + 16) * ACC * (np.abs(v).T @ np.abs(x))
        _close(_np(u16), r, 1.01 * bound + U[t] * np.abs(r) + TINY[t], what)
        _norm_close(_np(u16), r, 1.2 * U[t], what)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward_is_the_forwards_difference_quotient(act):
    """Along a direction in x, from the kernel's own h: each h is off by its bound, so the
    quotient of L = sum(dh h) by the bounds' sum over h; the h^2 term is the reference's own."""
    import torch
    pkg = _pkg()
    tokens, d, f, t = 6, 64, 48, "f16"
    x, wg, wu, dh, dx, _, _ = _backward(tokens, d, f, t, act, seed=8)
    v = torch.randn((tokens, d), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").half()
    step = 2.0 ** -3
    code, a = _codes(t, act)
    g = pkg.tfl_glu_create(d, f, code, code, a)

    def loss(sign):
        p, h = (x + sign * step * v).contiguous(), torch.empty_like(dh)
        pkg.tfl_glu_forward(g, tokens, p.data_ptr(), None, wg.data_ptr(), None, wu.data_ptr(), None, h.data_ptr(),
                            _stream())
        r, b = _forward_bound(_np(p), _np(wg), _np(wu), act, t)
        return p, np.sum(_np(h) * _np(dh)), np.sum(r * _np(dh)), np.sum(b * np.abs(_np(dh)))

    up, down = loss(1), loss(-1)
    pkg.tfl_glu_destroy(g)
    moved = _np(up[0]) - _np(down[0])  # the points as fp16 holds them
    q, qref, noise = (up[1] - down[1]) / 2, (up[2] - down[2]) / 2, (up[3] + down[3]) / 2
    assert abs(q - qref) <= noise
    ref = ops.glu_backward(_np(x), _np(wg), _np(wu), _np(dh), act)[0]
    along, ref_along = np.sum(_np(dx) * moved) / 2, np.sum(ref * moved) / 2
    assert abs(along - ref_along) <= 4 * U[t] * np.sum(np.abs(ref * moved)) / 2 + 1e-3
    assert abs(along - q) <= noise + abs(qref - ref_along) + 4 * U[t] * np.sum(np.abs(ref * moved)) / 2 + 1e-3


def test_rows_do_not_affect_one_another():
    import torch
    pkg = _pkg()
    for tokens in (4, 150):
        x, wg, wu, dh = _inputs(tokens, 128, 136, "bf16", 2)
        code, a = _codes("bf16", "silu")
        g = pkg.tfl_glu_create(128, 136, code, code, a, tokens)
        out = []
        for bad in (False, True):
            if bad:
                x[1, 3] = float("nan")
                x[2, 5] = float("inf")
            h, dx = torch.empty_like(dh), torch.empty_like(x)
            dwg, dwu = torch.empty_like(wg), torch.empty_like(wu)
            pkg.tfl_glu_forward(g, tokens, x.data_ptr(), None, wg.data_ptr(), None, wu.data_ptr(), None, h.data_ptr(),
                                _stream())
            pkg.tfl_glu_backward(g, tokens, x.data_ptr(), wg.data_ptr(), wu.data_ptr(), dh.data_ptr(), dx.data_ptr(),
                                 dwg.data_ptr(), dwu.data_ptr(), _stream())
            out.append((h, dx))
        assert pkg.tfl_glu_status(g, _stream()) == 0
        pkg.tfl_glu_destroy(g)
        keep = [i for i in range(tokens) if i not in (1, 2)]
        for clean, dirty in zip(*out):
            assert torch.equal(clean[keep], dirty[keep]) and dirty[1].isnan().all()


def test_large_gates_saturate():
    """Gates of +-60: SiLU and GELU are the identity and zero there (e^-60 is below any bound)."""
    import torch
    pkg = _pkg()
    x = torch.zeros(2, 16, device="cuda").half()
    x[0, 0], x[1, 0], x[:, 1] = 60.0, -60.0, 1.0
    wg, wu = torch.zeros(16, 16, device="cuda").half(), torch.zeros(16, 16, device="cuda").half()
    wg[:, 0], wu[:, 1] = 1.0, 2.0
    for act in ("silu", "gelu"):
        code, a = _codes("f16", act)
        g = pkg.tfl_glu_create(16, 16, code, code, a)
        h = torch.empty(2, 16, device="cuda").half()
        pkg.tfl_glu_forward(g, 2, x.data_ptr(), None, wg.data_ptr(), None, wu.data_ptr(), None, h.data_ptr(), _stream())
        torch.cuda.synchronize()
        pkg.tfl_glu_destroy(g)
        assert (h[0] == 120).all() and (h[1] == 0).all()


def test_same_bits_every_time_captured_and_replayed_on_another_stream():
    import torch
    pkg = _pkg()
    tokens, d, f = 700, 320, 456
    x, wg, wu, dh, dx, dwg, dwu = _backward(tokens, d, f, "bf16", "silu", seed=3)
    code, a = _codes("bf16", "silu")
    op = pkg.tfl_glu_create(d, f, code, code, a, tokens)
    h, h2 = torch.empty_like(dh), torch.empty_like(dh)
    out = [torch.empty_like(v) for v in (dx, dwg, dwu)]
    pkg.tfl_glu_forward(op, tokens, x.data_ptr(), None, wg.data_ptr(), None, wu.data_ptr(), None, h.data_ptr(), _stream())
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=st):
        pkg.tfl_glu_forward(op, tokens, x.data_ptr(), None, wg.data_ptr(), None, wu.data_ptr(), None, h2.data_ptr(),
                            st.cuda_stream)
        pkg.tfl_glu_backward(op, tokens, x.data_ptr(), wg.data_ptr(), wu.data_ptr(), dh.data_ptr(), out[0].data_ptr(),
                             out[1].data_ptr(), out[2].data_ptr(), st.cuda_stream)
    for _ in range(2):
        for v in (h2, *out):
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h2, h)
        for v, r in zip(out, (dx, dwg, dwu)):
            assert torch.equal(v, r)
    assert pkg.tfl_glu_status(op, _stream()) == 0
    pkg.tfl_glu_destroy(op)


def test_forwards_of_one_handle_may_overlap():
    import torch
    pkg = _pkg()
    code, a = _codes("bf16", "silu")
    op = pkg.tfl_glu_create(256, 512, code, code, a)
    calls = []
    for i in range(6):
        x, wg, wu, dh = _inputs(3 if i % 2 else 1500, 256, 512, "bf16", i)
        ref, h = torch.empty_like(dh), torch.empty_like(dh)
        pkg.tfl_glu_forward(op, x.shape[0], x.data_ptr(), None, wg.data_ptr(), None, wu.data_ptr(), None,
                            ref.data_ptr(), _stream())
        calls.append((x, wg, wu, ref, h, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for x, wg, wu, _, h, st in calls:
        pkg.tfl_glu_forward(op, x.shape[0], x.data_ptr(), None, wg.data_ptr(), None, wu.data_ptr(), None, h.data_ptr(),
                            st.cuda_stream)
    torch.cuda.synchronize()
    for _, _, _, ref, h, _ in calls:
        assert torch.equal(ref, h)
    pkg.tfl_glu_destroy(op)


def test_no_tokens():
    import torch
    pkg = _pkg()
    op = pkg.tfl_glu_create(64, 64, 2, 2, 0, 4)
    dwg, dwu = torch.ones(64, 64, device="cuda").bfloat16(), torch.ones(64, 64, device="cuda").bfloat16()
    pkg.tfl_glu_forward(op, 0, None, None, None, None, None, None, None, _stream())
    pkg.tfl_glu_backward(op, 0, None, None, None, None, None, dwg.data_ptr(), dwu.data_ptr(), _stream())
    torch.cuda.synchronize()
    assert (dwg == 0).all() and (dwu == 0).all()
    pkg.tfl_glu_destroy(op)


def test_refusals():
    import torch
    pkg = _pkg()
    op = pkg.tfl_glu_create(64, 128, 2, 2, 0, 4)
    q = pkg.tfl_glu_create(64, 128, 3, 2, 0)
    x, wg, wu, dh = _inputs(8, 64, 128, "bf16", 0)
    h, dx, dwg, dwu = torch.empty_like(dh), torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    s = torch.ones(256, device="cuda")
    P = lambda t: t.data_ptr()  # noqa: E731

    def refused(fn, *args, code=pkg.TFL_ERR_INVALID_ARG):
        with pytest.raises(pkg.TflError) as e:
            fn(*args, _stream())
        assert e.value.code == code and str(e.value)

    f, b = pkg.tfl_glu_forward, pkg.tfl_glu_backward
    good = [P(x), None, P(wg), None, P(wu), None, P(h)]
    refused(f, None, 4, *good)
    refused(f, op, -1, *good)
    refused(f, op, 2 ** 31, *good)
    for i in (0, 2, 4, 6):
        refused(f, op, 4, *good[:i], None, *good[i + 1:])
        refused(f, op, 4, *good[:i], good[i] + 8, *good[i + 1:])
    refused(f, op, 4, P(x), P(s), P(wg), P(s), P(wu), P(s), P(h))
    refused(f, q, 4, *good)
    refused(f, q, 4, P(x), P(s), P(wg), P(s) + 4, P(wu), P(s), P(h))
    refused(f, op, 4, *good[:6], P(x))
    refused(f, op, 4, *good[:6], P(wu) + 128)
    good = [P(x), P(wg), P(wu), P(dh), P(dx), P(dwg), P(dwu)]
    refused(b, None, 4, *good)
    refused(b, op, 5, *good)                                # more than it has room for
    for i in range(7):
        refused(b, op, 4, *good[:i], None, *good[i + 1:])
        refused(b, op, 4, *good[:i], good[i] + 8, *good[i + 1:])
    refused(b, op, 4, *good[:4], P(x), *good[5:])
    refused(b, op, 4, *good[:5], P(dwu), P(dwu))
    refused(b, op, 4, *good[:6], P(wu))
    refused(b, q, 4, *good, code=pkg.TFL_ERR_UNSUPPORTED)
    assert pkg.tfl_glu_status(op, _stream()) == 0
    pkg.tfl_glu_destroy(op)
    pkg.tfl_glu_destroy(q)
