"""Layer norm on the GPU against float64 (oracle/ops.py) on the same inputs.

Bounds, with u = eps / 2 of the stored type, e = 2^-24 (fp32's half step), t = (s - m) r, and
n = max(32, D / 256 + 8) + 42 the most terms that a row's sum adds in a row (a thread's own, then
the threads'):
  res_out  one fp32 addition and one rounding: u|s| + e|s|
  s - m    each s is off by e|s| (its addition), so their mean by e mean|s|; the kernel's first mean
           drops out, since it subtracts the centred values' own mean, a sum good to
           (n + 2) e mean|s - m|; two subtractions, e|s - m| each, of values that may be larger by
           the first mean's error, n e mean|s|:
           c = e (|s| + mean|s|) + 3 e|s - m| + (n + 2) e mean|s - m|   (terms of e^2 n^2 left to the
           rounding up of n)
  var      mean(|s - m| 2 c) and its own sum, (n + 3) e var; so r is off by
           q = mean(|s - m| c) / (var + eps) + (n / 2 + 7) e relative, rsqrtf's 4 e among them
  y        |gamma| (r c + |t| (q + 2 e)) + 2 e (|y| + |beta|), plus the rounding u|y|
  m        e mean|s| + (n + 2) e mean|s - m| + 2 e|m|;   r  q r
  scale    the row's largest error of y / 448, and 3 e for the division
  e4m3     the stored value times the scale: half a step of e4m3, 2^-4 |y| + 2^-10 scale (below
           e4m3's normal range), twice y's own error, and the scale's relative error times |y|
  ds       from the rows' statistics as given: with w = |dres| + r (|a| + mean|a| + |t| mean|a t|),
           (n + 12) e w for the two sums and the products, plus u|ds|
  dgamma   at most rows / 152 + 96 terms in a row: (that + 4) e sum|dy t|;  dbeta  the same of sum|dy|
and half a step at the type's smallest value everywhere.
"""
import numpy as np
import pytest

from oracle import ops
from tests.test_gpu_rmsnorm import E, TYPES, _close, _code, _n, _np, _pkg, _randn, _stream, _tiny, _type, _u

pytestmark = pytest.mark.gpu

EPS = 1e-5


def _bounds(s, gamma, beta, eps):
    """Errors of y, of the mean and (relative) of r, before y's rounding."""
    n = _n(s.shape[1])
    m = s.mean(axis=1, keepdims=True)
    d, size = np.abs(s - m), np.abs(s).mean(axis=1, keepdims=True)
    v = (d * d).mean(axis=1, keepdims=True) + eps
    spread = d.mean(axis=1, keepdims=True)
    c = E * (np.abs(s) + size) + 3 * E * d + (n + 2) * E * spread
    q = (d * c).mean(axis=1, keepdims=True) / v + (n / 2 + 7) * E
    r = 1 / np.sqrt(v)
    y = (s - m) * r * gamma + beta
    own = np.abs(gamma) * (r * c + d * r * (q + 2 * E)) + 2 * E * (np.abs(y) + np.abs(beta))
    return own, (E * size + (n + 2) * E * spread + 2 * E * np.abs(m))[:, 0], q[:, 0]


def _forward(rows, d, xt, rt, yt, with_res=True, store=True, with_beta=True, mean=1.0, seed=0, offset=0, eps=EPS):
    """Runs the forward; `offset` shifts every buffer but stats by that many elements (unaligned)."""
    import torch
    pkg = _pkg()
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def place(t):
        flat = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")[offset:]
        flat.copy_(t.reshape(-1))
        return flat.view(t.shape)

    x = place((_randn(gen, (rows, d), "f32") + mean).to(_type(xt)))
    res = place(_randn(gen, (rows, d), rt, 2.0)) if with_res else None
    gamma = place(1 + _randn(gen, (d,), "f32", 0.2))
    beta = place(_randn(gen, (d,), "f32", 0.2)) if with_beta else None
    out = place(torch.full((rows, d), 7.0, dtype=_type(rt), device="cuda")) if store else None
    y = place(torch.zeros((rows, d), device="cuda").to(_type(yt)))
    scale = place(torch.full((rows,), -1.0, device="cuda")) if yt == "e4m3" else None
    stats = torch.full((rows, 2), -1.0, device="cuda") if store else None
    h = pkg.tfl_layernorm_create(d, _code(xt), _code(rt), _code(yt), eps)
    P = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    try:
        pkg.tfl_layernorm_forward(h, rows, P(x), P(res), P(gamma), P(beta), P(out), P(y), P(scale), P(stats), _stream())
        torch.cuda.synchronize()
    finally:
        pkg.tfl_layernorm_destroy(h)
    return x, res, gamma, beta, out, y, scale, stats


def _check_forward(rows, d, xt, rt, yt, got, eps=EPS):
    x, res, gamma, beta, out, y, scale, stats = got
    eps = float(np.float32(eps))
    gamma, beta = _np(gamma), np.zeros(d) if beta is None else _np(beta)
    s, ref, m, r = ops.layer_norm(_np(x), None if res is None else _np(res), gamma, beta, eps)
    own, own_m, own_r = _bounds(s, gamma, beta, eps)
    if out is not None:
        _close(_np(out), s, (_u(rt) + E) * np.abs(s) + _tiny(rt), "res_out")
    if stats is not None:
        _close(_np(stats)[:, 0], m, own_m + _tiny("f32"), "mean")
        _close(_np(stats)[:, 1], r, own_r * r, "1 / sqrt(var + eps)")
    if yt != "e4m3":
        _close(_np(y), ref, own + _u(yt) * np.abs(ref) + _tiny(yt), "y")
        return
    rs = ops.row_scale(ref)
    own_s = own.max(axis=1) / 448 + 3 * E * rs
    _close(_np(scale), rs, own_s, "scale")
    _close(_np(y) * _np(scale)[:, None], ref,
           2.0 ** -4 * np.abs(ref) + 2.0 ** -10 * rs[:, None] + 2 * own + (own_s / rs)[:, None] * np.abs(ref), "e4m3 y")


@pytest.mark.parametrize("xt,rt,yt", TYPES)
def test_forward_of_every_type(xt, rt, yt):
    for rows, d in ((1, 1024), (37, 264), (5, 8)):
        _check_forward(rows, d, xt, rt, yt, _forward(rows, d, xt, rt, yt, seed=d))


# one value, less than a warp, ragged vectors, one warp and more a row, the widest row kept in
# registers and the first that is not, widths no vector divides
@pytest.mark.parametrize("rows,d", [(1, 1), (3, 7), (9, 64), (300, 72), (33, 256), (17, 512), (12, 1000), (1000, 1024),
                                    (3, 1032), (5, 4096), (3, 8200), (2, 32768), (2, 32776), (4, 1001), (3, 1025),
                                    (70, 4095), (2, 4097), (30, 8191), (3, 8193), (2, 50001)])
@pytest.mark.parametrize("xt,rt,yt", [("bf16", "f32", "e4m3"), ("f16", "f16", "f16"), ("f32", "f32", "f32")])
def test_forward_of_every_width(rows, d, xt, rt, yt):
    _check_forward(rows, d, xt, rt, yt, _forward(rows, d, xt, rt, yt, seed=rows + d))


@pytest.mark.parametrize("rows,d", [(351000, 8), (45001, 72), (22000, 256), (11003, 400), (5603, 1000), (1501, 4096),
                                    (2500, 8193)])
@pytest.mark.parametrize("xt,rt,yt", [("bf16", "f32", "e4m3"), ("f16", "f16", "f16"), ("f32", "f32", "f32")])
def test_forward_of_many_rows(rows, d, xt, rt, yt):
    _check_forward(rows, d, xt, rt, yt, _forward(rows, d, xt, rt, yt, seed=d))


# rows that begin inside a 16-byte vector: every shift, widths around those where the thread groups change, one
# row a group and several turns of the blocks
@pytest.mark.parametrize("d", [9, 10, 12, 15, 17, 250, 251, 1001, 1002, 1004, 2033, 2034, 2035, 4081, 4082, 4083])
@pytest.mark.parametrize("xt,rt,yt", [("bf16", "f32", "e4m3"), ("f16", "f16", "f16"), ("f32", "f32", "bf16"), ("f16", "f16", "e4m3")])
def test_forward_of_rows_that_begin_inside_a_vector(d, xt, rt, yt):
    for rows in (1, 2, 9, 160, 6007 if d < 2000 else 1501, 40009 if d < 20 else 303):
        _check_forward(rows, d, xt, rt, yt, _forward(rows, d, xt, rt, yt, rows != 9, rows != 2, rows != 160, seed=rows + d))


@pytest.mark.parametrize("with_res,store,with_beta", [(False, True, True), (True, False, True), (True, True, False),
                                                      (False, False, False)])
@pytest.mark.parametrize("rows,d", [(6, 256), (6, 129), (2001, 1024), (3, 9001)])
def test_forward_without_residual_stores_or_beta(rows, d, with_res, store, with_beta):
    for yt in ("bf16", "e4m3"):
        _check_forward(rows, d, "bf16", "f32", yt, _forward(rows, d, "bf16", "f32", yt, with_res, store, with_beta))


@pytest.mark.parametrize("offset", [1, 4])
def test_forward_of_unaligned_buffers(offset):
    _check_forward(7, 512, "bf16", "f32", "e4m3", _forward(7, 512, "bf16", "f32", "e4m3", offset=offset))
    _check_forward(7, 512, "f16", "f16", "f16", _forward(7, 512, "f16", "f16", "f16", offset=offset))


@pytest.mark.parametrize("rows,d", [(40, 256), (40, 1024), (40, 1001), (3, 9001)])
@pytest.mark.parametrize("mean", [300.0, 3e5])
def test_a_large_mean_costs_only_what_fp32_loses_of_the_differences(rows, d, mean):
    """mean(s^2) - mean(s)^2 would have nothing left of a variance of 5 beside 3e5^2 (2^-24 of it is 5364)."""
    got = _forward(rows, d, "f32", "f32", "f32", mean=mean, seed=2)
    _check_forward(rows, d, "f32", "f32", "f32", got)
    # the input's own rounding is gone without an addition: s - m is then good to the sums' rounding
    got = _forward(rows, d, "f32", "f32", "f32", with_res=False, mean=mean, seed=2)
    s, ref, m, r = ops.layer_norm(_np(got[0]), None, _np(got[2]), _np(got[3]), EPS)
    # s - m0 is a difference of nearby numbers (exact); m0's error, below n e |m|, is taken out again to (n + 6) e of itself
    n = _n(d)
    dev = np.abs(s - m[:, None])
    c = 3 * E * dev + (n + 6) * E * (dev.mean(axis=1) + n * E * np.abs(m))[:, None] + 3 * E * n * E * np.abs(m)[:, None]
    q = (dev * c).mean(axis=1) * r ** 2 + (n / 2 + 7) * E
    bound = np.abs(_np(got[2])) * (r[:, None] * c + dev * r[:, None] * (q[:, None] + 2 * E)) + 3 * E * (np.abs(ref) + 1)
    _close(_np(got[5]), ref, bound, "y of exact differences")


@pytest.mark.parametrize("rows,d", [(5, 8), (700, 1024), (5, 103), (3, 8193), (3, 16384)])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_constant_rows_give_beta(rows, d, xt):
    """The centred values of a constant row c are c's rounding in the sums, at most n e|c|; their own mean
    is taken out again to (n + 3) e of that, and eps = 1e-5 multiplies what is left by 316."""
    import torch
    pkg = _pkg()
    x = (torch.arange(rows, device="cuda")[:, None] * 1.7 - 2).expand(rows, d).contiguous().to(_type(xt))
    gamma, beta = torch.ones(d, device="cuda"), torch.linspace(-1, 1, d, device="cuda")
    y, stats = torch.empty((rows, d), device="cuda"), torch.empty((rows, 2), device="cuda")
    yt = "f32" if xt == "f32" else "bf16"
    y = y.to(_type(yt))
    h = pkg.tfl_layernorm_create(d, _code(xt), _code(xt), _code(yt), EPS)
    pkg.tfl_layernorm_forward(h, rows, x.data_ptr(), None, gamma.data_ptr(), beta.data_ptr(), None, y.data_ptr(), None,
                              stats.data_ptr(), _stream())
    torch.cuda.synchronize()
    pkg.tfl_layernorm_destroy(h)
    n, c = _n(d), np.abs(_np(x))
    _close(_np(y), np.broadcast_to(_np(beta), (rows, d)),
           317 * (n * E) * ((n + 6) * E) * c + (_u(yt) + 2 * E) * np.abs(_np(beta)) + 1e-30, "y")
    _close(_np(stats)[:, 0], _np(x)[:, 0], 3 * E * c[:, 0] + 1e-30, "mean")


@pytest.mark.parametrize("rows,d", [(6, 8), (700, 1024), (6, 103), (6, 5001), (6, 8193), (6, 16384)])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_e4m3_of_rows_below_the_least_scale(rows, d, xt):
    """gamma of 2^-110 puts every |y| below 2^-100 (|t| <= sqrt(16384) = 2^7), beside rows of zeros."""
    import torch
    pkg = _pkg()
    gen = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn((rows, d), generator=gen, device="cuda")
    x[1::6] = 0
    x, gamma = x.to(_type(xt)), torch.full((d,), 2.0 ** -110, device="cuda")
    y, scale = torch.zeros((rows, d), device="cuda").to(_type("e4m3")), torch.zeros(rows, device="cuda")
    h = pkg.tfl_layernorm_create(d, _code(xt), _code(xt), _code("e4m3"), EPS)
    pkg.tfl_layernorm_forward(h, rows, x.data_ptr(), None, gamma.data_ptr(), None, None, y.data_ptr(), scale.data_ptr(),
                              None, _stream())
    torch.cuda.synchronize()
    pkg.tfl_layernorm_destroy(h)
    assert (_np(y)[1::6] == 0).all()
    assert (_np(scale) == np.float32(2.0 ** -100) / np.float32(448)).all()
    ref = ops.layer_norm(_np(x), None, _np(gamma), None, EPS)[1] / (2.0 ** -100 / 448)
    own = _bounds(_np(x), _np(gamma), np.zeros(d), EPS)[0] / (2.0 ** -100 / 448)
    _close(_np(y), ref, 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 + 2 * own + 4 * E * np.abs(ref), "y")


@pytest.mark.parametrize("rows,d", [(40, 512), (40, 515), (11003, 512), (11003, 515), (3000, 2500), (3, 9001)])
def test_forward_in_place_equals_out_of_place(rows, d):
    import torch
    pkg = _pkg()
    x, res, gamma, beta, out, y, _, stats = _forward(rows, d, "bf16", "bf16", "bf16", seed=3)
    h = pkg.tfl_layernorm_create(d, _code("bf16"), _code("bf16"), _code("bf16"), EPS)
    P = lambda t: t.data_ptr()  # noqa: E731
    try:
        x2, r2, st = x.clone(), res.clone(), torch.empty_like(stats)
        pkg.tfl_layernorm_forward(h, rows, P(x2), P(r2), P(gamma), P(beta), P(r2), P(x2), None, P(st), _stream())
        assert torch.equal(r2, out) and torch.equal(x2, y) and torch.equal(st, stats)
        x3, y3 = x.clone(), torch.empty_like(y)
        pkg.tfl_layernorm_forward(h, rows, P(x3), P(res), P(gamma), P(beta), P(x3), P(y3), None, None, _stream())
        assert torch.equal(x3, out) and torch.equal(y3, y)
    finally:
        pkg.tfl_layernorm_destroy(h)


@pytest.mark.parametrize("rows,d", [(6, 256), (6, 255), (22000, 256), (22000, 255), (9000, 1001), (6, 9001), (700, 4099), (400, 8177)])
def test_rows_of_nan_and_infinity_stay_their_own(rows, d):
    import torch
    pkg = _pkg()
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = _randn(gen, (rows, d), "bf16")
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    gamma = torch.ones(d, device="cuda")
    for yt in ("bf16", "e4m3"):
        y = torch.zeros((rows, d), device="cuda").to(_type(yt))
        scale, stats = torch.zeros(rows, device="cuda"), torch.zeros(rows, 2, device="cuda")
        h = pkg.tfl_layernorm_create(d, _code("bf16"), _code("bf16"), _code(yt), EPS)
        pkg.tfl_layernorm_forward(h, rows, x.data_ptr(), None, gamma.data_ptr(), None, None, y.data_ptr(),
                                  scale.data_ptr() if yt == "e4m3" else None, stats.data_ptr(), _stream())
        torch.cuda.synchronize()
        pkg.tfl_layernorm_destroy(h)
        f = y.float()
        others = [0, 1, *range(4, rows)]
        assert f[2].isnan().all() and f[3].isnan().all() and stats[2].isnan().all() and stats[3, 1].isnan()
        assert f[others].isfinite().all() and stats[others].isfinite().all()
        if yt == "e4m3":
            assert scale[2].isnan() and scale[3].isnan() and scale[others].isfinite().all()


def _backward(rows, d, xt, rt, with_dres=True, both=True, with_beta=True, seed=0):
    import torch
    pkg = _pkg()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = (_randn(gen, (rows, d), "f32", 2.0) + 1).to(_type(rt))
    dy = _randn(gen, (rows, d), xt)
    dres = _randn(gen, (rows, d), rt) if with_dres else None
    gamma = 1 + _randn(gen, (d,), "f32", 0.2)
    var, m = torch.var_mean(s.double(), dim=1, correction=0)
    stats = torch.stack([m, (var + EPS) ** -0.5], dim=1).float()
    dx = torch.full((rows, d), 7.0, dtype=_type(xt), device="cuda")
    dsum = torch.full((rows, d), 7.0, dtype=_type(rt), device="cuda") if both else None
    dgamma, dbeta = torch.full((d,), 7.0, device="cuda"), torch.full((d,), 7.0, device="cuda") if with_beta else None
    h = pkg.tfl_layernorm_create(d, _code(xt), _code(rt), _code(xt), EPS)
    P = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    try:
        for _ in range(2):  # the second call finds the first one's scratch
            pkg.tfl_layernorm_backward(h, rows, P(s), P(stats), P(gamma), P(dy), P(dres), P(dx), P(dsum), P(dgamma),
                                       P(dbeta), _stream())
        torch.cuda.synchronize()
    finally:
        pkg.tfl_layernorm_destroy(h)
    return s, stats, dy, dres, gamma, dx, dsum, dgamma, dbeta


def _check_backward(rows, d, xt, rt, got):
    s, stats, dy, dres, gamma, dx, dsum, dgamma, dbeta = got
    s, dy, gamma, m, r = _np(s), _np(dy), _np(gamma), _np(stats)[:, 0], _np(stats)[:, 1]
    dres = None if dres is None else _np(dres)
    ds, dg, db = ops.layer_norm_backward(s, m, r, gamma, dy, dres)
    a, t, r = np.abs(dy * gamma), np.abs(s - m[:, None]) * r[:, None], r[:, None]
    w = r * (a + a.mean(axis=1, keepdims=True) + t * (a * t).mean(axis=1, keepdims=True))
    w = w if dres is None else w + np.abs(dres)
    own = (_n(d) + 12) * E * w
    if dx is not None:
        _close(_np(dx), ds, own + _u(xt) * np.abs(ds) + _tiny(xt), "dx")
    if dsum is not None:
        _close(_np(dsum), ds, own + _u(rt) * np.abs(ds) + _tiny(rt), "dsum")
    k = (rows / 152 + 100) * E
    _close(_np(dgamma), dg, k * np.sum(np.abs(dy) * t, axis=0) + 1e-30, "dgamma")
    if dbeta is not None:
        _close(_np(dbeta), db, k * np.sum(np.abs(dy), axis=0) + 1e-30, "dbeta")


@pytest.mark.parametrize("rows,d", [(1, 1), (3, 7), (9, 64), (4001, 72), (33, 256), (700, 1000), (2500, 1024), (3, 1032),
                                    (5, 4096), (700, 4096), (3, 8200), (700, 8192), (700, 16384), (2, 16392), (5, 32768),
                                    (40, 1001), (900, 1025), (3, 4095), (700, 4097), (300, 8191), (2, 50001)])
@pytest.mark.parametrize("xt,rt", [("bf16", "f32"), ("f16", "f16")])
def test_backward_of_every_width(rows, d, xt, rt):
    _check_backward(rows, d, xt, rt, _backward(rows, d, xt, rt, seed=rows + d))


@pytest.mark.parametrize("xt,rt", [("f32", "f32"), ("f16", "f32"), ("bf16", "bf16")])
def test_backward_of_the_other_types_and_without_what_may_be_left_out(xt, rt):
    for rows, d in ((50, 264), (50, 65), (2, 9001), (600, 2048)):
        _check_backward(rows, d, xt, rt, _backward(rows, d, xt, rt, seed=d))
        _check_backward(rows, d, xt, rt, _backward(rows, d, xt, rt, with_dres=False, both=False, seed=d))
        _check_backward(rows, d, xt, rt, _backward(rows, d, xt, rt, with_beta=False, seed=d))


@pytest.mark.parametrize("d", [8, 16, 64, 256, 264])
@pytest.mark.parametrize("xt,rt", [("bf16", "f32"), ("f16", "f16")])
def test_backward_of_many_short_rows(d, xt, rt):
    for rows in (300, 160001 // d * 8):
        _check_backward(rows, d, xt, rt, _backward(rows, d, xt, rt, seed=rows + d))


@pytest.mark.parametrize("d", [31, 127, 129, 255, 257, 510, 513, 1023, 2047, 2049, 4094, 4097, 6143, 6145, 8191])
@pytest.mark.parametrize("xt,rt", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
def test_backward_of_the_widths_where_the_row_groups_change(d, xt, rt):
    for rows in (1, 5, 1301):
        _check_backward(rows, d, xt, rt, _backward(rows, d, xt, rt, seed=rows + d))


@pytest.mark.parametrize("rows,d", [(1300, 32776), (100, 400001)])
def test_wide_rows_over_several_turns(rows, d):
    """More rows than the backward's blocks; the last row's partial sums do not fit for that many blocks."""
    _check_forward(rows, d, "bf16", "f32", "e4m3", _forward(rows, d, "bf16", "f32", "e4m3", seed=d))
    _check_backward(rows, d, "bf16", "f32", _backward(rows, d, "bf16", "f32", seed=d))


# rows that begin inside a 16-byte vector: every shift, widths around those where the thread groups change, one
# row a group and several turns of the blocks
@pytest.mark.parametrize("d", [9, 10, 12, 15, 17, 250, 1001, 1002, 1004, 2033, 2034, 2035, 4081, 4082, 4083])
@pytest.mark.parametrize("xt,rt", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
def test_backward_of_rows_that_begin_inside_a_vector(d, xt, rt):
    for rows in (1, 2, 7, 9, 160, 6007 if d < 2000 else 1501, 40009 if d < 20 else 303):
        _check_backward(rows, d, xt, rt, _backward(rows, d, xt, rt, with_beta=rows != 9, seed=rows + d))


# the same of wide rows, in a block of 1024 threads (the backward: two vectors a thread)
WIDE_ODD = [4086, 4099, 4100, 4607, 4609, 7001, 8177, 8178, 8179]


@pytest.mark.parametrize("d", WIDE_ODD)
@pytest.mark.parametrize("xt,rt,yt", [("bf16", "f32", "e4m3"), ("f16", "f16", "f16"), ("f32", "f32", "bf16"), ("f32", "f32", "e4m3")])
def test_forward_of_wide_rows_that_begin_inside_a_vector(d, xt, rt, yt):
    for rows in (152, 160, 601):
        _check_forward(rows, d, xt, rt, yt, _forward(rows, d, xt, rt, yt, rows != 152, rows != 160, rows != 601, seed=rows + d))


# (and where the threads of wide rows change, even widths too)
@pytest.mark.parametrize("d", WIDE_ODD + [4104, 5120, 6129, 6130, 6131, 6144, 6152])
@pytest.mark.parametrize("xt,rt", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
def test_backward_of_wide_rows_that_begin_inside_a_vector(d, xt, rt):
    for rows in (490, 1958, 2411):
        _check_backward(rows, d, xt, rt, _backward(rows, d, xt, rt, with_dres=rows != 1958, with_beta=rows != 2411, seed=rows + d))


@pytest.mark.parametrize("rows,d", [(30, 9), (6011, 1001), (700, 1002), (40, 4081), (6011, 1000), (30, 4099), (2003, 4099), (1001, 8177)])
@pytest.mark.parametrize("xt,rt", [("bf16", "f32"), ("f16", "f16")])
def test_backward_keeps_rows_without_numbers_to_themselves(rows, d, xt, rt):
    import torch
    pkg = _pkg()
    s, stats, dy, dres, gamma, dx, dsum, _, _ = _backward(rows, d, xt, rt, seed=2)
    bad = sorted({1, rows // 2, rows - 2})
    s2, dy2, dres2 = s.clone(), dy.clone(), dres.clone()
    s2[bad[0]], dy2[bad[1]], dres2[bad[2]] = float("nan"), float("inf"), float("nan")
    dx2, dsum2, g, b = torch.empty_like(dx), torch.empty_like(s), torch.empty_like(gamma), torch.empty_like(gamma)
    h = pkg.tfl_layernorm_create(d, _code(xt), _code(rt), _code(xt), EPS)
    pkg.tfl_layernorm_backward(h, rows, s2.data_ptr(), stats.data_ptr(), gamma.data_ptr(), dy2.data_ptr(), dres2.data_ptr(),
                               dx2.data_ptr(), dsum2.data_ptr() if xt != rt else None, g.data_ptr(), b.data_ptr(), _stream())
    torch.cuda.synchronize()
    pkg.tfl_layernorm_destroy(h)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[bad] = False
    assert torch.equal(dx2[keep], dx[keep]) and not dx2[bad].isfinite().all(dim=1).any()
    if xt != rt:
        assert torch.equal(dsum2[keep], dsum[keep])


BUFFERS = ("sum", "gamma", "dy", "dres", "dx", "dsum", "dgamma", "dbeta")


# each buffer alone one element past its alignment, then all
@pytest.mark.parametrize("which", [(b,) for b in BUFFERS] + [BUFFERS])
@pytest.mark.parametrize("rows,d", [(1, 512), (3, 8), (333, 1024), (333, 1002), (40, 8192), (700, 16384)])
def test_backward_of_unaligned_buffers(rows, d, which):
    import torch
    pkg = _pkg()
    s, stats, dy, dres, gamma, *_ = _backward(rows, d, "bf16", "f32", seed=d)
    room = {}

    def place(name, t):
        at = 1 if name in which else 0
        flat = torch.full((t.numel() + 2,), 7.0, dtype=t.dtype, device="cuda")
        v = flat[at:at + t.numel()].view(t.shape)
        v.copy_(t)
        room[name] = (flat, at, t.numel())
        return v

    zero = lambda t: torch.zeros_like(t)  # noqa: E731
    b = {"sum": s, "gamma": gamma, "dy": dy, "dres": dres, "dx": zero(dy), "dsum": zero(s), "dgamma": zero(gamma),
         "dbeta": zero(gamma)}
    b = {k: place(k, v) for k, v in b.items()}
    h = pkg.tfl_layernorm_create(d, 2, 0, 2, EPS)
    P = lambda k: b[k].data_ptr()  # noqa: E731
    pkg.tfl_layernorm_backward(h, rows, P("sum"), stats.data_ptr(), P("gamma"), P("dy"), P("dres"), P("dx"), P("dsum"),
                               P("dgamma"), P("dbeta"), _stream())
    torch.cuda.synchronize()
    pkg.tfl_layernorm_destroy(h)
    _check_backward(rows, d, "bf16", "f32", (b["sum"], stats, b["dy"], b["dres"], b["gamma"], b["dx"], b["dsum"],
                                             b["dgamma"], b["dbeta"]))
    for flat, at, n in room.values():  # nothing around the buffers is touched
        assert (flat[:at] == 7).all() and (flat[at + n:] == 7).all()


def test_backward_is_the_forwards_difference_quotient():
    """L = sum(dy y) from the kernel's fp32 y, against ds along a direction.  Each y is off by the
    forward's bound, so the quotient by their sum with |dy| over 2 h; its h^2 term is the reference's own."""
    import torch
    pkg = _pkg()
    rows, d, h = 4, 96, 2.0 ** -5
    s, _, dy, _, gamma, dx, *_ = _backward(rows, d, "f32", "f32", with_dres=False, both=False, seed=9)
    v = torch.randn((rows, d), generator=torch.Generator(device="cuda").manual_seed(10), device="cuda")
    op = pkg.tfl_layernorm_create(d, 0, 0, 0, EPS)

    def loss(sign):
        p, y = (s + sign * h * v).contiguous(), torch.empty_like(s)
        pkg.tfl_layernorm_forward(op, rows, p.data_ptr(), None, gamma.data_ptr(), None, None, y.data_ptr(), None, None,
                                  _stream())
        ref = ops.layer_norm(_np(p), None, _np(gamma), None, EPS)[1]
        own = _bounds(_np(p), _np(gamma), np.zeros(d), EPS)[0] + E * np.abs(ref)
        return np.sum(_np(y) * _np(dy)), np.sum(ref * _np(dy)), np.sum(own * np.abs(_np(dy)))

    up, down = loss(1), loss(-1)
    pkg.tfl_layernorm_destroy(op)
    q, qref = (up[0] - down[0]) / (2 * h), (up[1] - down[1]) / (2 * h)
    noise = (up[2] + down[2]) / (2 * h)
    assert abs(q - qref) <= noise
    _, _, m, r = ops.layer_norm(_np(s), None, _np(gamma), None, EPS)
    ds = ops.layer_norm_backward(_np(s), m, r, _np(gamma), _np(dy), None)[0]
    along, ref_along = np.sum(_np(dx) * _np(v)), np.sum(ds * _np(v))
    # dx itself: (n + 12) e of its terms and the statistics' rounding, 2 e (|m| r + |t|): far below 1e-4
    assert abs(along - q) <= noise + abs(qref - ref_along) + 1e-4 * np.sum(np.abs(ds * _np(v)))


def test_backward_gives_the_same_bits_every_time_and_in_place():
    import torch
    pkg = _pkg()
    P = lambda t: t.data_ptr()  # noqa: E731
    for d in (512, 513, 516):
        s, stats, dy, dres, gamma, dx, _, dgamma, dbeta = _backward(3000, d, "bf16", "bf16", both=False, seed=4)
        again = _backward(3000, d, "bf16", "bf16", both=False, seed=4)
        assert torch.equal(dx, again[5]) and torch.equal(dgamma, again[7]) and torch.equal(dbeta, again[8])
        h = pkg.tfl_layernorm_create(d, 2, 2, 2, EPS)
        for name in ("dy", "dres", "sum"):
            b = {"sum": s.clone(), "dy": dy.clone(), "dres": dres.clone()}
            g2, b2 = torch.empty_like(dgamma), torch.empty_like(dbeta)
            pkg.tfl_layernorm_backward(h, 3000, P(b["sum"]), P(stats), P(gamma), P(b["dy"]), P(b["dres"]), P(b[name]),
                                       None, P(g2), P(b2), _stream())
            assert torch.equal(b[name], dx) and torch.equal(g2, dgamma) and torch.equal(b2, dbeta), name
        pkg.tfl_layernorm_destroy(h)


def test_no_rows():
    import torch
    pkg = _pkg()
    h = pkg.tfl_layernorm_create(64, 2, 0, 2, EPS)
    g, b = torch.full((64,), 3.0, device="cuda"), torch.full((64,), 3.0, device="cuda")
    pkg.tfl_layernorm_forward(h, 0, None, None, None, None, None, None, None, None, _stream())
    pkg.tfl_layernorm_backward(h, 0, None, None, None, None, None, None, None, g.data_ptr(), b.data_ptr(), _stream())
    torch.cuda.synchronize()
    assert (g == 0).all() and (b == 0).all()
    pkg.tfl_layernorm_destroy(h)


def test_rows_behind_the_last_stay_as_they_were():
    import torch
    pkg = _pkg()
    for d in (128, 130, 1030, 8194):
        x = torch.randn(9, d, device="cuda").bfloat16()
        y, out, stats = torch.full_like(x, 5.0), torch.full_like(x, 6.0), torch.full((9, 2), 4.0, device="cuda")
        gamma = torch.ones(d, device="cuda")
        h = pkg.tfl_layernorm_create(d, 2, 2, 2, EPS)
        pkg.tfl_layernorm_forward(h, 7, x.data_ptr(), x.data_ptr(), gamma.data_ptr(), gamma.data_ptr(), out.data_ptr(),
                                  y.data_ptr(), None, stats.data_ptr(), _stream())
        torch.cuda.synchronize()
        pkg.tfl_layernorm_destroy(h)
        assert (y[7:] == 5).all() and (out[7:] == 6).all() and (stats[7:] == 4).all() and (y[:7] != 5).any()


def test_captured_and_replayed_on_another_stream():
    import torch
    pkg = _pkg()
    rows, d = 333, 768
    s, stats, dy, dres, gamma, dx, dsum, dgamma, dbeta = _backward(rows, d, "bf16", "f32", seed=6)
    h = pkg.tfl_layernorm_create(d, 2, 0, 2, EPS)
    y, st2, out = torch.empty_like(dx), torch.empty_like(stats), torch.empty_like(s)
    P = lambda t: t.data_ptr()  # noqa: E731
    pkg.tfl_layernorm_forward(h, rows, P(dy), P(s), P(gamma), P(gamma), P(out), P(y), None, P(st2), _stream())
    want = [t.clone() for t in (out, y, st2, dx, dgamma, dbeta)]
    dx2, dg2, db2 = torch.empty_like(dx), torch.empty_like(dgamma), torch.empty_like(dbeta)
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=st):
        pkg.tfl_layernorm_forward(h, rows, P(dy), P(s), P(gamma), P(gamma), P(out), P(y), None, P(st2), st.cuda_stream)
        pkg.tfl_layernorm_backward(h, rows, P(s), P(stats), P(gamma), P(dy), P(dres), P(dx2), None, P(dg2), P(db2),
                                   st.cuda_stream)
    for _ in range(2):
        for t in (out, y, st2, dx2, dg2, db2):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((out, y, st2, dx2, dg2, db2), want))
    pkg.tfl_layernorm_destroy(h)


def test_refusals():
    import torch
    pkg = _pkg()
    h = pkg.tfl_layernorm_create(64, 2, 2, 2, EPS)
    q = pkg.tfl_layernorm_create(64, 2, 2, 3, EPS)
    x = torch.zeros(8, 64, device="cuda").bfloat16()
    o, y, res = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    g, b, sc, st = torch.ones(64, device="cuda"), torch.ones(64, device="cuda"), torch.ones(8, device="cuda"), torch.ones(8, 2, device="cuda")
    g2, b2 = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    P = lambda t: t.data_ptr()  # noqa: E731

    def refused(fn, *args, code=pkg.TFL_ERR_INVALID_ARG):
        with pytest.raises(pkg.TflError) as e:
            fn(*args, _stream())
        assert e.value.code == code and str(e.value)

    f, k = pkg.tfl_layernorm_forward, pkg.tfl_layernorm_backward
    refused(f, None, 4, P(x), None, P(g), None, None, P(y), None, None)
    refused(f, h, -1, P(x), None, P(g), None, None, P(y), None, None)
    refused(f, h, 1 << 31, P(x), None, P(g), None, None, P(y), None, None)
    refused(f, h, 4, None, None, P(g), None, None, P(y), None, None)
    refused(f, h, 4, P(x), None, None, None, None, P(y), None, None)
    refused(f, h, 4, P(x), None, P(g), None, None, None, None, None)
    refused(f, h, 4, P(x), None, P(g), None, None, P(y), P(sc), None)        # a scale without e4m3
    refused(f, q, 4, P(x), None, P(g), None, None, P(y), None, None)         # e4m3 without a scale
    refused(f, h, 4, P(x) + 1, None, P(g), None, None, P(y), None, None)     # not element-aligned
    refused(f, h, 4, P(x), None, P(g), P(b) + 2, None, P(y), None, None)
    refused(f, h, 4, P(x), None, P(g), None, None, P(y), None, P(st) + 4)    # stats come in pairs
    refused(f, h, 4, P(x), None, P(g), None, P(y), P(y), None, None)         # two outputs in one buffer
    refused(f, h, 4, P(x), None, P(g), None, None, P(x) + 128, None, None)   # shifted over its input
    refused(f, q, 4, P(x), None, P(g), None, None, P(x), P(sc), None)        # another type over its input
    refused(f, h, 4, P(x), P(res), P(g), None, P(res) + 128, P(y), None, None)
    refused(f, h, 4, P(x), P(res), P(g), None, None, P(res), None, None)     # y over the residual
    refused(f, h, 4, P(x), None, P(g), P(b), None, P(y), None, P(b))         # stats over beta
    refused(f, q, 4, P(x), None, P(g), None, None, P(y), P(st), P(st))
    refused(k, h, 4, P(x), P(st), P(g), P(y), None, None, None, P(g2), P(b2))       # nothing to write ds to
    refused(k, h, 4, P(x), None, P(g), P(y), None, P(o), None, P(g2), P(b2))        # no statistics
    refused(k, h, 4, P(x), P(st) + 4, P(g), P(y), None, P(o), None, P(g2), P(b2))
    refused(k, h, 4, P(x), P(st), P(g), P(y), None, P(o), P(o), P(g2), P(b2))       # outputs in one buffer
    refused(k, h, 4, P(x), P(st), P(g), P(y), None, P(o), None, P(g), P(b2))        # dgamma over gamma
    refused(k, h, 4, P(x), P(st), P(g), P(y), None, P(o), None, P(g2), P(g2) + 4)   # dbeta over dgamma
    refused(k, h, 4, P(x), P(st), P(g), P(y), None, P(st), None, P(g2), P(b2))
    refused(k, h, 4, P(x), P(st), P(g), P(y), None, P(y) + 128, None, P(g2), P(b2))
    refused(k, h, 4, P(x), P(st), P(g), P(y), None, P(o), None, None, P(b2))
    refused(k, q, 4, P(x), P(st), P(g), P(y), None, P(o), None, P(g2), P(b2), code=pkg.TFL_ERR_UNSUPPORTED)
    pkg.tfl_layernorm_destroy(h)
    pkg.tfl_layernorm_destroy(q)
