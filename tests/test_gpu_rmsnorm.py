"""The root-mean-square norm on the GPU against float64 (oracle/ops.py) on the same inputs.

Bounds, with u = eps / 2 of the stored type and e = 2^-24 (fp32's half step):
  res_out  one fp32 addition and one rounding: u|s| + e|s|
  y        the sum of squares adds at most n = max(32, D / 256 + 8) + 42 terms in a row (a
           thread's own, then the threads'), so its square root is off by n e / 2 relative;
           rsqrtf by 4 e, the additions, products and the mean by 6 e more: (n / 2 + 10) e |y|,
           plus the rounding u|y|
  scale    the same relative error, (n / 2 + 14) e with its division
  e4m3     the stored value times the scale: half a step of e4m3, 2^-4 |y| + 2^-10 scale
           (below e4m3's normal range), plus twice y's own error
  ds       with m = |dres| + r|a| + |s| r^3 mean|a s|: (3 n / 2 + n + 24) e m for the two sums
           and the products, plus u|ds|
  dgamma   sums of at most rows / 304 + 64 terms in a row: (that + n / 2 + 12) e sum|dy s r|
and half a step at the type's smallest value everywhere (2^-25 for fp16).
"""
import numpy as np
import pytest

from oracle import ops

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
EPS = 1e-5
NAMES = ("f32", "f16", "bf16")


def _pkg():
    import attention_qkv_gemm_gb300 as pkg
    return pkg


def _type(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[name]


def _code(name):
    pkg = _pkg()
    return {"f32": pkg.TFL_F32, "f16": pkg.TFL_F16, "bf16": pkg.TFL_BF16, "e4m3": pkg.TFL_E4M3}[name]


def _u(name):
    return {"f32": E, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[name]


def _tiny(name):
    return {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}[name]


def _n(d):
    return max(32, d / 256 + 8) + 42


def _np(t):
    return t.double().cpu().numpy()


def _stream():
    import torch
    return torch.cuda.current_stream().cuda_stream


def _randn(gen, shape, name, std=1.0):
    import torch
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(_type(name))


def _close(u, r, bound, what):
    assert np.isfinite(u).all(), f"{what}: non-finite"
    over = np.abs(u - r) / bound
    assert (over <= 1).all(), f"{what}: {int((over > 1).sum())} of {u.size} outside, worst {over.max():.3f} of the bound"


def _forward(rows, d, xt, rt, yt, with_res=True, store=True, seed=0, offset=0):
    """Runs the forward; `offset` shifts every buffer by that many elements (unaligned)."""
    import torch
    pkg = _pkg()
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def place(t):
        flat = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")[offset:]
        flat.copy_(t.reshape(-1))
        return flat.view(t.shape)

    x = place(_randn(gen, (rows, d), xt))
    res = place(_randn(gen, (rows, d), rt, 2.0)) if with_res else None
    gamma = place(1 + _randn(gen, (d,), "f32", 0.2))
    out = place(torch.full((rows, d), 7.0, dtype=_type(rt), device="cuda")) if store else None
    y = place(torch.zeros((rows, d), device="cuda").to(_type(yt)))
    scale = place(torch.full((rows,), -1.0, device="cuda")) if yt == "e4m3" else None
    h = pkg.tfl_rmsnorm_create(d, _code(xt), _code(rt), _code(yt), EPS)
    try:
        pkg.tfl_rmsnorm_forward(h, rows, x.data_ptr(), res.data_ptr() if with_res else None, gamma.data_ptr(),
                                out.data_ptr() if store else None, y.data_ptr(),
                                scale.data_ptr() if scale is not None else None, _stream())
        torch.cuda.synchronize()
    finally:
        pkg.tfl_rmsnorm_destroy(h)
    return x, res, gamma, out, y, scale


def _check_forward(rows, d, xt, rt, yt, got):
    x, res, gamma, out, y, scale = got
    s, ref = ops.rms_norm(_np(x), None if res is None else _np(res), _np(gamma), EPS)
    if out is not None:
        _close(_np(out), s, (_u(rt) + E) * np.abs(s) + _tiny(rt), "res_out")
    own = (_n(d) / 2 + 10) * E * np.abs(ref)
    if yt != "e4m3":
        _close(_np(y), ref, own + _u(yt) * np.abs(ref) + _tiny(yt), "y")
        return
    rs = ops.row_scale(ref)
    _close(_np(scale), rs, (_n(d) / 2 + 14) * E * rs, "scale")
    _close(_np(y) * _np(scale)[:, None], ref, 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 * rs[:, None] + 2 * own, "e4m3 y")


TYPES = [("f32", "f32", "f32"), ("f32", "f32", "f16"), ("f32", "f32", "bf16"), ("f32", "f32", "e4m3"),
         ("f16", "f16", "f16"), ("f16", "f32", "f16"), ("f16", "f16", "e4m3"), ("f16", "f32", "e4m3"),
         ("bf16", "bf16", "bf16"), ("bf16", "f32", "bf16"), ("bf16", "bf16", "e4m3"), ("bf16", "f32", "e4m3")]


@pytest.mark.parametrize("xt,rt,yt", TYPES)
def test_forward_of_every_type(xt, rt, yt):
    for rows, d in ((1, 1024), (37, 264), (5, 8)):
        _check_forward(rows, d, xt, rt, yt, _forward(rows, d, xt, rt, yt, seed=d))


# one value, less than a warp, ragged vectors, one warp and more a row, the widest row kept in
# registers and the first that is not, widths no vector divides
@pytest.mark.parametrize("rows,d", [(1, 1), (3, 7), (9, 64), (300, 72), (33, 256), (17, 512), (12, 1000), (1000, 1024),
                                    (3, 1032), (5, 4096), (3, 8200), (2, 32768), (2, 32776), (4, 1001), (3, 1025), (70, 4095), (2, 4097), (30, 8191), (3, 8193), (2, 50001)])
@pytest.mark.parametrize("xt,rt,yt", [("bf16", "f32", "e4m3"), ("f16", "f16", "f16"), ("f32", "f32", "f32")])
def test_forward_of_every_width(rows, d, xt, rt, yt):
    _check_forward(rows, d, xt, rt, yt, _forward(rows, d, xt, rt, yt, seed=rows + d))


# enough rows for the kernel that loops over them: groups of one thread to the whole block, a
# ragged last round
@pytest.mark.parametrize("rows,d", [(351000, 8), (45001, 72), (22000, 256), (11003, 400), (5603, 1000), (1501, 4096)])
@pytest.mark.parametrize("xt,rt,yt", [("bf16", "f32", "e4m3"), ("f16", "f16", "f16"), ("f32", "f32", "f32"),
                                      ("bf16", "bf16", "e4m3")])
def test_forward_of_many_rows(rows, d, xt, rt, yt):
    _check_forward(rows, d, xt, rt, yt, _forward(rows, d, xt, rt, yt, seed=d))


@pytest.mark.parametrize("xt,rt,yt", TYPES)
def test_forward_of_many_rows_of_every_type(xt, rt, yt):
    _check_forward(11003, 512, xt, rt, yt, _forward(11003, 512, xt, rt, yt, seed=1))


@pytest.mark.parametrize("with_res,store", [(False, True), (True, False)])
def test_forward_of_many_rows_without_residual_or_its_store(with_res, store):
    _check_forward(6001, 1024, "bf16", "f32", "bf16", _forward(6001, 1024, "bf16", "f32", "bf16", with_res, store))


@pytest.mark.parametrize("with_res,store", [(False, True), (True, False), (False, False)])
def test_forward_without_residual_or_its_store(with_res, store):
    for d in (256, 129):
        _check_forward(6, d, "bf16", "f32", "bf16", _forward(6, d, "bf16", "f32", "bf16", with_res, store))


@pytest.mark.parametrize("offset", [1, 4])
def test_forward_of_unaligned_buffers(offset):
    _check_forward(7, 512, "bf16", "f32", "e4m3", _forward(7, 512, "bf16", "f32", "e4m3", offset=offset))
    _check_forward(7, 512, "f16", "f16", "f16", _forward(7, 512, "f16", "f16", "f16", offset=offset))


@pytest.mark.parametrize("rows,d", [(40, 512), (40, 515), (11003, 512)])
def test_forward_in_place_equals_out_of_place(rows, d):
    import torch
    pkg = _pkg()
    x, res, gamma, out, y, _ = _forward(rows, d, "bf16", "bf16", "bf16", seed=3)
    h = pkg.tfl_rmsnorm_create(d, _code("bf16"), _code("bf16"), _code("bf16"), EPS)
    try:
        x2, r2 = x.clone(), res.clone()
        pkg.tfl_rmsnorm_forward(h, rows, x2.data_ptr(), r2.data_ptr(), gamma.data_ptr(), r2.data_ptr(), x2.data_ptr(),
                                None, _stream())
        assert torch.equal(r2, out) and torch.equal(x2, y)
        x3, y3 = x.clone(), torch.empty_like(y)
        pkg.tfl_rmsnorm_forward(h, rows, x3.data_ptr(), res.data_ptr(), gamma.data_ptr(), x3.data_ptr(), y3.data_ptr(),
                                None, _stream())
        assert torch.equal(x3, out) and torch.equal(y3, y)
    finally:
        pkg.tfl_rmsnorm_destroy(h)


@pytest.mark.parametrize("rows,d", [(6, 256), (6, 255), (22000, 256)])
def test_rows_of_zeros_nan_and_infinity_stay_their_own(rows, d):
    import torch
    pkg = _pkg()
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = _randn(gen, (rows, d), "bf16")
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    gamma = torch.ones(d, device="cuda")
    for yt in ("bf16", "e4m3"):
        y = torch.zeros((rows, d), device="cuda").to(_type(yt))
        scale = torch.zeros(rows, device="cuda")
        h = pkg.tfl_rmsnorm_create(d, _code("bf16"), _code("bf16"), _code(yt), EPS)
        pkg.tfl_rmsnorm_forward(h, rows, x.data_ptr(), None, gamma.data_ptr(), None, y.data_ptr(),
                                scale.data_ptr() if yt == "e4m3" else None, _stream())
        torch.cuda.synchronize()
        pkg.tfl_rmsnorm_destroy(h)
        f = y.float()
        assert (f[1] == 0).all()
        assert f[2].isnan().all()
        assert f[3, 7].isnan()
        assert f[[0, 1, *range(4, rows)]].isfinite().all()
        if yt == "e4m3":
            assert scale[1].item() == np.float32(2.0 ** -100) / np.float32(448) and scale[2].isnan()


def _backward(rows, d, xt, rt, with_dres=True, both=True, seed=0):
    import torch
    pkg = _pkg()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = _randn(gen, (rows, d), rt, 2.0)
    dy = _randn(gen, (rows, d), xt)
    dres = _randn(gen, (rows, d), rt) if with_dres else None
    gamma = 1 + _randn(gen, (d,), "f32", 0.2)
    dx = torch.full((rows, d), 7.0, dtype=_type(xt), device="cuda")
    dsum = torch.full((rows, d), 7.0, dtype=_type(rt), device="cuda") if both else None
    dgamma = torch.full((d,), 7.0, device="cuda")
    h = pkg.tfl_rmsnorm_create(d, _code(xt), _code(rt), _code(xt), EPS)
    try:
        for _ in range(2):  # the second call finds the first one's scratch
            pkg.tfl_rmsnorm_backward(h, rows, s.data_ptr(), gamma.data_ptr(), dy.data_ptr(),
                                     dres.data_ptr() if with_dres else None, dx.data_ptr(),
                                     dsum.data_ptr() if both else None, dgamma.data_ptr(), _stream())
        torch.cuda.synchronize()
    finally:
        pkg.tfl_rmsnorm_destroy(h)
    return s, dy, dres, gamma, dx, dsum, dgamma


def _check_backward(rows, d, xt, rt, got):
    s, dy, dres, gamma, dx, dsum, dgamma = got
    s, dy, gamma = _np(s), _np(dy), _np(gamma)
    dres = None if dres is None else _np(dres)
    ds, dg = ops.rms_norm_backward(s, gamma, dy, dres, EPS)
    r = 1 / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + EPS)
    a = dy * gamma
    m = r * np.abs(a) + np.abs(s) * r ** 3 * np.mean(np.abs(a * s), axis=1, keepdims=True)
    m = m if dres is None else m + np.abs(dres)
    own = (2.5 * _n(d) + 24) * E * m
    _close(_np(dx), ds, own + _u(xt) * np.abs(ds) + _tiny(xt), "dx")
    if dsum is not None:
        _close(_np(dsum), ds, own + _u(rt) * np.abs(ds) + _tiny(rt), "dsum")
    _close(_np(dgamma), dg, (rows / 304 + 64 + _n(d) / 2 + 12) * E * np.sum(np.abs(dy * s * r), axis=0) + 1e-30,
           "dgamma")


@pytest.mark.parametrize("rows,d", [(1, 1), (3, 7), (9, 64), (4001, 72), (33, 256), (700, 1000), (2500, 1024), (3, 1032),
                                    (5, 4096), (700, 4096), (3, 8200), (700, 8192), (700, 16384), (2, 16392), (5, 32768), (40, 1001), (900, 1025), (3, 4095), (700, 4097), (300, 8191),
                                    (2, 50001)])
@pytest.mark.parametrize("xt,rt", [("bf16", "f32"), ("f16", "f16")])
def test_backward_of_every_width(rows, d, xt, rt):
    _check_backward(rows, d, xt, rt, _backward(rows, d, xt, rt, seed=rows + d))


@pytest.mark.parametrize("xt,rt", [("f32", "f32"), ("f16", "f32"), ("bf16", "bf16")])
def test_backward_of_the_other_types(xt, rt):
    for d in (264, 65):
        _check_backward(50, d, xt, rt, _backward(50, d, xt, rt, seed=d))
        _check_backward(50, d, xt, rt, _backward(50, d, xt, rt, with_dres=False, both=False, seed=d))


@pytest.mark.parametrize("d", [8, 16, 64, 256, 264])
@pytest.mark.parametrize("xt,rt", [("bf16", "f32"), ("f16", "f16")])
def test_backward_of_many_short_rows(d, xt, rt):
    for rows in (300, 160001 // d * 8):
        _check_backward(rows, d, xt, rt, _backward(rows, d, xt, rt, seed=rows + d))


@pytest.mark.parametrize("d", [31, 127, 129, 255, 257, 510, 513, 1023, 2047, 2049, 4094, 5119, 5121, 6143, 6145, 8191])
@pytest.mark.parametrize("xt,rt", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
def test_backward_of_the_widths_where_the_row_groups_change(d, xt, rt):
    for rows in (1, 5, 1301):
        _check_backward(rows, d, xt, rt, _backward(rows, d, xt, rt, seed=rows + d))


def test_backward_is_the_forwards_difference_quotient():
    """L = sum(dy y) from the kernel's fp32 y, against ds along a direction.  Each y is off by
    c|y| (c of the forward's bound), so the quotient by c sum|y dy| / h; its h^2 term is the
    reference's own."""
    import torch
    pkg = _pkg()
    rows, d, h = 4, 96, 2.0 ** -5
    s, dy, _, gamma, dx, _, _ = _backward(rows, d, "f32", "f32", with_dres=False, both=False, seed=9)
    v = torch.randn((rows, d), generator=torch.Generator(device="cuda").manual_seed(10), device="cuda")
    op = pkg.tfl_rmsnorm_create(d, 0, 0, 0, EPS)

    def loss(sign):
        p, y = (s + sign * h * v).contiguous(), torch.empty_like(s)
        pkg.tfl_rmsnorm_forward(op, rows, p.data_ptr(), None, gamma.data_ptr(), None, y.data_ptr(), None, _stream())
        ref = ops.rms_norm(_np(p), None, _np(gamma), EPS)[1]
        return np.sum(_np(y) * _np(dy)), np.sum(ref * _np(dy)), np.sum(np.abs(ref * _np(dy)))

    up, down = loss(1), loss(-1)
    pkg.tfl_rmsnorm_destroy(op)
    q, qref = (up[0] - down[0]) / (2 * h), (up[1] - down[1]) / (2 * h)
    noise = (_n(d) / 2 + 11) * E * (up[2] + down[2]) / (2 * h)
    assert abs(q - qref) <= noise
    ds = ops.rms_norm_backward(_np(s), _np(gamma), _np(dy), None, EPS)[0]
    along, ref_along = np.sum(_np(dx) * _np(v)), np.sum(ds * _np(v))
    assert abs(along - q) <= noise + abs(qref - ref_along) + 1e-4 * np.sum(np.abs(ds * _np(v)))


def test_backward_gives_the_same_bits_every_time_and_in_place():
    import torch
    pkg = _pkg()
    for d in (512, 513):
        s, dy, dres, gamma, dx, _, dgamma = _backward(3000, d, "bf16", "bf16", both=False, seed=4)
        again = _backward(3000, d, "bf16", "bf16", both=False, seed=4)
        assert torch.equal(dx, again[4]) and torch.equal(dgamma, again[6])
        h = pkg.tfl_rmsnorm_create(d, 2, 2, 2, EPS)
        for name in ("dy", "dres", "sum"):
            b = {"sum": s.clone(), "dy": dy.clone(), "dres": dres.clone()}
            g2 = torch.empty_like(dgamma)
            pkg.tfl_rmsnorm_backward(h, 3000, b["sum"].data_ptr(), gamma.data_ptr(), b["dy"].data_ptr(),
                                     b["dres"].data_ptr(), b[name].data_ptr(), None, g2.data_ptr(), _stream())
            assert torch.equal(b[name], dx) and torch.equal(g2, dgamma), name
        pkg.tfl_rmsnorm_destroy(h)


@pytest.mark.parametrize("rows", [1, 3, 700])
@pytest.mark.parametrize("d", [64, 512, 513, 2048, 8200])
def test_backward_into_a_dgamma_that_is_only_aligned_to_its_elements(rows, d):
    import torch
    pkg = _pkg()
    s, dy, dres, gamma, dx, dsum, dgamma = got = _backward(rows, d, "bf16", "f32", seed=rows)
    _check_backward(rows, d, "bf16", "f32", got)
    room = torch.full((d + 2,), 7.0, device="cuda")
    h = pkg.tfl_rmsnorm_create(d, 2, 0, 2, EPS)
    pkg.tfl_rmsnorm_backward(h, rows, s.data_ptr(), gamma.data_ptr(), dy.data_ptr(), dres.data_ptr(), dx.data_ptr(),
                             dsum.data_ptr(), room[1:].data_ptr(), _stream())
    torch.cuda.synchronize()
    pkg.tfl_rmsnorm_destroy(h)
    assert torch.equal(room[1:-1], dgamma) and room[0] == 7 and room[-1] == 7


def test_no_rows():
    import torch
    pkg = _pkg()
    h = pkg.tfl_rmsnorm_create(64, 2, 0, 2, EPS)
    g = torch.full((64,), 3.0, device="cuda")
    pkg.tfl_rmsnorm_forward(h, 0, None, None, None, None, None, None, _stream())
    pkg.tfl_rmsnorm_backward(h, 0, None, None, None, None, None, None, g.data_ptr(), _stream())
    torch.cuda.synchronize()
    assert (g == 0).all()
    pkg.tfl_rmsnorm_destroy(h)


def test_rows_behind_the_last_stay_as_they_were():
    import torch
    pkg = _pkg()
    for d in (128, 130):
        x = torch.randn(9, d, device="cuda").bfloat16()
        y, out = torch.full_like(x, 5.0), torch.full_like(x, 6.0)
        gamma = torch.ones(d, device="cuda")
        h = pkg.tfl_rmsnorm_create(d, 2, 2, 2, EPS)
        pkg.tfl_rmsnorm_forward(h, 7, x.data_ptr(), x.data_ptr(), gamma.data_ptr(), out.data_ptr(), y.data_ptr(), None,
                                _stream())
        torch.cuda.synchronize()
        pkg.tfl_rmsnorm_destroy(h)
        assert (y[7:] == 5).all() and (out[7:] == 6).all() and (y[:7] != 5).any()


def test_captured_and_replayed_on_another_stream():
    import torch
    pkg = _pkg()
    rows, d = 333, 768
    s, dy, dres, gamma, dx, dsum, dgamma = _backward(rows, d, "bf16", "f32", seed=6)
    h = pkg.tfl_rmsnorm_create(d, 2, 0, 2, EPS)
    dx2, dg2 = torch.empty_like(dx), torch.empty_like(dgamma)
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=st):
        pkg.tfl_rmsnorm_backward(h, rows, s.data_ptr(), gamma.data_ptr(), dy.data_ptr(), dres.data_ptr(),
                                 dx2.data_ptr(), None, dg2.data_ptr(), st.cuda_stream)
    for _ in range(2):
        dx2.zero_(), dg2.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(dx2, dx) and torch.equal(dg2, dgamma)
    pkg.tfl_rmsnorm_destroy(h)


def test_refusals():
    import torch
    pkg = _pkg()
    h = pkg.tfl_rmsnorm_create(64, 2, 2, 2, EPS)
    q = pkg.tfl_rmsnorm_create(64, 2, 2, 3, EPS)
    x = torch.zeros(8, 64, device="cuda").bfloat16()
    o, y, res = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    g, sc = torch.ones(64, device="cuda"), torch.ones(8, device="cuda")
    P = lambda t: t.data_ptr()  # noqa: E731

    def refused(fn, *args, code=pkg.TFL_ERR_INVALID_ARG):
        with pytest.raises(pkg.TflError) as e:
            fn(*args, _stream())
        assert e.value.code == code and str(e.value)

    f, b = pkg.tfl_rmsnorm_forward, pkg.tfl_rmsnorm_backward
    refused(f, None, 4, P(x), None, P(g), None, P(y), None)
    refused(f, h, -1, P(x), None, P(g), None, P(y), None)
    refused(f, h, 1 << 31, P(x), None, P(g), None, P(y), None)
    refused(f, h, 4, None, None, P(g), None, P(y), None)
    refused(f, h, 4, P(x), None, None, None, P(y), None)
    refused(f, h, 4, P(x), None, P(g), None, None, None)
    refused(f, h, 4, P(x), None, P(g), None, P(y), P(sc))       # a scale without e4m3
    refused(f, q, 4, P(x), None, P(g), None, P(y), None)        # e4m3 without a scale
    refused(f, h, 4, P(x) + 1, None, P(g), None, P(y), None)    # not element-aligned
    refused(f, h, 4, P(x), None, P(g), P(y), P(y), None)        # two outputs in one buffer
    refused(f, h, 4, P(x), None, P(g), None, P(x) + 128, None)  # shifted over its input
    refused(f, q, 4, P(x), None, P(g), None, P(x), P(sc))       # another type over its input
    refused(f, h, 4, P(x), P(res), P(g), P(res) + 128, P(y), None)
    refused(b, h, 4, P(x), P(g), P(y), None, None, None, P(sc))        # nothing to write ds to
    refused(b, h, 4, P(x), P(g), P(y), None, P(o), P(o), P(g))         # outputs in one buffer
    refused(b, h, 4, P(x), P(g), P(y), None, P(o), None, P(g))         # dgamma over gamma
    refused(b, h, 4, P(x), P(g), P(y), None, P(y) + 128, None, P(sc))
    refused(b, h, 4, P(x), P(g), P(y), None, P(o), None, None)
    refused(b, q, 4, P(x), P(g), P(y), None, P(o), None, P(sc), code=pkg.TFL_ERR_UNSUPPORTED)
    pkg.tfl_rmsnorm_destroy(h)
    pkg.tfl_rmsnorm_destroy(q)
