"""The linear layer on the GPU against its definition in float64 on the same inputs.

Bounds per element.  u = eps / 2 of the stored type, e = 2^-24; products of the operands are exact in
fp32 and a sum over K takes K / 16 + 16 accumulation steps, each off by at most a = 2^-22 of the
absolute sum (the tensor cores' accumulation need not round to nearest):
  z        dz0 = (K / 16 + 16) a |x||W|^T + 2 e (|z| + |bias|); e4m3 scales: 2^-22 of |x||W|^T more;
           stored: plus u|z|
  act      |act'| <= 1.13; evaluating it: 2^-20 relative plus 4e-7 (1 + |z|) (Abramowitz & Stegun
           7.1.26 is good to 1.5e-7 absolute)
  y        1.13 dz0 + the evaluation + 2 e (|act(z)| + |res|), plus u|y|
  dz       |dy| times the slope's evaluation, 2^-19 |act'| + 4e-7 (1 + |z|); rounded: plus u|dz|
  dx, dW   dz's through the products, their own accumulation, plus u|.|
  db       dz's before its rounding, and at most rows / 64 + 300 additions in a row: that times e sum|dz|
and half a step at the type's smallest value.  Worst-case sums are wide for long sums, so the
2-norm of 16-bit outputs is held as well: independent roundings of relative size at most u have an rms of
at most u / sqrt 3, two of them (dz, and the output) 0.82 u, so 1.2 u with the fp32 terms.
"""
import numpy as np
import pytest

from oracle import ops
from tests import linear_forms

pytestmark = pytest.mark.gpu

ACC, E = 2.0 ** -22, 2.0 ** -24
U = {"f32": E, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def _pkg():
    import attention_qkv_gemm_gb300 as pkg
    return pkg


def _type(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def _code(name):
    pkg = _pkg()
    return {"f32": pkg.TFL_F32, "f16": pkg.TFL_F16, "bf16": pkg.TFL_BF16, "e4m3": pkg.TFL_E4M3, "none": pkg.TFL_ACT_NONE,
            "silu": pkg.TFL_ACT_SILU, "gelu": pkg.TFL_ACT_GELU}[name]


def _stream():
    import torch
    return torch.cuda.current_stream().cuda_stream


def P(t):
    return None if t is None else t.data_ptr()


def _close(u, r, bound, what, limit=None):
    u = u.double()
    assert u.isfinite().all(), f"{what}: non-finite"
    over = (u - r).abs() / bound
    assert bool((over <= 1).all()), (f"{what}: {int((over > 1).sum())} of {u.numel()} outside, worst {float(over.max()):.3f} "
                                     f"of the bound, first at {(over > 1).nonzero()[:3].tolist()}")
    if limit is not None and r.numel() >= 1000:
        rel = float((u - r).norm() / r.norm())
        assert rel <= limit, f"{what}: relative 2-norm {rel:.2e} over {limit:.2e}"


def _activation(z, kind):
    import torch
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    cdf = 0.5 * (1 + torch.special.erf(z * 0.5 ** 0.5))
    return z * cdf, cdf + z * torch.exp(-0.5 * z * z) * 0.3989422804014327


def _rows8(t):
    import torch
    scale = t.abs().amax(dim=1).clamp_min(2.0 ** -100) / 448
    return (t / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn), scale


class Case:
    """Inputs of a call; e4m3 operands where t8 is given."""

    def __init__(self, tokens, k, n, t="bf16", out="bf16", act="none", bias=True, res=False, train=False, e4m3=False, seed=0):
        import torch
        gen = torch.Generator(device="cuda").manual_seed(seed + tokens + k)
        rnd = lambda *s, std=1.0: torch.randn(*s, generator=gen, device="cuda") * std  # noqa: E731
        self.tokens, self.k, self.n, self.t, self.out, self.act, self.e4m3 = tokens, k, n, t, out, act, e4m3
        x, w = rnd(tokens, k), rnd(n, k, std=k ** -0.5)
        self.xs = self.ws = None
        if e4m3:
            x = x * 2.0 ** torch.randint(-6, 4, (tokens, 1), generator=gen, device="cuda")
            (self.x, self.xs), (self.w, self.ws) = _rows8(x), _rows8(w)
        else:
            self.x, self.w = x.to(_type(t)), w.to(_type(t))
        self.bias = rnd(n, std=0.5) if bias else None
        self.res = rnd(tokens, n, std=2.0).to(_type(out)) if res else None
        self.y = torch.full((tokens + 3, n), 7.0, dtype=_type(out), device="cuda")
        self.z = torch.full((tokens + 3, n), 7.0, dtype=_type(t), device="cuda") if train else None

    def create(self, max_grad=0, dy="f32"):
        return _pkg().tfl_linear_create(self.k, self.n, _code("e4m3" if self.e4m3 else self.t), _code(self.out),
                                        _code(self.act), _code(dy), max_grad)

    def forward(self, op, stream=None, y=None):
        _pkg().tfl_linear_forward(op, self.tokens, P(self.x), P(self.xs), P(self.w), P(self.ws), P(self.bias), P(self.res),
                                  P(self.z), P(self.y) if y is None else P(y), _stream() if stream is None else stream)

    def run(self):
        pkg, op = _pkg(), self.create()
        try:
            self.forward(op)
            assert pkg.tfl_linear_status(op, _stream()) == 0, pkg.tfl_last_error()
        finally:
            pkg.tfl_linear_destroy(op)
        assert (self.y[self.tokens:] == 7).all()  # rows behind the last stay as they were
        return self

    def check(self):
        x, w = self.x.double(), self.w.double()
        if self.e4m3:
            x, w = x * self.xs.double()[:, None], w * self.ws.double()[:, None]
        z = x @ w.t()
        own = ((self.k / 16 + 16) * ACC + (ACC if self.e4m3 else 0)) * (x.abs() @ w.abs().t())
        if self.bias is not None:
            z = z + self.bias.double()
            own = own + 2 * E * self.bias.double().abs()
        own = own + 2 * E * z.abs()
        if self.z is not None:
            assert (self.z[self.tokens:] == 7).all()
            _close(self.z[:self.tokens], z, own + U[self.t] * z.abs() + TINY[self.t], "z", 0.8 * U[self.t])
        y = _activation(z, self.act)[0]
        if self.act != "none":
            own = 1.13 * own + 2.0 ** -20 * y.abs() + 4e-7 * (1 + z.abs())
        own = own + 2 * E * y.abs()
        if self.res is not None:
            y = y + self.res.double()
            own = own + 2 * E * self.res.double().abs()
        _close(self.y[:self.tokens], y, own + U[self.out] * y.abs() + TINY[self.out], "y",
               None if self.out == "f32" else 0.8 * U[self.out])


# one token and few, one value of width, k and columns that no tile divides, tile edges, more tiles than the
# GPU holds at a time, few tiles of long rows
SIZES = [(1, 8, 8), (1, 1024, 520), (3, 72, 16), (8, 264, 40), (9, 1000, 136), (16, 512, 24), (17, 64, 256),
         (33, 136, 1000), (64, 2056, 128), (65, 64, 136), (127, 72, 136), (128, 64, 128), (129, 200, 264),
         (300, 1160, 712), (513, 64, 1000), (4100, 72, 1032), (20, 4104, 72), (100, 2056, 520), (128, 1096, 4096),
         (300, 4096, 264), (257, 8, 2000), (40000, 64, 24)]


@pytest.mark.parametrize("tokens,k,n", SIZES)
@pytest.mark.parametrize("t,out,act,bias,res,train", [("bf16", "bf16", "gelu", True, True, True), ("f16", "f32", "none", True, True, False),
                                                      ("f16", "f16", "silu", False, False, True),
                                                      ("bf16", "f32", "none", False, False, False)])
def test_forward(tokens, k, n, t, out, act, bias, res, train):
    Case(tokens, k, n, t, out, act, bias, res, train).run().check()


@pytest.mark.parametrize("tokens,k,n", [(5, 88, 72), (200, 88, 200), (500, 1024, 520), (24, 2048, 264)])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("bias,res,train", [(b, r, z) for b in (False, True) for r in (False, True) for z in (False, True)])
def test_forward_of_every_epilogue(tokens, k, n, act, bias, res, train):
    for t, out in (("bf16", "bf16"), ("f16", "f32"), ("f16", "f16"), ("bf16", "f32")):
        Case(tokens, k, n, t, out, act, bias, res, train and act != "none").run().check()


@pytest.mark.parametrize("tokens,k,n", linear_forms.FORWARD)
@pytest.mark.parametrize("t,out,act,res,train", [("bf16", "bf16", "gelu", True, True), ("f16", "f32", "silu", True, False),
                                                 ("f16", "f16", "none", False, False)])
def test_forward_in_every_form(tokens, k, n, t, out, act, res, train):
    Case(tokens, k, n, t, out, act, True, res, train).run().check()


@pytest.mark.parametrize("tokens,k,n", linear_forms.E4M3 + [(1, 16, 16), (1, 2064, 528), (7, 144, 32), (33, 144, 272),
                                                            (100, 4112, 144), (30, 8192, 544), (200, 1024, 512)])
@pytest.mark.parametrize("out,act,bias,res", [("bf16", "none", True, True), ("f16", "gelu", True, False),
                                              ("f32", "silu", True, True), ("f32", "none", False, False)])
def test_forward_of_e4m3_operands(tokens, k, n, out, act, bias, res):
    Case(tokens, k, n, "bf16" if out == "f32" else out, out, act, bias, res, e4m3=True).run().check()


def test_the_sizes_reach_every_form_on_this_gpu():
    assert linear_forms.reached() >= linear_forms.WANTED


@pytest.mark.parametrize("k,n", [(1032, 40), (1160, 72), (1400, 1200), (2048, 5120), (2056, 48), (2600, 64), (4056, 56),
                                 (4096, 1032), (8192, 16), (8200, 16), (64, 20000)])
@pytest.mark.parametrize("tokens", [1, 8, 15])
def test_forward_of_a_few_tokens_and_long_rows(tokens, k, n):
    Case(tokens, k, n, "bf16", "bf16", "gelu", True, True, True).run().check()


@pytest.mark.parametrize("tokens,k,n", [(3, 264, 72), (40, 2048, 136), (300, 264, 520), (2600, 512, 1032)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_the_residual_may_be_the_output(tokens, k, n, out):
    import torch
    c = Case(tokens, k, n, "bf16", out, "none", True, True).run()
    op, y = c.create(), c.res.clone()
    c.res = y
    c.forward(op, y=y)
    torch.cuda.synchronize()
    _pkg().tfl_linear_destroy(op)
    assert torch.equal(y, c.y[:tokens])


def _backward(tokens, k, n, t="bf16", act="none", dy="f32", seed=0, room=5, want=("dx", "dw", "db"), z_std=1.5):
    import torch
    pkg = _pkg()
    gen = torch.Generator(device="cuda").manual_seed(seed + tokens + n)
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=gen, device="cuda") * std  # noqa: E731
    x, w = rnd(tokens, k).to(_type(t)), rnd(n, k, std=k ** -0.5).to(_type(t))
    z = rnd(tokens, n, std=z_std).to(_type(t)) if act != "none" else None
    g = rnd(tokens, n).to(_type(dy))
    out = {"dx": torch.full((tokens + 3, k), 7.0, dtype=_type(t), device="cuda"), "dw": torch.full_like(w, 7.0),
           "db": torch.full((n,), 7.0, device="cuda")}
    out = {name: v if name in want else None for name, v in out.items()}
    op = pkg.tfl_linear_create(k, n, _code(t), _code(t), _code(act), _code(dy), tokens + room)
    try:
        for _ in range(2):  # the second call finds the first one's scratch
            pkg.tfl_linear_backward(op, tokens, P(x) if "dw" in want else None, P(w) if "dx" in want else None, P(z), P(g),
                                    P(out["dx"]), P(out["dw"]), P(out["db"]), _stream())
        assert pkg.tfl_linear_status(op, _stream()) == 0, pkg.tfl_last_error()
    finally:
        pkg.tfl_linear_destroy(op)
    if out["dx"] is not None:
        assert (out["dx"][tokens:] == 7).all()
        out["dx"] = out["dx"][:tokens]
    return x, w, z, g, out


def _check_backward(x, w, z, g, out, t, act):
    tokens, (n, k) = x.shape[0], w.shape
    x, w, g = x.double(), w.double(), g.double()
    dz, fine = g, 0 * g
    if act != "none":
        slope = _activation(z.double(), act)[1]
        dz, fine = g * slope, g.abs() * (2.0 ** -19 * slope.abs() + 4e-7 * (1 + z.double().abs()))
    e = fine + U[t] * dz.abs() + TINY[t]
    if out["dx"] is not None:
        r = dz @ w
        _close(out["dx"], r, 1.01 * (e @ w.abs() + (n / 16 + 16) * ACC * (dz.abs() @ w.abs())) + U[t] * r.abs() + TINY[t], "dx",
               1.2 * U[t])
    if out["dw"] is not None:
        r = dz.t() @ x
        bound = 1.01 * (e.t() @ x.abs() + (tokens / 16 + 16) * ACC * (dz.abs().t() @ x.abs())) + U[t] * r.abs() + TINY[t]
        _close(out["dw"], r, bound, "dw", 1.2 * U[t])
    if out["db"] is not None:
        _close(out["db"], dz.sum(0), (fine + E * dz.abs()).sum(0) + (tokens / 64 + 300) * E * dz.abs().sum(0) + 1e-30, "db")


KINDS = [("bf16", "gelu", "bf16"), ("f16", "none", "f32"), ("f16", "silu", "f32"), ("bf16", "none", "bf16")]


@pytest.mark.parametrize("tokens,k,n", [(1, 8, 8), (1, 264, 72), (3, 72, 16), (65, 64, 136), (128, 256, 64), (129, 200, 264),
                                        (300, 1160, 712), (1000, 72, 328), (70, 1000, 2568), (5000, 2056, 72),
                                        (20, 520, 2056), (5, 2056, 1032), (200, 264, 4104), (6000, 136, 200), (40000, 64, 24)])
@pytest.mark.parametrize("t,act,dy", KINDS)
def test_backward(tokens, k, n, t, act, dy):
    _check_backward(*_backward(tokens, k, n, t, act, dy), t, act)


@pytest.mark.parametrize("tokens,k,n", sorted(set(linear_forms.DX + linear_forms.DW)))
@pytest.mark.parametrize("t,act,dy", KINDS[:2])
def test_backward_in_every_form(tokens, k, n, t, act, dy):
    _check_backward(*_backward(tokens, k, n, t, act, dy), t, act)


# few outputs and many tokens: dw over shares of the tokens, of lone CTAs and pairs, narrow and wide
SHARES = linear_forms.SHARES


def test_the_sizes_deal_the_tokens_out():
    assert linear_forms.dealt() >= linear_forms.DEALT


@pytest.mark.parametrize("tokens,k,n", SHARES)
@pytest.mark.parametrize("t,act,dy", KINDS[:2])
def test_backward_over_shares_of_the_tokens(tokens, k, n, t, act, dy):
    got = _backward(tokens, k, n, t, act, dy)
    _check_backward(*got, t, act)


def test_a_handle_for_more_tokens_serves_fewer():
    """Its room for shares is that of its largest call."""
    for tokens, room in ((700, 40000), (9000, 100000), (5, 30000)):
        _check_backward(*_backward(tokens, 128, 136, "bf16", "gelu", "f32", room=room), "bf16", "gelu")


@pytest.mark.parametrize("want", [("dx",), ("dw",), ("db",), ("dx", "dw"), ("dx", "db"), ("dw", "db")])
@pytest.mark.parametrize("t,act,dy", KINDS)
def test_backward_of_some_of_the_gradients(t, act, dy, want):
    import torch
    full = _backward(300, 136, 200, t, act, dy)[4]
    some = _backward(300, 136, 200, t, act, dy, want=want)[4]
    assert all(torch.equal(some[name], full[name]) if name in want else some[name] is None for name in full)


@pytest.mark.parametrize("rows,cols", [(1, 8), (2, 8), (700, 8), (50001, 16), (33, 264), (9, 4096), (20000, 264), (3001, 20000)])
@pytest.mark.parametrize("t,act,dy", KINDS)
def test_db_of_every_shape(rows, cols, t, act, dy):
    _check_backward(*_backward(rows, 8, cols, t, act, dy, want=("db",)), t, act)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_infinite_and_large_z_have_slopes_of_0_and_1(act):
    """fp16's z overflows to infinity past 65504.  SiLU's slope at -60 is p (1 - 60 (1 - p)) with p = e^-60 =
    8.8e-27, so -5.2e-25, and GELU's far less: below the 4e-7 that the evaluation may be off by, as is dy = 2 times it."""
    import torch
    pkg = _pkg()
    z = torch.tensor([[float("inf"), float("-inf"), 60.0, -60.0, 65504.0, -65504.0, 0.0, float("nan")]], device="cuda").half()
    dy, x, w = torch.full((1, 8), 2.0, device="cuda").half(), torch.ones(1, 8, device="cuda").half(), torch.eye(8, device="cuda").half()
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(8, device="cuda")
    op = pkg.tfl_linear_create(8, 8, 1, 1, _code(act), 1, 1)
    pkg.tfl_linear_backward(op, 1, P(x), P(w), P(z), P(dy), P(dx), P(dw), P(db), _stream())
    torch.cuda.synchronize()
    pkg.tfl_linear_destroy(op)
    want = torch.tensor([2.0, 0, 2, 0, 2, 0, 1], device="cuda")
    assert (db[:7] - want).abs().max() <= 2 * 4e-7 and db[7].isnan()
    assert torch.equal(dw[:7, 0], want.half()) and dw[7].isnan().all()


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_backward_is_the_forwards_difference_quotient(act):
    """Along a direction in x, from the kernel's own fp32 y: each y is off by its bound, so the quotient of
    L = sum(dy y) by the bounds' sum over h; the h^2 term is the reference's own."""
    import torch
    pkg = _pkg()
    tokens, k, n, t = 6, 64, 48, "f16"
    c = Case(tokens, k, n, t, "f32", act, True, False, act != "none", seed=8).run()
    gen = torch.Generator(device="cuda").manual_seed(1)
    dy = torch.randn(tokens, n, generator=gen, device="cuda")
    v = torch.randn(tokens, k, generator=gen, device="cuda").half()
    step = 2.0 ** -3
    op = c.create(tokens, "f32")
    dx, dw, db = torch.empty_like(c.x), torch.empty_like(c.w), torch.empty_like(c.bias)
    pkg.tfl_linear_backward(op, tokens, P(c.x), P(c.w), P(c.z), P(dy), P(dx), P(dw), P(db), _stream())
    torch.cuda.synchronize()
    N = lambda a: a.double().cpu().numpy()  # noqa: E731
    x0, g, w, b = c.x.clone(), N(dy), N(c.w), N(c.bias)

    def loss(sign):
        c.x = (x0 + sign * step * v).contiguous()
        c.forward(op)
        y, z = ops.linear(N(c.x), w, b, None, act)
        own = (k / 16 + 16) * ACC * (np.abs(N(c.x)) @ np.abs(w).T) + 2 * E * (np.abs(z) + np.abs(b))
        own = 1.13 * own + (2.0 ** -20 + 3 * E) * np.abs(y) + 4e-7 * (1 + np.abs(z))
        return N(c.x), np.sum(N(c.y[:tokens]) * g), np.sum(y * g), np.sum(own * np.abs(g))

    up, down = loss(1), loss(-1)
    pkg.tfl_linear_destroy(op)
    moved = up[0] - down[0]  # the points as fp16 holds them
    q, qref, noise = (up[1] - down[1]) / 2, (up[2] - down[2]) / 2, (up[3] + down[3]) / 2
    assert abs(q - qref) <= noise
    ref = ops.linear_backward(N(x0), w, ops.linear(N(x0), w, b, None, act)[1], g, act)[0]
    along, ref_along = np.sum(N(dx) * moved) / 2, np.sum(ref * moved) / 2
    # z's own rounding, dz's and dx's, each u of what it rounds
    slack = 4 * U[t] * np.sum(np.abs(ref * moved)) / 2 + 1e-3 + U[t] * np.sum((np.abs(g) @ np.abs(w)) * np.abs(moved))
    assert abs(along - ref_along) <= slack
    assert abs(along - q) <= noise + abs(qref - ref_along) + slack


@pytest.mark.parametrize("tokens,k,n", [(4, 128, 136), (150, 128, 136)] + linear_forms.FORWARD[1:5])
def test_rows_do_not_affect_one_another(tokens, k, n):
    import torch
    pkg = _pkg()
    bad = sorted({1, min(127, tokens - 1), tokens // 2, tokens - 2})
    c = Case(tokens, k, n, "bf16", "bf16", "gelu", True, True, True)
    dy = torch.randn(tokens, n, device="cuda").bfloat16()
    op, out = c.create(tokens, "bf16"), []
    for dirty in (False, True):
        if dirty:
            c.x[bad, 3] = float("nan")
            c.x[bad[0], 5] = float("inf")
            c.res[bad, 1] = float("nan")
            dy[bad, 2] = float("nan")
        dx, dw, db = torch.empty_like(c.x), torch.empty_like(c.w), torch.empty_like(c.bias)
        c.y.zero_(), c.z.zero_()
        c.forward(op)
        pkg.tfl_linear_backward(op, tokens, P(c.x), P(c.w), P(c.z), P(dy), P(dx), P(dw), P(db), _stream())
        out.append((c.y[:tokens].clone(), c.z[:tokens].clone(), dx))
    assert pkg.tfl_linear_status(op, _stream()) == 0
    pkg.tfl_linear_destroy(op)
    keep = torch.ones(tokens, dtype=torch.bool, device="cuda")
    keep[bad] = False
    for clean, dirty in zip(*out):
        assert torch.equal(clean[keep], dirty[keep]) and dirty[bad].isnan().any(dim=1).all()


def test_same_bits_every_time_captured_and_replayed_on_another_stream():
    import torch
    pkg = _pkg()
    for tokens, k, n, dy in ((700, 320, 456, "bf16"), (5, 320, 456, "f32"), (40, 2048, 136, "f32")):
        x, w, z, g, want = _backward(tokens, k, n, "bf16", "silu", dy, seed=3)
        c = Case(tokens, k, n, "bf16", "f32", "silu", True, True, True).run()
        y, zz = c.y.clone(), c.z.clone()
        op = pkg.tfl_linear_create(k, n, 2, 0, _code("silu"), _code(dy), tokens)
        out = {name: torch.empty_like(v) for name, v in want.items()}
        st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=st):
            c.forward(op, st.cuda_stream)
            pkg.tfl_linear_backward(op, tokens, P(x), P(w), P(z), P(g), P(out["dx"]), P(out["dw"]), P(out["db"]), st.cuda_stream)
        for _ in range(2):
            for v in (c.y, c.z, *out.values()):
                v.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(c.y, y) and torch.equal(c.z, zz)
            assert all(torch.equal(out[name], want[name]) for name in want)
        assert pkg.tfl_linear_status(op, _stream()) == 0
        pkg.tfl_linear_destroy(op)


def test_forwards_of_one_handle_may_overlap():
    import torch
    pkg = _pkg()
    cases = [Case(3 if i % 2 else 1500, 256, 512, "bf16", "bf16", "gelu", True, True, True, seed=i).run() for i in range(6)]
    op = cases[0].create()
    refs = [(c.y.clone(), c.z.clone()) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for c in cases:
        c.y.zero_(), c.z.zero_()
    torch.cuda.synchronize()
    for c, st in zip(cases, streams):
        c.forward(op, st.cuda_stream)
    torch.cuda.synchronize()
    for c, (y, z) in zip(cases, refs):
        assert torch.equal(c.y[:c.tokens], y[:c.tokens]) and torch.equal(c.z[:c.tokens], z[:c.tokens])
    pkg.tfl_linear_destroy(op)


def test_no_tokens():
    import torch
    pkg = _pkg()
    op = pkg.tfl_linear_create(64, 64, 2, 2, 1, 2, 4)
    dw, db = torch.ones(64, 64, device="cuda").bfloat16(), torch.ones(64, device="cuda")
    pkg.tfl_linear_forward(op, 0, None, None, None, None, None, None, None, None, _stream())
    pkg.tfl_linear_backward(op, 0, None, None, None, None, None, P(dw), P(db), _stream())
    torch.cuda.synchronize()
    assert (dw == 0).all() and (db == 0).all()
    pkg.tfl_linear_destroy(op)


def test_refusals():
    import torch
    pkg = _pkg()
    op = pkg.tfl_linear_create(64, 128, 2, 2, _code("gelu"), 2, 4)
    plain = pkg.tfl_linear_create(64, 128, 2, 0, _code("none"), 0, 4)
    q = pkg.tfl_linear_create(64, 128, 3, 2, _code("gelu"))
    x, w = torch.zeros(8, 64, device="cuda").bfloat16(), torch.zeros(128, 64, device="cuda").bfloat16()
    res, z, y, dy = (torch.zeros(8, 128, device="cuda").bfloat16() for _ in range(4))
    y32, dy32 = torch.zeros(8, 128, device="cuda"), torch.zeros(8, 128, device="cuda")
    b, s, db = torch.zeros(128, device="cuda"), torch.ones(256, device="cuda"), torch.zeros(128, device="cuda")
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)

    def refused(fn, *args, code=pkg.TFL_ERR_INVALID_ARG):
        with pytest.raises(pkg.TflError) as e:
            fn(*args, _stream())
        assert e.value.code == code and str(e.value)

    f, k = pkg.tfl_linear_forward, pkg.tfl_linear_backward
    good = [P(x), None, P(w), None, P(b), P(res), P(z), P(y)]
    refused(f, None, 4, *good)
    refused(f, op, -1, *good)
    refused(f, op, 2 ** 31, *good)
    for i in (0, 2, 7):
        refused(f, op, 4, *good[:i], None, *good[i + 1:])
    for i in (0, 2, 4, 5, 6, 7):
        refused(f, op, 4, *good[:i], good[i] + 8, *good[i + 1:])
    refused(f, op, 4, P(x), P(s), P(w), P(s), P(b), None, None, P(y))     # scales without e4m3
    refused(f, q, 4, P(x), None, P(w), None, P(b), None, None, P(y))      # e4m3 without scales
    refused(f, q, 4, P(x), P(s), P(w), P(s), P(b), None, P(z), P(y))      # z of e4m3 operands
    refused(f, q, 4, P(x), P(s), P(w), P(s) + 4, P(b), None, None, P(y))
    refused(f, plain, 4, P(x), None, P(w), None, P(b), None, P(z), P(y32))  # z without an activation
    refused(f, op, 4, *good[:7], P(x))
    refused(f, op, 4, *good[:7], P(z))
    refused(f, op, 4, *good[:6], P(res), P(y))                            # z over the residual
    refused(f, op, 4, *good[:7], P(res) + 128)                            # shifted over the residual
    refused(f, op, 4, *good[:7], P(w) + 128)
    refused(f, op, 4, *good[:6], P(b), P(y))
    good = [P(x), P(w), P(z), P(dy), P(dx), P(dw), P(db)]
    refused(k, None, 4, *good)
    refused(k, op, 5, *good)                                              # more than it has room for
    for i in (0, 1, 2, 3):
        refused(k, op, 4, *good[:i], None, *good[i + 1:])
    for i in range(7):
        refused(k, op, 4, *good[:i], good[i] + 8, *good[i + 1:])
    refused(k, op, 4, *good[:4], None, None, None)
    refused(k, op, 4, *good[:4], P(x), *good[5:])
    refused(k, op, 4, *good[:5], P(dx), P(db))
    refused(k, op, 4, *good[:6], P(dy))
    refused(k, plain, 4, P(x), P(w), P(z), P(dy32), *good[4:])            # z without an activation
    refused(k, q, 0, *good, code=pkg.TFL_ERR_UNSUPPORTED)
    assert pkg.tfl_linear_status(op, _stream()) == 0
    for h in (op, plain, q):
        pkg.tfl_linear_destroy(h)
