"""The operators of a block used together, as a program would: a pre-norm block's training step
(norm, attention, norm, gated feed-forward and back), and its 8-bit feed-forward half.

The projections around them are torch matrix products in fp32 on the same 16-bit values.  The
reference runs the same block in float64 under autograd.  Bounds are on the 2-norm: with u = 2^-11
(fp16's half step), every 16-bit tensor on the way (x, qkv, o, y, h, their gradients, P and dS
inside attention) is rounded at most once more, with an rms of at most u / sqrt 3 relative to it;
a gradient passes at most 14 such roundings, whose independent errors add in squares: at most
sqrt 14 / sqrt 3 u = 2.2 u, and parts of it pass through layers that enlarge an error (the norm's
division by a smaller rms, the softmax's slope) by at most 4 here: 9 u.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -11
EPS = 1e-5


def _rel(u, r):
    u, r = u.double().cpu(), r.double().cpu()
    assert u.isfinite().all()
    return float((u - r).norm() / r.norm())


def _reference(p, B, S, H, hd, causal, lens):
    """out and the gradients of every leaf, in float64."""
    import torch
    leaves = {k: v.double().detach().requires_grad_() for k, v in p.items() if k != "dout"}

    def norm(s, g):
        return s / torch.sqrt((s * s).mean(-1, keepdim=True) + EPS) * g

    q = leaves
    D = H * hd
    y1 = norm(q["x"], q["g1"])
    qkv = (y1 @ q["wqkv"].t()).view(B, S, 3, H, hd)
    qq, kk, vv = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    sc = qq @ kk.transpose(-1, -2) / hd ** 0.5
    j = torch.arange(S, device=sc.device)
    mask = (j[None, None, :] < lens[:, None, None]).expand(B, S, S)
    if causal:
        mask = mask & (j[None, None, :] <= j[None, :, None])
    sc = sc.masked_fill(~mask[:, None], float("-inf"))
    o = (sc.softmax(-1) @ vv).transpose(1, 2).reshape(B * S, D)
    valid = (j[None, :] < lens[:, None]).reshape(-1, 1)
    o = torch.where(valid, o, torch.zeros_like(o))
    a = o @ q["wo"].t()
    s2 = q["x"] + a
    y2 = norm(s2, q["g2"])
    h = torch.nn.functional.silu(y2 @ q["wg"].t()) * (y2 @ q["wu"].t())
    out = s2 + h @ q["wd"].t()
    dout = p["dout"].double() * valid
    grads = torch.autograd.grad(out, list(leaves.values()), dout)
    return out.detach(), dict(zip(leaves, grads)), valid


@pytest.mark.parametrize("causal,lens", [(True, [200, 131]), (False, [200, 57])])
def test_a_training_step_of_a_block(causal, lens):
    import torch
    import attention_qkv_gemm_gb300 as pkg
    B, S, H, hd, F = 2, 200, 4, 64, 712
    D, T = H * hd, B * S
    gen = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device="cuda") * std).half()  # noqa: E731
    p = {"x": rnd(T, D), "g1": 1 + 0.1 * rnd(D).float(), "g2": 1 + 0.1 * rnd(D).float(),
         "wqkv": rnd(3 * D, D, std=D ** -0.5), "wo": rnd(D, D, std=D ** -0.5), "wg": rnd(F, D, std=D ** -0.5),
         "wu": rnd(F, D, std=D ** -0.5), "wd": rnd(D, F, std=F ** -0.5), "dout": rnd(T, D)}
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ref, rgrad, valid = _reference(p, B, S, H, hd, causal, ln.long())
    mm = lambda a, b: (a.float() @ b.float()).half()  # noqa: E731
    st = torch.cuda.current_stream().cuda_stream
    P = lambda t: t.data_ptr()  # noqa: E731
    new = lambda *s, t=torch.float16: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    n = pkg.tfl_rmsnorm_create(D, pkg.TFL_F16, pkg.TFL_F16, pkg.TFL_F16, EPS)
    at = pkg.tfl_attn_create(B, S, H, hd)
    ff = pkg.tfl_glu_create(D, F, pkg.TFL_F16, pkg.TFL_F16, pkg.TFL_ACT_SILU, T)
    try:
        # forward
        y1, o, lse, s2, y2, h = new(T, D), new(T, D), new(B, H, S, t=torch.float32), new(T, D), new(T, D), new(T, F)
        pkg.tfl_rmsnorm_forward(n, T, P(p["x"]), None, P(p["g1"]), None, P(y1), None, st)
        qkv = mm(y1, p["wqkv"].t())
        pkg.tfl_attn_forward(at, P(qkv), P(ln), int(causal), P(o), P(lse), st)
        o = torch.where(valid, o, torch.zeros_like(o))
        a = mm(o, p["wo"].t())
        pkg.tfl_rmsnorm_forward(n, T, P(a), P(p["x"]), P(p["g2"]), P(s2), P(y2), None, st)
        pkg.tfl_glu_forward(ff, T, P(y2), None, P(p["wg"]), None, P(p["wu"]), None, P(h), st)
        out = s2.float() + h.float() @ p["wd"].float().t()
        # backward
        dout = torch.where(valid, p["dout"], torch.zeros_like(p["dout"]))
        g = {"wd": mm(dout.t(), h)}
        dh = mm(dout, p["wd"])
        dy2, g["wg"], g["wu"] = new(T, D), new(F, D), new(F, D)
        pkg.tfl_glu_backward(ff, T, P(y2), P(p["wg"]), P(p["wu"]), P(dh), P(dy2), P(g["wg"]), P(g["wu"]), st)
        ds2, g["g2"], g["g1"] = new(T, D), new(D, t=torch.float32), new(D, t=torch.float32)
        pkg.tfl_rmsnorm_backward(n, T, P(s2), P(p["g2"]), P(dy2), P(dout), P(ds2), None, P(g["g2"]), st)
        g["wo"] = mm(ds2.t(), o)
        do = mm(ds2, p["wo"])
        dqkv = new(T, 3 * D, t=torch.float32)
        pkg.tfl_attn_backward(at, P(qkv), P(o), P(do), P(lse), P(ln), int(causal), P(dqkv), st)
        dqkv = dqkv.half()
        g["wqkv"] = mm(dqkv.t(), y1)
        dy1 = mm(dqkv, p["wqkv"])
        g["x"] = new(T, D)
        pkg.tfl_rmsnorm_backward(n, T, P(p["x"]), P(p["g1"]), P(dy1), P(ds2), P(g["x"]), None, P(g["g1"]), st)
        assert pkg.tfl_attn_status(at, st) == 0 and pkg.tfl_glu_status(ff, st) == 0
    finally:
        pkg.tfl_rmsnorm_destroy(n)
        pkg.tfl_attn_destroy(at)
        pkg.tfl_glu_destroy(ff)
    rows = valid.reshape(-1)
    assert _rel(out[rows], ref[rows]) <= 9 * U
    for k, v in g.items():
        assert _rel(v, rgrad[k]) <= 9 * U, (k, _rel(v, rgrad[k]) / U)


@pytest.mark.parametrize("tokens", [1, 5, 70, 700])
def test_the_norms_8_bit_rows_feed_the_feed_forward(tokens):
    """fp32 residual stream, e4m3 rows and weights.  The feed-forward's own error is checked against
    the values its 8-bit operands stand for; against the unquantised block, the e4m3 roundings of y
    and of the weights (half a step 2^-4, rms at most 2^-4 / sqrt 3 = 0.036 each) reach h through
    both projections: sqrt(2 (0.036^2 + 0.036^2)) = 0.073, with act' up to 1.13: 0.085."""
    import torch
    import attention_qkv_gemm_gb300 as pkg
    D, F = 512, 1040
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=gen, device="cuda") * std  # noqa: E731

    def rows8(t):
        sc = t.abs().amax(dim=1) / 448
        return (t / sc[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn), sc

    x, res, gamma = rnd(tokens, D).bfloat16(), rnd(tokens, D), 1 + 0.1 * rnd(D)
    wg, wu = rnd(F, D, std=D ** -0.5), rnd(F, D, std=D ** -0.5)
    (qg, sg), (qu, su) = rows8(wg), rows8(wu)
    st = torch.cuda.current_stream().cuda_stream
    P = lambda t: t.data_ptr()  # noqa: E731
    y, ys = torch.empty(tokens, D, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(tokens, device="cuda")
    out, h = torch.empty_like(res), torch.empty(tokens, F, dtype=torch.bfloat16, device="cuda")
    n = pkg.tfl_rmsnorm_create(D, pkg.TFL_BF16, pkg.TFL_F32, pkg.TFL_E4M3, EPS)
    ff = pkg.tfl_glu_create(D, F, pkg.TFL_E4M3, pkg.TFL_BF16, pkg.TFL_ACT_GELU)
    pkg.tfl_rmsnorm_forward(n, tokens, P(x), P(res), P(gamma), P(out), P(y), P(ys), st)
    pkg.tfl_glu_forward(ff, tokens, P(y), P(ys), P(qg), P(sg), P(qu), P(su), P(h), st)
    assert pkg.tfl_glu_status(ff, st) == 0
    pkg.tfl_rmsnorm_destroy(n)
    pkg.tfl_glu_destroy(ff)

    def glu(a, b, c):
        return torch.nn.functional.gelu(a @ b.t()) * (a @ c.t())

    stands = glu(y.double() * ys.double()[:, None], qg.double() * sg.double()[:, None], qu.double() * su.double()[:, None])
    assert _rel(h, stands) <= 2.0 ** -8
    s = x.double() + res.double()
    plain = glu(s / torch.sqrt((s * s).mean(-1, keepdim=True) + EPS) * gamma.double(), wg.double(), wu.double())
    assert _rel(h, plain) <= 0.085
    np.testing.assert_allclose(out.double().cpu().numpy(), s.cpu().numpy(), rtol=2.0 ** -23)
