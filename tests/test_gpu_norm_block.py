"""Layer norm and the linear layer used with the attention operator, as a program would: a training step of
one of the stack's own pre-norm blocks (every product, norm and gradient from this library), and the 8-bit
rows that the norm writes fed to a projection.

The reference runs the same block in float64 under autograd.  Bounds are on the 2-norm: with u = 2^-11
(fp16's half step), every 16-bit tensor on the way is rounded at most once more, with an rms of at most
u / sqrt 3 relative to it.  The gradient of the input passes the most of them, 18: y1, qkv, P, o, a, y2, z, h,
the 16-bit dz of four layers, dh, dy2, ds, do, dS and dy1, whose independent errors add in squares:
sqrt 18 / sqrt 3 u = 2.45 u; parts of it pass through layers that enlarge an error (the norm's division, the
softmax's slope) by at most 4 here: 10 u.
"""
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -11
EPS = 1e-5


def _rel(u, r):
    u, r = u.double(), r.double()
    assert u.isfinite().all()
    return float((u - r).norm() / r.norm())


def P(t):
    return None if t is None else t.data_ptr()


def _reference(p, B, S, H, hd, causal, lens):
    """out and the gradients of every leaf, in float64."""
    import torch
    q = {k: v.double().detach().requires_grad_() for k, v in p.items() if k != "dout"}
    D = H * hd
    norm = torch.nn.functional.layer_norm
    lin = torch.nn.functional.linear
    y1 = norm(q["x"], (D,), q["g1"], q["be1"], EPS)
    qkv = lin(y1, q["wqkv"], q["bqkv"]).view(B, S, 3, H, hd)
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
    s2 = q["x"] + lin(o, q["wo"], q["bo"])
    h = torch.nn.functional.gelu(lin(norm(s2, (D,), q["g2"], q["be2"], EPS), q["w1"], q["b1"]))
    out = s2 + lin(h, q["w2"], q["b2"])
    grads = torch.autograd.grad(out, list(q.values()), p["dout"].double() * valid)
    return out.detach(), dict(zip(q, grads)), valid


@pytest.mark.parametrize("causal,lens", [(True, [200, 131]), (False, [200, 57])])
@pytest.mark.parametrize("captured", [False, True])
def test_a_training_step_of_the_stacks_block(causal, lens, captured):
    import torch
    import attention_qkv_gemm_gb300 as pkg
    B, S, H, hd, F = 2, 200, 4, 64, 1032
    D, T = H * hd, B * S
    gen = torch.Generator(device="cuda").manual_seed(0)
    f32 = lambda *s, std=1.0: torch.randn(*s, generator=gen, device="cuda") * std  # noqa: E731
    rnd = lambda *s, std=1.0: f32(*s, std=std).half()  # noqa: E731
    p = {"x": rnd(T, D), "g1": 1 + f32(D, std=0.1), "be1": f32(D, std=0.1), "g2": 1 + f32(D, std=0.1), "be2": f32(D, std=0.1),
         "wqkv": rnd(3 * D, D, std=D ** -0.5), "bqkv": f32(3 * D, std=0.1), "wo": rnd(D, D, std=D ** -0.5), "bo": f32(D, std=0.1),
         "w1": rnd(F, D, std=D ** -0.5), "b1": f32(F, std=0.1), "w2": rnd(D, F, std=F ** -0.5), "b2": f32(D, std=0.1),
         "dout": f32(T, D)}
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ref, rgrad, valid = _reference(p, B, S, H, hd, causal, ln.long())
    dout = torch.where(valid, p["dout"], torch.zeros_like(p["dout"]))
    x32, rows = p["x"].float(), valid.reshape(-1)
    new = lambda *s, t=torch.float16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    F16, F32, NONE, GELU = pkg.TFL_F16, pkg.TFL_F32, pkg.TFL_ACT_NONE, pkg.TFL_ACT_GELU
    n1, n2 = pkg.tfl_layernorm_create(D, F16, F16, F16, EPS), pkg.tfl_layernorm_create(D, F16, F32, F16, EPS)
    at = pkg.tfl_attn_create(B, S, H, hd)
    lqkv = pkg.tfl_linear_create(D, 3 * D, F16, F16, NONE, F32, T)
    lo = pkg.tfl_linear_create(D, D, F16, F16, NONE, F16, T)
    l1 = pkg.tfl_linear_create(D, F, F16, F16, GELU, F16, T)
    l2 = pkg.tfl_linear_create(F, D, F16, F32, NONE, F32, T)
    b = {"y1": new(T, D), "st1": new(T, 2, t=torch.float32), "qkv": new(T, 3 * D), "o": new(T, D), "lse": new(B, H, S, t=torch.float32),
         "a": new(T, D), "s2": new(T, D, t=torch.float32), "y2": new(T, D), "st2": new(T, 2, t=torch.float32), "z": new(T, F),
         "h": new(T, F), "out": new(T, D, t=torch.float32), "dh": new(T, F), "dy2": new(T, D), "ds16": new(T, D),
         "ds": new(T, D, t=torch.float32), "do": new(T, D), "dqkv": new(T, 3 * D, t=torch.float32), "dy1": new(T, D)}
    g = {k: torch.zeros_like(v) for k, v in p.items() if k != "dout"}

    def step(st):
        v = {k: P(t) for k, t in (*p.items(), *b.items())}
        G = {k: P(t) for k, t in g.items()}
        pkg.tfl_layernorm_forward(n1, T, v["x"], None, v["g1"], v["be1"], None, v["y1"], None, v["st1"], st)
        pkg.tfl_linear_forward(lqkv, T, v["y1"], None, v["wqkv"], None, v["bqkv"], None, None, v["qkv"], st)
        pkg.tfl_attn_forward(at, v["qkv"], P(ln), int(causal), v["o"], v["lse"], st)
        b["o"].mul_(valid)  # padding rows of o are unspecified (finite here)
        pkg.tfl_linear_forward(lo, T, v["o"], None, v["wo"], None, v["bo"], None, None, v["a"], st)
        pkg.tfl_layernorm_forward(n2, T, v["a"], P(x32), v["g2"], v["be2"], v["s2"], v["y2"], None, v["st2"], st)
        pkg.tfl_linear_forward(l1, T, v["y2"], None, v["w1"], None, v["b1"], None, v["z"], v["h"], st)
        pkg.tfl_linear_forward(l2, T, v["h"], None, v["w2"], None, v["b2"], v["s2"], None, v["out"], st)
        pkg.tfl_linear_backward(l2, T, v["h"], v["w2"], None, P(dout), v["dh"], G["w2"], G["b2"], st)
        pkg.tfl_linear_backward(l1, T, v["y2"], v["w1"], v["z"], v["dh"], v["dy2"], G["w1"], G["b1"], st)
        pkg.tfl_layernorm_backward(n2, T, v["s2"], v["st2"], v["g2"], v["dy2"], P(dout), v["ds16"], v["ds"], G["g2"], G["be2"], st)
        pkg.tfl_linear_backward(lo, T, v["o"], v["wo"], None, v["ds16"], v["do"], G["wo"], G["bo"], st)
        pkg.tfl_attn_backward(at, v["qkv"], v["o"], v["do"], v["lse"], P(ln), int(causal), v["dqkv"], st)
        pkg.tfl_linear_backward(lqkv, T, v["y1"], v["wqkv"], None, v["dqkv"], v["dy1"], G["wqkv"], G["bqkv"], st)
        pkg.tfl_layernorm_backward(n1, T, v["x"], v["st1"], v["g1"], v["dy1"], v["ds16"], G["x"], None, G["g1"], G["be1"], st)

    try:
        if captured:
            st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=st):
                step(st.cuda_stream)
            for _ in range(2):
                for t in (*b.values(), *g.values()):
                    t.zero_()
                graph.replay()
        else:
            step(torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert pkg.tfl_attn_status(at) == 0 and all(pkg.tfl_linear_status(h) == 0 for h in (lqkv, lo, l1, l2))
    finally:
        for h in (n1, n2):
            pkg.tfl_layernorm_destroy(h)
        for h in (lqkv, lo, l1, l2):
            pkg.tfl_linear_destroy(h)
        pkg.tfl_attn_destroy(at)
    assert _rel(b["out"][rows], ref[rows]) <= 10 * U
    for k, v in g.items():
        if k == "bqkv":  # the keys' bias moves all of a row's scores alike: its gradient is 0 but for rounding
            kb = slice(D, 2 * D)
            assert float((v[kb].double() - rgrad[k][kb]).norm()) <= 10 * U * float(rgrad[k].norm())
            v, rgrad[k] = (torch.cat((t[:D], t[2 * D:])) for t in (v, rgrad[k]))
        assert _rel(v, rgrad[k]) <= 10 * U, (k, _rel(v, rgrad[k]) / U)


@pytest.mark.parametrize("tokens", [1, 5, 70, 700])
def test_the_norms_8_bit_rows_feed_a_projection(tokens):
    """fp32 residual stream, e4m3 rows and weight.  The projection's own error is checked against the values its
    8-bit operands stand for; against the unquantised layers, the e4m3 roundings of y and of the weight (half a
    step 2^-4, rms at most 2^-4 / sqrt 3 = 0.036 each) make sqrt(0.036^2 + 0.036^2) = 0.051 of x W^T."""
    import torch
    import attention_qkv_gemm_gb300 as pkg
    D, N = 512, 1040
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=gen, device="cuda") * std  # noqa: E731
    x, res, gamma, beta = rnd(tokens, D).bfloat16(), rnd(tokens, D) + 0.5, 1 + 0.1 * rnd(D), 0.1 * rnd(D)
    w, bias = rnd(N, D, std=D ** -0.5), rnd(N, std=0.1)
    sw = w.abs().amax(dim=1) / 448
    q = (w / sw[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    st = torch.cuda.current_stream().cuda_stream
    y, ys = torch.empty(tokens, D, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(tokens, device="cuda")
    out, z = torch.empty_like(res), torch.empty(tokens, N, dtype=torch.bfloat16, device="cuda")
    n = pkg.tfl_layernorm_create(D, pkg.TFL_BF16, pkg.TFL_F32, pkg.TFL_E4M3, EPS)
    l = pkg.tfl_linear_create(D, N, pkg.TFL_E4M3, pkg.TFL_BF16)
    pkg.tfl_layernorm_forward(n, tokens, P(x), P(res), P(gamma), P(beta), P(out), P(y), P(ys), None, st)
    pkg.tfl_linear_forward(l, tokens, P(y), P(ys), P(q), P(sw), P(bias), None, None, P(z), st)
    assert pkg.tfl_linear_status(l, st) == 0
    pkg.tfl_layernorm_destroy(n)
    pkg.tfl_linear_destroy(l)
    lin = torch.nn.functional.linear
    assert _rel(z, lin(y.double() * ys.double()[:, None], q.double() * sw.double()[:, None], bias.double())) <= 2.0 ** -8
    plain = torch.nn.functional.layer_norm(x.double() + res.double(), (D,), gamma.double(), beta.double(), EPS)
    err = (z.double() - lin(plain, w.double(), bias.double())).norm() / lin(plain, w.double()).norm()
    assert float(err) <= 0.051 + 2.0 ** -8


TURNS = 40


@pytest.mark.parametrize("tokens,d,f", [(1, 1024, 1040), (1, 4096, 512), (8, 2048, 2080), (16, 512, 2048), (40, 4096, 2048),
                                        (200, 1024, 2048), (1500, 512, 2064)])
def test_turns_on_the_same_buffers_equal_turns_alone(tokens, d, f):
    """A norm and the two halves of a feed-forward behind it, turn after turn without a pause: each kernel may
    start while the one before it still runs, so what it reads has to be the newest.  The residual stream is
    updated in place."""
    import torch
    import attention_qkv_gemm_gb300 as pkg
    gen = torch.Generator(device="cuda").manual_seed(tokens + d)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x = rnd(TURNS, tokens, d).bfloat16()
    gamma, beta, b1, b2 = 1 + 0.1 * rnd(d), 0.1 * rnd(d), 0.1 * rnd(f), 0.1 * rnd(d)
    w1, w2 = (rnd(f, d) * d ** -0.5).bfloat16(), (rnd(d, f) * f ** -0.5).bfloat16()
    n = pkg.tfl_layernorm_create(d, pkg.TFL_BF16, pkg.TFL_BF16, pkg.TFL_BF16, EPS)
    l1 = pkg.tfl_linear_create(d, f, pkg.TFL_BF16, pkg.TFL_BF16, pkg.TFL_ACT_GELU)
    l2 = pkg.tfl_linear_create(f, d, pkg.TFL_BF16, pkg.TFL_BF16)
    out = torch.empty_like(x)

    def buffers():
        y, h = torch.zeros(tokens, d, device="cuda").bfloat16(), torch.zeros(tokens, f, device="cuda").bfloat16()
        return y, h, torch.zeros(tokens, d, device="cuda").bfloat16()

    def turn(i, y, h, s, st):  # s: the residual stream, over all turns
        pkg.tfl_layernorm_forward(n, tokens, P(x[i]), P(s), P(gamma), P(beta), P(s), P(y), None, None, st)
        pkg.tfl_linear_forward(l1, tokens, P(y), None, P(w1), None, P(b1), None, None, P(h), st)
        pkg.tfl_linear_forward(l2, tokens, P(h), None, P(w2), None, P(b2), P(s), None, P(out[i]), st)

    def alone():
        stream, s = torch.cuda.current_stream().cuda_stream, buffers()[2]
        for i in range(TURNS):
            y, h, _ = buffers()
            torch.cuda.synchronize()
            turn(i, y, h, s, stream)
            torch.cuda.synchronize()
        return out.clone()

    try:
        ref = alone()
        y, h, s = buffers()
        out.zero_()
        for i in range(TURNS):
            turn(i, y, h, s, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
        st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            for i in range(TURNS):
                turn(i, y, h, s, st.cuda_stream)
        for _ in range(2):
            x.copy_(rnd(*x.shape))
            ref = alone()
            out.zero_(), s.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, ref)
        assert pkg.tfl_linear_status(l1) == 0 and pkg.tfl_linear_status(l2) == 0
    finally:
        pkg.tfl_layernorm_destroy(n)
        pkg.tfl_linear_destroy(l1)
        pkg.tfl_linear_destroy(l2)


def test_backwards_of_two_handles_may_overlap():
    import torch
    import attention_qkv_gemm_gb300 as pkg
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    T, K, N = 900, 264, 520
    calls = []
    for _ in range(3):
        x, w, z, dy = rnd(T, K).bfloat16(), rnd(N, K).bfloat16(), rnd(T, N).bfloat16(), rnd(T, N)
        s, stats, gamma, dn = rnd(T, K), torch.stack([rnd(T), 1 + rnd(T).abs()], 1), rnd(K), rnd(T, K).bfloat16()
        l = pkg.tfl_linear_create(K, N, pkg.TFL_BF16, pkg.TFL_BF16, pkg.TFL_ACT_SILU, pkg.TFL_F32, T)
        n = pkg.tfl_layernorm_create(K, pkg.TFL_BF16, pkg.TFL_F32, pkg.TFL_BF16, EPS)
        out = [torch.zeros_like(x), torch.zeros_like(w), torch.zeros(N, device="cuda"), torch.zeros_like(x), torch.zeros_like(s),
               torch.zeros(K, device="cuda"), torch.zeros(K, device="cuda")]

        def run(st, l=l, n=n, t=(x, w, z, dy, s, stats, gamma, dn), out=out):
            x, w, z, dy, s, stats, gamma, dn = t
            pkg.tfl_linear_backward(l, T, P(x), P(w), P(z), P(dy), *(P(o) for o in out[:3]), st)
            pkg.tfl_layernorm_backward(n, T, P(s), P(stats), P(gamma), P(dn), None, *(P(o) for o in out[3:]), st)
        run(torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        calls.append((run, out, [o.clone() for o in out], torch.cuda.Stream(), l, n))
    for _, out, *_ in calls:
        for o in out:
            o.zero_()
    torch.cuda.synchronize()
    for _ in range(4):
        for run, _, _, st, *_ in calls:
            run(st.cuda_stream)
    torch.cuda.synchronize()
    for _, out, ref, _, l, n in calls:
        assert all(torch.equal(a, r) for a, r in zip(out, ref))
        assert pkg.tfl_linear_status(l) == 0
        pkg.tfl_linear_destroy(l)
        pkg.tfl_layernorm_destroy(n)
