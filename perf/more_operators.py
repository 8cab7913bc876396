"""Layer norm and the linear layer with bias, activation and residual: cases, plain forms and work.

``ln``        s = x + res; y = (s - mean) / sqrt(var + eps) * gamma + beta; returns s (in the residual's
              type) and y, and for training each row's mean and 1 / sqrt(var + eps)
``ln8``       the same with y as e4m3 values and one float32 scale a row
``ln_grad``   the norm's gradients: of s (in x's type, and in the residual's where that differs), of gamma
              and of beta, from s, the rows' statistics, dy and the gradient that reaches s from later layers
``lin``       y = act(x W^T + b) + res, W as an nn.Linear weight [n, k]; for training also z = x W^T + b
``lin8``      the same from e4m3 x and W with one float32 scale a row of each
``lin_grad``  dx, dW, db from x, W, z and dy

``rows`` is the number of tokens, ``k`` and ``n`` the linear layer's input and output widths.  Types: f32,
f16, bf16; act: none, silu, gelu.
"""
import math

import torch

own = False

EPS = 1e-5
E4M3_MAX = 448.0
E4M3_MIN_AMAX = 2.0 ** -100

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one token of a generation step, residual stream in fp32
        {"name": "ln one token", "op": "ln", "rows": 1, "d": 1024, "x": "bf16", "res": "f32", "train": False},
        # a training step's forward: a batch of 16 prompts of 512 tokens
        {"name": "ln batch", "op": "ln", "rows": 8192, "d": 1024, "x": "f16", "res": "f32", "train": True},
        # one sequence of 100000 tokens, everything in bf16, rows for an 8-bit projection
        {"name": "ln8 long", "op": "ln8", "rows": 100000, "d": 1024, "x": "bf16", "res": "bf16", "train": False},
        # the same batch's backward
        {"name": "ln_grad batch", "op": "ln_grad", "rows": 8192, "d": 1024, "x": "bf16", "res": "f32"},
        # a ragged number of tokens of a width that no vector load divides
        {"name": "ln_grad odd width", "op": "ln_grad", "rows": 6011, "d": 1001, "x": "f16", "res": "f16"},
        # one token through the wider feed-forward projection: the weight is read for a single row
        {"name": "lin one token", "op": "lin", "rows": 1, "k": 1024, "n": 4096, "x": "bf16", "out": "bf16",
         "act": "gelu", "bias": True, "res": False, "train": False},
        # forty requests generating together: the narrower projection in 8 bits, added to the residual stream
        {"name": "lin8 generation", "op": "lin8", "rows": 40, "k": 10240, "n": 4096, "x": "bf16", "out": "bf16",
         "act": "none", "bias": True, "res": True, "train": False},
        # the fused q, k, v projection of a small model: 64 sequences of 1024 tokens, bound by memory
        {"name": "lin narrow", "op": "lin", "rows": 65536, "k": 128, "n": 384, "x": "f16", "out": "f16",
         "act": "none", "bias": True, "res": False, "train": False},
        # a training step's forward, which keeps z for the backward
        {"name": "lin batch", "op": "lin", "rows": 8192, "k": 1024, "n": 4096, "x": "f16", "out": "f16",
         "act": "gelu", "bias": True, "res": False, "train": True},
        # one sequence of 100000 tokens back onto the fp32 residual stream
        {"name": "lin long", "op": "lin", "rows": 100000, "k": 4096, "n": 1024, "x": "bf16", "out": "f32",
         "act": "none", "bias": True, "res": True, "train": False},
        # a training step's backward through the activation
        {"name": "lin_grad step", "op": "lin_grad", "rows": 16384, "k": 2048, "n": 8192, "x": "bf16", "dy": "bf16",
         "act": "gelu"},
        # a small model's, with sizes that no tile divides and the output's gradient in fp32
        {"name": "lin_grad ragged", "op": "lin_grad", "rows": 2979, "k": 1160, "n": 2856, "x": "f16", "dy": "f32",
         "act": "none"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["ln", "ln8", "ln_grad", "lin", "lin8", "lin_grad"])
    rows = _log(rng, 1, 100000)
    if op.startswith("ln"):
        x, res = rng.choice([("f32", "f32"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
        d = _log(rng, 64, 8192)
        if rng.random() < 0.75:
            d = (d + 7) // 8 * 8
        rows = max(1, min(rows, 40_000_000 // d))
        case = {"op": op, "rows": rows, "d": d, "x": x, "res": res}
        if op != "ln_grad":
            case["train"] = rng.random() < 0.5
        return case
    step = 16 if op == "lin8" else 8
    k = (_log(rng, 64, 10240) + step - 1) // step * step
    n = (_log(rng, 64, 10240) + step - 1) // step * step
    # no more products and no more values than the largest listed cases have
    if op == "lin_grad":
        rows = max(1, min(rows, int(1.0e12 / (4 * k * n)), 100_000_000 // (k + n)))
    else:
        rows = max(1, min(rows, int(0.8e12 / (2 * k * n)), 200_000_000 // (k + 2 * n)))
    x = rng.choice(["f16", "bf16"])
    case = {"op": op, "rows": rows, "k": k, "n": n, "x": x, "act": rng.choice(["none", "silu", "gelu"])}
    if op == "lin_grad":
        case["dy"] = rng.choice([x, "f32"])
    else:
        case["out"] = rng.choice([x, "f32"])
        case["bias"] = rng.random() < 0.75
        case["res"] = rng.random() < 0.5
        case["train"] = op == "lin" and case["act"] != "none" and rng.random() < 0.5
    return case


def work(case):
    r, op = case["rows"], case["op"]
    sx = SIZES[case["x"]]
    if op.startswith("ln"):
        d = case["d"]
        sr, n = SIZES[case["res"]], r * d
        if op == "ln_grad":
            outs = sx if sx == sr else sx + sr
            return {"bytes": n * (2 * sr + sx + outs) + 8 * r + 12 * d, "flops": 14 * n}
        stats = 8 * r if case["train"] else 0
        if op == "ln":
            return {"bytes": n * (2 * sx + 2 * sr) + stats + 8 * d, "flops": 8 * n}
        return {"bytes": n * (sx + 2 * sr + 1) + stats + 8 * d + 4 * r, "flops": 10 * n}
    k, n = case["k"], case["n"]
    if op == "lin_grad":
        values = sx * (2 * r * k + 2 * n * k) + SIZES[case["dy"]] * r * n + 4 * n
        return {"bytes": values + (0 if case["act"] == "none" else sx * r * n), "flops": 4 * r * k * n}
    so = SIZES[case["out"]]
    outs = so * r * n * (2 if case["res"] else 1) + (sx * r * n if case["train"] else 0) + (4 * n if case["bias"] else 0)
    if op == "lin8":
        return {"bytes": r * k + n * k + 4 * (r + n) + outs, "flops": 2 * r * k * n}
    return {"bytes": sx * (r * k + n * k) + outs, "flops": 2 * r * k * n}


# ------------------------------------------------------------------ inputs

def _rows8(t):
    """t as e4m3 values with one scale a row."""
    scale = t.abs().amax(dim=1).clamp_min(E4M3_MIN_AMAX) / E4M3_MAX
    return (t / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    r, op = case["rows"], case["op"]
    xt = TYPES[case["x"]]
    s = {"case": dict(case)}
    if op.startswith("ln"):
        d, rt = case["d"], TYPES[case["res"]]
        s["gamma"] = 1.0 + normal(d, std=0.1)
        # rows of a residual stream: each with a mean of its own
        stream = (normal(r, d, std=2.0) + normal(r, 1)).to(rt)
        if op == "ln_grad":
            s["sum"] = stream
            # the statistics as the forward leaves them
            mean = torch.empty(r, dtype=torch.float64, device="cuda")
            rstd = torch.empty(r, dtype=torch.float64, device="cuda")
            for i in range(0, r, 8192):
                var, mean[i:i + 8192] = torch.var_mean(stream[i:i + 8192].double(), dim=1, correction=0)
                rstd[i:i + 8192] = 1.0 / torch.sqrt(var + EPS)
            s["stats"] = torch.stack([mean, rstd], dim=1).float()
            s["dy"] = normal(r, d, std=0.02).to(xt)
            s["dres"] = normal(r, d, std=0.02).to(rt)
        else:
            s["beta"] = normal(d, std=0.1)
            s["x"], s["res"] = normal(r, d).to(xt), stream
        return s
    k, n = case["k"], case["n"]
    x, w = normal(r, k), normal(n, k, std=k ** -0.5)
    if op == "lin8":
        s["x"], s["x_scale"] = _rows8(x)
        s["w"], s["w_scale"] = _rows8(w)
    else:
        s["x"], s["w"] = x.to(xt), w.to(xt)
    if op == "lin_grad":
        s["dy"] = normal(r, n, std=0.02).to(TYPES[case["dy"]])
        s["z"] = None  # as the forward keeps it
        if case["act"] != "none":
            s["z"] = (s["x"] @ s["w"].t() + normal(n, std=0.1)).to(xt)
        return s
    s["bias"] = normal(n, std=0.1) if case["bias"] else None
    s["res"] = normal(r, n, std=2.0).to(TYPES[case["out"]]) if case["res"] else None
    return s


class _Handle:
    """A handle of the library, given back with its state."""

    def __init__(self, value, destroy):
        self.value, self.destroy = value, destroy

    def __del__(self):
        self.destroy(self.value)


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:  # what a program that uses the operators keeps: the handle and its output buffers
        import attention_qkv_gemm_gb300 as tfl
        code = {"f32": tfl.TFL_F32, "f16": tfl.TFL_F16, "bf16": tfl.TFL_BF16}
        r, op = case["rows"], case["op"]
        xt = TYPES[case["x"]]
        new = lambda shape, t: torch.empty(shape, dtype=t, device="cuda")  # noqa: E731
        s["tfl"], s["stream"] = tfl, torch.cuda.current_stream().cuda_stream
        if op.startswith("ln"):
            d, rt = case["d"], TYPES[case["res"]]
            y = tfl.TFL_E4M3 if op == "ln8" else code[case["x"]]
            s["handle"] = _Handle(tfl.tfl_layernorm_create(d, code[case["x"]], code[case["res"]], y, EPS),
                                  tfl.tfl_layernorm_destroy)
            if op == "ln_grad":
                s["dx"] = new((r, d), xt)
                s["dsum"] = new((r, d), rt) if rt != xt else None
                s["dgamma"], s["dbeta"] = new((d,), torch.float32), new((d,), torch.float32)
            else:
                s["sum"] = new((r, d), rt)
                s["y"] = new((r, d), torch.float8_e4m3fn if op == "ln8" else xt)
                s["y_scale"] = new((r,), torch.float32) if op == "ln8" else None
                s["stats"] = new((r, 2), torch.float32) if case["train"] else None
        else:
            k, n = case["k"], case["n"]
            act = {"none": tfl.TFL_ACT_NONE, "silu": tfl.TFL_ACT_SILU, "gelu": tfl.TFL_ACT_GELU}[case["act"]]
            kind = tfl.TFL_E4M3 if op == "lin8" else code[case["x"]]
            grad = op == "lin_grad"
            out = case["x"] if grad else case["out"]
            s["handle"] = _Handle(tfl.tfl_linear_create(k, n, kind, code[out], act, code[case["dy"] if grad else out],
                                                        r if grad else 0), tfl.tfl_linear_destroy)
            if grad:
                s["dx"], s["dw"], s["db"] = new((r, k), xt), new((n, k), xt), new((n,), torch.float32)
            else:
                s["y"] = new((r, n), TYPES[out])
                s["z"] = new((r, n), xt) if case["train"] else None
    return s


# ------------------------------------------------------------------ one pass

def _p(t):
    return None if t is None else t.data_ptr()


def _run_own(s):
    c, tfl = s["case"], s["tfl"]
    h, r, op = s["handle"].value, c["rows"], c["op"]
    if op in ("ln", "ln8"):
        tfl.tfl_layernorm_forward(h, r, _p(s["x"]), _p(s["res"]), _p(s["gamma"]), _p(s["beta"]), _p(s["sum"]),
                                  _p(s["y"]), _p(s["y_scale"]), _p(s["stats"]), s["stream"])
        return [t for t in (s["sum"], s["y"], s["y_scale"], s["stats"]) if t is not None]
    if op == "ln_grad":
        tfl.tfl_layernorm_backward(h, r, _p(s["sum"]), _p(s["stats"]), _p(s["gamma"]), _p(s["dy"]), _p(s["dres"]),
                                   _p(s["dx"]), _p(s["dsum"]), _p(s["dgamma"]), _p(s["dbeta"]), s["stream"])
        return [s["dx"], s["dgamma"], s["dbeta"]] + ([s["dsum"]] if s["dsum"] is not None else [])
    if op == "lin_grad":
        tfl.tfl_linear_backward(h, r, _p(s["x"]), _p(s["w"]), _p(s["z"]), _p(s["dy"]), _p(s["dx"]), _p(s["dw"]),
                                _p(s["db"]), s["stream"])
        return [s["dx"], s["dw"], s["db"]]
    tfl.tfl_linear_forward(h, r, _p(s["x"]), _p(s.get("x_scale")), _p(s["w"]), _p(s.get("w_scale")), _p(s["bias"]),
                           _p(s["res"]), _p(s["z"]), _p(s["y"]), s["stream"])
    return [s["y"]] + ([s["z"]] if s["z"] is not None else [])


def _act(z, kind):
    """The activation and its derivative."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return z * p, p * (1.0 + z * (1.0 - p))
    cdf = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return z * cdf, cdf + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))


def _run_plain(s):
    c = s["case"]
    op, xt = c["op"], TYPES[c["x"]]
    if op in ("ln", "ln8"):
        t = s["x"].float() + s["res"].float()
        mean = t.mean(dim=1, keepdim=True)
        centred = t - mean
        rstd = torch.rsqrt(centred.square().mean(dim=1, keepdim=True) + EPS)
        y = centred * rstd * s["gamma"] + s["beta"]
        out = t.to(s["res"].dtype)
        stats = [torch.cat([mean, rstd], dim=1)] if c["train"] else []
        if op == "ln":
            return [out, y.to(xt)] + stats
        q, scale = _rows8(y)
        return [out, q, scale] + stats
    if op == "ln_grad":
        t, dy = s["sum"].float(), s["dy"].float()
        mean, rstd = s["stats"][:, :1], s["stats"][:, 1:]
        hat = (t - mean) * rstd
        a = dy * s["gamma"]
        ds = s["dres"].float() + rstd * (a - a.mean(dim=1, keepdim=True) - hat * (a * hat).mean(dim=1, keepdim=True))
        other = [ds.to(s["sum"].dtype)] if s["sum"].dtype != xt else []
        return [ds.to(xt), (dy * hat).sum(dim=0), dy.sum(dim=0)] + other
    x, w = s["x"].float(), s["w"].float()
    if op == "lin_grad":
        dz = s["dy"].float()
        if c["act"] != "none":
            dz = dz * _act(s["z"].float(), c["act"])[1]
        return [(dz @ w).to(xt), (dz.t() @ x).to(xt), dz.sum(dim=0)]
    z = x @ w.t()
    if op == "lin8":
        z = z * s["x_scale"][:, None] * s["w_scale"]
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(z, c["act"])[0]
    if s["res"] is not None:
        y = y + s["res"].float()
    return [y.to(TYPES[c["out"]])] + ([z.to(xt)] if c["train"] else [])


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """From the definitions in float64; gradients by differentiating the definition's own forward."""
    s = _inputs(case, seed)
    w = {k: v.to(torch.float64) for k, v in s.items() if isinstance(v, torch.Tensor)}
    op = case["op"]
    functional = torch.nn.functional
    if op in ("ln", "ln8"):
        total = torch.add(w["x"], w["res"])
        var, mean = torch.var_mean(total, dim=-1, correction=0)
        y = functional.layer_norm(total, total.shape[-1:], w["gamma"], w["beta"], EPS)
        stats = [torch.stack([mean, (var + EPS) ** -0.5], dim=-1)] if case["train"] else []
        if op == "ln":
            return [total, y] + stats
        scale = torch.clamp(torch.max(torch.abs(y), -1).values, min=E4M3_MIN_AMAX) / E4M3_MAX
        return [total, y / scale.unsqueeze(-1), scale] + stats
    if op == "ln_grad":
        total, gamma = w["sum"].requires_grad_(), w["gamma"].requires_grad_()
        beta = torch.zeros_like(gamma).requires_grad_()
        y = functional.layer_norm(total, total.shape[-1:], gamma, beta, EPS)
        ds, dgamma, dbeta = torch.autograd.grad(y, (total, gamma, beta), w["dy"])
        ds = ds + w["dres"]
        return [ds, dgamma, dbeta] + ([ds] if case["x"] != case["res"] else [])
    act = {"none": lambda t: t, "silu": functional.silu, "gelu": functional.gelu}[case["act"]]
    if op == "lin_grad":
        dz = w["dy"]
        if case["act"] != "none":
            z = w["z"].requires_grad_()
            dz = torch.autograd.grad(act(z), z, dz)[0]
        x, weight = w["x"].requires_grad_(), w["w"].requires_grad_()
        bias = torch.zeros(case["n"], dtype=torch.float64, device="cuda").requires_grad_()
        return list(torch.autograd.grad(functional.linear(x, weight, bias), (x, weight, bias), dz))
    if op == "lin8":
        for name in ("x", "w"):
            w[name] = w[name] * w[name + "_scale"].unsqueeze(-1)
    z = functional.linear(w["x"], w["w"], w.get("bias"))
    y = act(z)
    if "res" in w:
        y = y + w["res"]
    return [y] + ([z] if case["train"] else [])
