"""The root-mean-square norm and the gated feed-forward on their own: cases, plain forms and work.

``norm``       s = x + res; y = s / rms(s) * gamma; returns s (in the residual's type) and y
``norm8``      the same with y as e4m3 values and one float32 scale a row
``norm_grad``  the norm's gradients: of s (in x's type, and in the residual's where that differs)
               and of gamma, from s, dy and the gradient that reaches s from later layers
``glu``        h = act(x Wg^T) * (x Wu^T), Wg and Wu as nn.Linear weights [f, d]
``glu8``       the same from e4m3 x and weights with one float32 scale a row of each
``glu_grad``   dx, dWg, dWu from x, Wg, Wu and dh

``rows`` is the number of tokens.  Types: f32, f16, bf16.
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
        # one token of a generation step: the norm in front of an 8-bit feed-forward
        {"name": "norm8 one token", "op": "norm8", "rows": 1, "d": 1024, "x": "bf16", "res": "f32"},
        # a batch of 16 prompts of 512 tokens, residual stream in fp32 as the stack keeps it
        {"name": "norm batch", "op": "norm", "rows": 8192, "d": 1024, "x": "f16", "res": "f32"},
        # one sequence of 100000 tokens, everything in bf16, rows for an 8-bit feed-forward
        {"name": "norm8 long", "op": "norm8", "rows": 100000, "d": 1024, "x": "bf16", "res": "bf16"},
        # a width that no vector load divides
        {"name": "norm odd width", "op": "norm", "rows": 1531, "d": 1001, "x": "f32", "res": "f32"},
        # a training step's norm: 16 sequences of 512 tokens
        {"name": "norm_grad batch", "op": "norm_grad", "rows": 8192, "d": 1024, "x": "bf16", "res": "f32"},
        # a wide model's norm in training, with a ragged number of tokens
        {"name": "norm_grad wide", "op": "norm_grad", "rows": 20011, "d": 4096, "x": "f16", "res": "f16"},
        # one token of a generation step: the weights are read for a single row
        {"name": "glu one token", "op": "glu", "rows": 1, "d": 1024, "f": 4096, "x": "bf16", "act": "silu"},
        # forty requests generating together in 8 bits
        {"name": "glu8 generation", "op": "glu8", "rows": 40, "d": 4096, "f": 10240, "x": "bf16", "act": "silu"},
        # the batch of prompts
        {"name": "glu batch", "op": "glu", "rows": 8192, "d": 1024, "f": 4096, "x": "f16", "act": "gelu"},
        # a long ragged prompt of a wide model in 8 bits
        {"name": "glu8 prompt", "op": "glu8", "rows": 6007, "d": 4096, "f": 12288, "x": "bf16", "act": "silu"},
        # a training step
        {"name": "glu_grad step", "op": "glu_grad", "rows": 16384, "d": 2048, "f": 8192, "x": "bf16", "act": "silu"},
        # a training step of a small model with sizes that no tile divides
        {"name": "glu_grad ragged", "op": "glu_grad", "rows": 2979, "d": 1160, "f": 2856, "x": "f16", "act": "gelu"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "norm8", "norm_grad", "glu", "glu8", "glu_grad"])
    if op.startswith("norm"):
        x, res = rng.choice([("f32", "f32"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
        d = _log(rng, 64, 8192)
        if rng.random() < 0.75:
            d = (d + 7) // 8 * 8
        # one token up to what 160 M values hold
        rows = min(_log(rng, 1, 100000), max(1, 40_000_000 // d))
        return {"op": op, "rows": rows, "d": d, "x": x, "res": res}
    step = 16 if op == "glu8" else 8
    d = (_log(rng, 256, 4096) + step - 1) // step * step
    f = (_log(rng, 512, 12288) + step - 1) // step * step
    rows = _log(rng, 1, 16384)
    most = 1.2e12 if op != "glu_grad" else 3.2e12
    rows = max(1, min(rows, int(most / ((12 if op == "glu_grad" else 4) * d * f))))
    return {"op": op, "rows": rows, "d": d, "f": f, "x": rng.choice(["f16", "bf16"]),
            "act": rng.choice(["silu", "gelu"])}


def work(case):
    r, d = case["rows"], case["d"]
    sx = SIZES[case["x"]]
    if case["op"] in ("norm", "norm8", "norm_grad"):
        sr = SIZES[case["res"]]
        n = r * d
        if case["op"] == "norm":
            return {"bytes": n * (2 * sx + 2 * sr) + 4 * d, "flops": 5 * n}
        if case["op"] == "norm8":
            return {"bytes": n * (sx + 2 * sr + 1) + 4 * d + 4 * r, "flops": 7 * n}
        outs = sx if sx == sr else sx + sr
        return {"bytes": n * (2 * sr + sx + outs) + 8 * d, "flops": 11 * n}
    f = case["f"]
    if case["op"] == "glu":
        return {"bytes": sx * (r * d + 2 * f * d + r * f), "flops": 4 * r * d * f}
    if case["op"] == "glu8":
        return {"bytes": r * d + 2 * f * d + sx * r * f + 4 * (r + 2 * f), "flops": 4 * r * d * f}
    return {"bytes": sx * (2 * r * d + 4 * f * d + r * f), "flops": 12 * r * d * f}


# ------------------------------------------------------------------ inputs

def _rows8(t):
    """t as e4m3 values with one scale a row."""
    scale = t.abs().amax(dim=1).clamp_min(E4M3_MIN_AMAX) / E4M3_MAX
    return (t / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    r, d = case["rows"], case["d"]
    xt = TYPES[case["x"]]
    s = {"case": dict(case)}
    if case["op"].startswith("norm"):
        rt = TYPES[case["res"]]
        s["gamma"] = 1.0 + normal(d, std=0.1)
        if case["op"] == "norm_grad":
            s["sum"] = normal(r, d, std=2.0).to(rt)
            s["dy"] = normal(r, d, std=0.02).to(xt)
            s["dres"] = normal(r, d, std=0.02).to(rt)
        else:
            s["x"] = normal(r, d).to(xt)
            s["res"] = normal(r, d, std=2.0).to(rt)
        return s
    f = case["f"]
    x = normal(r, d)
    wg, wu = normal(f, d, std=d ** -0.5), normal(f, d, std=d ** -0.5)
    if case["op"] == "glu8":
        s["x"], s["x_scale"] = _rows8(x)
        s["wg"], s["wg_scale"] = _rows8(wg)
        s["wu"], s["wu_scale"] = _rows8(wu)
    else:
        s["x"], s["wg"], s["wu"] = x.to(xt), wg.to(xt), wu.to(xt)
    if case["op"] == "glu_grad":
        s["dh"] = normal(r, f, std=0.02).to(xt)
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
        r, d, op = case["rows"], case["d"], case["op"]
        xt = TYPES[case["x"]]
        new = lambda shape, t: torch.empty(shape, dtype=t, device="cuda")  # noqa: E731
        s["tfl"], s["stream"] = tfl, torch.cuda.current_stream().cuda_stream
        if op.startswith("norm"):
            rt = TYPES[case["res"]]
            y = tfl.TFL_E4M3 if op == "norm8" else code[case["x"]]
            s["handle"] = _Handle(tfl.tfl_rmsnorm_create(d, code[case["x"]], code[case["res"]], y, EPS),
                                  tfl.tfl_rmsnorm_destroy)
            if op == "norm_grad":
                s["dx"] = new((r, d), xt)
                s["dsum"] = new((r, d), rt) if rt != xt else None
                s["dgamma"] = new((d,), torch.float32)
            else:
                s["out"] = new((r, d), rt)
                s["y"] = new((r, d), torch.float8_e4m3fn if op == "norm8" else xt)
                s["y_scale"] = new((r,), torch.float32) if op == "norm8" else None
        else:
            f = case["f"]
            act = tfl.TFL_ACT_SILU if case["act"] == "silu" else tfl.TFL_ACT_GELU
            kind = tfl.TFL_E4M3 if op == "glu8" else code[case["x"]]
            s["handle"] = _Handle(tfl.tfl_glu_create(d, f, kind, code[case["x"]], act, r if op == "glu_grad" else 0),
                                  tfl.tfl_glu_destroy)
            if op == "glu_grad":
                s["dx"], s["dwg"], s["dwu"] = new((r, d), xt), new((f, d), xt), new((f, d), xt)
            else:
                s["h"] = new((r, f), xt)
    return s


# ------------------------------------------------------------------ one pass

def _p(t):
    return None if t is None else t.data_ptr()


def _run_own(s):
    c, tfl = s["case"], s["tfl"]
    h, r = s["handle"].value, c["rows"]
    if c["op"] in ("norm", "norm8"):
        tfl.tfl_rmsnorm_forward(h, r, _p(s["x"]), _p(s["res"]), _p(s["gamma"]), _p(s["out"]), _p(s["y"]),
                                _p(s["y_scale"]), s["stream"])
        return [s["out"], s["y"]] + ([s["y_scale"]] if c["op"] == "norm8" else [])
    if c["op"] == "norm_grad":
        tfl.tfl_rmsnorm_backward(h, r, _p(s["sum"]), _p(s["gamma"]), _p(s["dy"]), _p(s["dres"]), _p(s["dx"]),
                                 _p(s["dsum"]), _p(s["dgamma"]), s["stream"])
        return [s["dx"], s["dgamma"]] + ([s["dsum"]] if s["dsum"] is not None else [])
    if c["op"] == "glu_grad":
        tfl.tfl_glu_backward(h, r, _p(s["x"]), _p(s["wg"]), _p(s["wu"]), _p(s["dh"]), _p(s["dx"]), _p(s["dwg"]),
                             _p(s["dwu"]), s["stream"])
        return [s["dx"], s["dwg"], s["dwu"]]
    tfl.tfl_glu_forward(h, r, _p(s["x"]), _p(s.get("x_scale")), _p(s["wg"]), _p(s.get("wg_scale")), _p(s["wu"]),
                        _p(s.get("wu_scale")), _p(s["h"]), s["stream"])
    return [s["h"]]


def _act(g, kind):
    """The activation and its derivative."""
    if kind == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return g * p, p * (1.0 + g * (1.0 - p))
    cdf = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))


def _run_plain(s):
    c = s["case"]
    xt = TYPES[c["x"]]
    if c["op"] in ("norm", "norm8"):
        t = s["x"].float() + s["res"].float()
        y = t * torch.rsqrt(t.square().mean(dim=1, keepdim=True) + EPS) * s["gamma"]
        out = t.to(s["res"].dtype)
        if c["op"] == "norm":
            return [out, y.to(xt)]
        q, scale = _rows8(y)
        return [out, q, scale]
    if c["op"] == "norm_grad":
        t, dy = s["sum"].float(), s["dy"].float()
        rstd = torch.rsqrt(t.square().mean(dim=1, keepdim=True) + EPS)
        a = dy * s["gamma"]
        ds = s["dres"].float() + rstd * a - t * (rstd * rstd * rstd) * (a * t).mean(dim=1, keepdim=True)
        dgamma = (dy * t * rstd).sum(dim=0)
        return [ds.to(xt), dgamma] + ([ds.to(s["sum"].dtype)] if s["sum"].dtype != xt else [])
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    g, u = x @ wg.t(), x @ wu.t()
    if c["op"] == "glu8":
        g = g * s["x_scale"][:, None] * s["wg_scale"]
        u = u * s["x_scale"][:, None] * s["wu_scale"]
    a, slope = _act(g, c["act"])
    if c["op"] != "glu_grad":
        return [(a * u).to(xt)]
    dh = s["dh"].float()
    dg, du = dh * u * slope, dh * a
    return [(dg @ wg + du @ wu).to(xt), (dg.t() @ x).to(xt), (du.t() @ x).to(xt)]


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
    if op in ("norm", "norm8"):
        total = torch.add(w["x"], w["res"])
        y = total / torch.sqrt(torch.mean(total ** 2, -1, keepdim=True) + EPS) * w["gamma"]
        if op == "norm":
            return [total, y]
        scale = torch.clamp(torch.max(torch.abs(y), -1).values, min=E4M3_MIN_AMAX) / E4M3_MAX
        return [total, y / scale.unsqueeze(-1), scale]
    if op == "norm_grad":
        total, gamma = w["sum"].requires_grad_(), w["gamma"].requires_grad_()
        y = total / torch.sqrt(torch.mean(total ** 2, -1, keepdim=True) + EPS) * gamma
        ds, dgamma = torch.autograd.grad(y, (total, gamma), w["dy"])
        ds = ds + w["dres"]
        return [ds, dgamma] + ([ds] if case["x"] != case["res"] else [])
    act = torch.nn.functional.silu if case["act"] == "silu" else torch.nn.functional.gelu
    if op == "glu8":
        for name in ("x", "wg", "wu"):
            w[name] = w[name] * w[name + "_scale"].unsqueeze(-1)
    leaves = [w["x"], w["wg"], w["wu"]]
    if op == "glu_grad":
        leaves = [t.requires_grad_() for t in leaves]
    linear = torch.nn.functional.linear
    h = act(linear(leaves[0], leaves[1])) * linear(leaves[0], leaves[2])
    if op != "glu_grad":
        return [h]
    return list(torch.autograd.grad(h, leaves, w["dh"]))
