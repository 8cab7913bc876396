"""Pins of oracle/ops.py (CPU): torch float64 autograd, central differences, planted mistakes."""
import numpy as np
import pytest
import torch

from oracle import ops


def _norm_inputs(seed, rows=5, d=24):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal((rows, d)), rng.standard_normal((rows, d)), 1 + 0.3 * rng.standard_normal(d),
            rng.standard_normal((rows, d)), rng.standard_normal((rows, d)))


def test_rms_norm_and_gradients_match_autograd():
    x, res, gamma, dy, dres = _norm_inputs(0)
    s, y = ops.rms_norm(x, res, gamma, 1e-5)
    ts, tg = torch.tensor(s, requires_grad=True), torch.tensor(gamma, requires_grad=True)
    ty = torch.nn.functional.rms_norm(ts, (ts.shape[1],), tg, 1e-5)
    np.testing.assert_allclose(y, ty.detach().numpy(), rtol=1e-12)
    ds, dgamma = torch.autograd.grad(ty, (ts, tg), torch.tensor(dy))
    got, ggot = ops.rms_norm_backward(s, gamma, dy, dres, 1e-5)
    np.testing.assert_allclose(got, ds.numpy() + dres, rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(ggot, dgamma.numpy(), rtol=1e-11, atol=1e-12)


def test_rms_norm_gradient_is_the_difference_quotient():
    x, res, gamma, dy, _ = _norm_inputs(1)
    s, _ = ops.rms_norm(x, res, gamma, 1e-5)
    ds, _ = ops.rms_norm_backward(s, gamma, dy, None, 1e-5)
    v = np.random.default_rng(2).standard_normal(s.shape)
    h = 1e-5
    q = (np.sum(dy * ops.rms_norm(s + h * v, None, gamma, 1e-5)[1])
         - np.sum(dy * ops.rms_norm(s - h * v, None, gamma, 1e-5)[1])) / (2 * h)
    assert abs(q - np.sum(ds * v)) < 1e-8
    wrong = ds + s * np.mean(dy * gamma * s, axis=1, keepdims=True) * 1e-3  # a wrong mean term is seen
    assert abs(q - np.sum(wrong * v)) > 1e-6


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_glu_and_gradients_match_autograd_and_differences(kind):
    rng = np.random.default_rng(3)
    x, wg, wu, dh = (rng.standard_normal(sh) for sh in ((7, 12), (9, 12), (9, 12), (7, 9)))
    leaves = [torch.tensor(t, requires_grad=True) for t in (x, wg, wu)]
    act = torch.nn.functional.silu if kind == "silu" else torch.nn.functional.gelu
    th = act(leaves[0] @ leaves[1].T) * (leaves[0] @ leaves[2].T)
    np.testing.assert_allclose(ops.glu(x, wg, wu, kind), th.detach().numpy(), rtol=1e-11, atol=1e-12)
    ref = torch.autograd.grad(th, leaves, torch.tensor(dh))
    got = ops.glu_backward(x, wg, wu, dh, kind)
    for g, r in zip(got, ref):
        np.testing.assert_allclose(g, r.numpy(), rtol=1e-10, atol=1e-11)
    h = 1e-5
    for k, t in enumerate((x, wg, wu)):
        v = rng.standard_normal(t.shape)
        args = [x, wg, wu]
        args[k] = t + h * v
        up = np.sum(dh * ops.glu(*args, kind))
        args[k] = t - h * v
        q = (up - np.sum(dh * ops.glu(*args, kind))) / (2 * h)
        assert abs(q - np.sum(got[k] * v)) < 1e-6 * (1 + abs(q))


def test_the_pins_tell_the_gate_from_the_other_projection():
    rng = np.random.default_rng(4)
    x, wg, wu = (rng.standard_normal(sh) for sh in ((3, 8), (4, 8), (4, 8)))
    assert np.abs(ops.glu(x, wg, wu, "silu") - ops.glu(x, wu, wg, "silu")).max() > 1e-2


def test_row_scale_of_zero_and_small_rows():
    y = np.array([[0.0, 0.0], [1e-35, -2e-35], [3.5, -448.0]])
    s = ops.row_scale(y)
    assert s[0] == s[1] == 2.0 ** -100 / 448 and s[2] == 1.0
