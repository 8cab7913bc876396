"""Pins of oracle/ops.py's layer norm and linear layer (CPU): torch float64 autograd, central
differences, planted mistakes."""
import numpy as np
import pytest
import torch

from oracle import ops

EPS = 1e-5


def _norm_inputs(seed, rows=5, d=24):
    rng = np.random.default_rng(seed)
    x, res, dy, dres = (rng.standard_normal((rows, d)) for _ in range(4))
    return x, res + 3.0, 1 + 0.3 * rng.standard_normal(d), 0.2 * rng.standard_normal(d), dy, dres


def test_layer_norm_and_gradients_match_autograd():
    x, res, gamma, beta, dy, dres = _norm_inputs(0)
    s, y, m, r = ops.layer_norm(x, res, gamma, beta, EPS)
    np.testing.assert_array_equal(s, x + res)
    leaves = [torch.tensor(t, requires_grad=True) for t in (s, gamma, beta)]
    ty = torch.nn.functional.layer_norm(leaves[0], (s.shape[1],), leaves[1], leaves[2], EPS)
    np.testing.assert_allclose(y, ty.detach().numpy(), rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(ops.layer_norm(x, res, gamma, None, EPS)[1], y - beta, rtol=1e-10, atol=1e-11)
    ref = torch.autograd.grad(ty, leaves, torch.tensor(dy))
    got = ops.layer_norm_backward(s, m, r, gamma, dy, dres)
    np.testing.assert_allclose(got[0], ref[0].numpy() + dres, rtol=1e-10, atol=1e-11)
    for g, w in zip(got[1:], ref[1:]):
        np.testing.assert_allclose(g, w.numpy(), rtol=1e-10, atol=1e-11)


def test_layer_norm_gradient_is_the_difference_quotient():
    x, res, gamma, beta, dy, _ = _norm_inputs(1)
    s, _, m, r = ops.layer_norm(x, res, gamma, beta, EPS)
    ds = ops.layer_norm_backward(s, m, r, gamma, dy, None)[0]
    v = np.random.default_rng(2).standard_normal(s.shape)
    h = 1e-5
    loss = lambda t: np.sum(dy * ops.layer_norm(t, None, gamma, beta, EPS)[1])  # noqa: E731
    q = (loss(s + h * v) - loss(s - h * v)) / (2 * h)
    assert abs(q - np.sum(ds * v)) < 1e-8
    wrong = ds + 1e-3 * r[:, None] * np.mean(dy * gamma, axis=1, keepdims=True)  # a wrong mean term is seen
    assert abs(q - np.sum(wrong * v)) > 1e-6


@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
def test_linear_and_gradients_match_autograd_and_differences(kind):
    rng = np.random.default_rng(3)
    x, w, b, res, dy = (rng.standard_normal(sh) for sh in ((7, 12), (9, 12), 9, (7, 9), (7, 9)))
    leaves = [torch.tensor(t, requires_grad=True) for t in (x, w, b)]
    act = {"none": lambda t: t, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[kind]
    ty = act(torch.nn.functional.linear(*leaves)) + torch.tensor(res)
    y, z = ops.linear(x, w, b, res, kind)
    np.testing.assert_allclose(y, ty.detach().numpy(), rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(ops.linear(x, w, None, None, kind)[1], z - b, rtol=1e-11, atol=1e-12)
    got = ops.linear_backward(x, w, z, dy, kind)
    for g, r in zip(got, torch.autograd.grad(ty, leaves, torch.tensor(dy))):
        np.testing.assert_allclose(g, r.numpy(), rtol=1e-10, atol=1e-11)
    h = 1e-5
    for k, t in enumerate((x, w, b)):
        v = rng.standard_normal(t.shape)
        args = [x, w, b]
        args[k] = t + h * v
        up = np.sum(dy * ops.linear(*args, res, kind)[0])
        args[k] = t - h * v
        q = (up - np.sum(dy * ops.linear(*args, res, kind)[0])) / (2 * h)
        assert abs(q - np.sum(got[k] * v)) < 1e-6 * (1 + abs(q))


def test_the_pins_tell_the_activation_before_the_residual_from_the_one_behind_it():
    rng = np.random.default_rng(4)
    x, w, res = (rng.standard_normal(sh) for sh in ((3, 8), (4, 8), (3, 4)))
    y, z = ops.linear(x, w, None, res, "gelu")
    assert np.abs(y - ops.activation(z + res, "gelu")[0]).max() > 1e-2
