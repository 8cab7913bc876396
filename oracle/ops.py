"""float64 definitions of the operators that stand on their own beside the stack.

The root-mean-square norm and layer norm with the residual's addition, the gated feed-forward
and the linear layer, forward and gradients, as plain numpy.
"""
from __future__ import annotations

import numpy as np
from scipy.special import erf as _erf

E4M3_MAX = 448.0
E4M3_MIN_AMAX = 2.0 ** -100


def rms_norm(x: np.ndarray, res, gamma: np.ndarray, eps: float):
    """(s, y): s = x + res (res may be None), y = s / sqrt(mean(s^2) + eps) * gamma, row by row."""
    s = x if res is None else x + res
    return s, s / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps) * gamma


def row_scale(y: np.ndarray) -> np.ndarray:
    """The scale of each row's e4m3 values."""
    return np.maximum(np.abs(y).max(axis=1), E4M3_MIN_AMAX) / E4M3_MAX


def rms_norm_backward(s: np.ndarray, gamma: np.ndarray, dy: np.ndarray, dres, eps: float):
    """(ds, dgamma) of y = rms_norm(s) and of what else reaches s (dres, or None)."""
    r = 1.0 / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps)
    a = dy * gamma
    ds = r * a - s * r ** 3 * np.mean(a * s, axis=1, keepdims=True)
    return (ds if dres is None else ds + dres), np.sum(dy * s * r, axis=0)


def layer_norm(x: np.ndarray, res, gamma: np.ndarray, beta, eps: float):
    """(s, y, m, r): s = x + res (res may be None), row by row its mean m and r = 1 / sqrt(var + eps),
    y = (s - m) r gamma + beta (beta may be None)."""
    s = x if res is None else x + res
    m = np.mean(s, axis=1)
    r = 1.0 / np.sqrt(np.mean((s - m[:, None]) ** 2, axis=1) + eps)
    y = (s - m[:, None]) * r[:, None] * gamma
    return s, (y if beta is None else y + beta), m, r


def layer_norm_backward(s: np.ndarray, m: np.ndarray, r: np.ndarray, gamma: np.ndarray, dy: np.ndarray, dres):
    """(ds, dgamma, dbeta) of y = layer_norm(s) and of what else reaches s (dres, or None)."""
    t, a = (s - m[:, None]) * r[:, None], dy * gamma
    ds = r[:, None] * (a - np.mean(a, axis=1, keepdims=True) - t * np.mean(a * t, axis=1, keepdims=True))
    return (ds if dres is None else ds + dres), np.sum(dy * t, axis=0), np.sum(dy, axis=0)


def activation(g: np.ndarray, kind: str):
    """An activation and its derivative: "silu", the exact "gelu" or "none"."""
    if kind == "none":
        return g, np.ones_like(g)
    if kind == "silu":
        p = 1.0 / (1.0 + np.exp(-g))
        return g * p, p + g * p * (1.0 - p)
    cdf = 0.5 * (1.0 + _erf(g / np.sqrt(2.0)))
    return g * cdf, cdf + g * np.exp(-0.5 * g * g) / np.sqrt(2.0 * np.pi)


def glu(x: np.ndarray, wg: np.ndarray, wu: np.ndarray, kind: str) -> np.ndarray:
    """act(x Wg^T) * (x Wu^T); Wg, Wu: [d_ff, d_model]."""
    return activation(x @ wg.T, kind)[0] * (x @ wu.T)


def glu_backward(x: np.ndarray, wg: np.ndarray, wu: np.ndarray, dh: np.ndarray, kind: str,
                 return_intermediates: bool = False):
    """(dx, dWg, dWu) of glu for the output gradient dh."""
    g, u = x @ wg.T, x @ wu.T
    a, slope = activation(g, kind)
    dg, du = dh * u * slope, dh * a
    out = (dg @ wg + du @ wu, dg.T @ x, du.T @ x)
    return (*out, g, u, dg, du) if return_intermediates else out


def linear(x: np.ndarray, w: np.ndarray, bias, res, kind: str):
    """(y, z): z = x W^T + bias, y = act(z) + res (bias and res may be None); W: [d_out, d_in]."""
    z = x @ w.T
    z = z if bias is None else z + bias
    y = activation(z, kind)[0]
    return (y if res is None else y + res), z


def linear_backward(x: np.ndarray, w: np.ndarray, z, dy: np.ndarray, kind: str):
    """(dx, dW, dbias, dz) for the output gradient dy at the pre-activation z (unused for "none")."""
    dz = dy if kind == "none" else dy * activation(z, kind)[1]
    return dz @ w, dz.T @ x, dz.sum(axis=0), dz
