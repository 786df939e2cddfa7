"""The gated linear recurrence, the projection with its epilogue and the clipping
of gradients in fp64 numpy, straight from their formulas."""
from __future__ import annotations

import numpy as np


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1 + e)


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def recurrence_parts(x, rgate, igate, lam, reset=None, rate=8.0):
    """(a, m, r, i, s): decay, input scale, both gates and the decay's exponent."""
    r, i = sigmoid(rgate), sigmoid(igate)
    s = rate * softplus(lam) * r
    a, m = np.exp(-s), np.sqrt(-np.expm1(-2 * s))
    if reset is not None:
        first = reset[..., None]
        a, m = np.where(first, 0.0, a), np.where(first, 1.0, m)
    return a, m, r, i, s


def gated_recurrence(x, rgate, igate, lam, h0=None, gate=None, reset=None, rate=8.0, dy=None, dh_last=None):
    """(y, h_last), or (y, h_last, gradients) with dy; also the states and what the
    recurrence back in time holds, in gradients["h"] and gradients["g"]."""
    B, L, D = x.shape
    a, m, r, i, s = recurrence_parts(x, rgate, igate, lam, reset, rate)
    first = None if reset is None else reset[..., None]
    h = np.zeros((B, D)) if h0 is None else h0.copy()
    states = np.empty((B, L + 1, D))
    states[:, 0] = h
    for t in range(L):
        kept = a[:, t] * h
        if first is not None:
            kept = np.where(first[:, t], 0.0, kept)
        h = kept + m[:, t] * i[:, t] * x[:, t]
        states[:, t + 1] = h
    H = states[:, 1:]
    y = H if gate is None else H * gate
    if dy is None:
        return y, h
    up = dy if gate is None else dy * gate
    c = np.zeros((B, D)) if dh_last is None else dh_last.copy()
    g = np.empty((B, L, D))
    for t in range(L - 1, -1, -1):
        g[:, t] = up[:, t] + c
        c = a[:, t] * g[:, t]
        if first is not None:
            c = np.where(first[:, t], 0.0, c)
    before = states[:, :-1]
    ix = i * x
    with np.errstate(divide="ignore", invalid="ignore"):
        ratio = np.where(m > 0, s / m, 0.0)
    # d a / d s = -a, d m / d s = a^2 / m, times s
    w = a * (a * ix * ratio - s * before)
    if first is not None:
        w = np.where(first, 0.0, w)
    lead = tuple(range(2))
    out = dict(dx=g * m * i, drgate=g * w * (1 - r), digate=g * m * ix * (1 - i),
               dlam=(g * w).sum(lead) * sigmoid(lam) / softplus(lam), dh0=c, h=states, g=g, w=w)
    if gate is not None:
        out["dgate"] = dy * H
    return y, h, out


GELU_K = 2 * np.sqrt(2 / np.pi)


def activation(z, name):
    if name == "silu":
        return z * sigmoid(z)
    if name == "gelu":
        return z * sigmoid(GELU_K * (z + 0.044715 * z ** 3))
    return sigmoid(z) if name == "sigmoid" else z


def activation_grad(z, name):
    if name == "silu":
        s = sigmoid(z)
        return s * (1 + z * (1 - s))
    if name == "gelu":
        s = sigmoid(GELU_K * (z + 0.044715 * z ** 3))
        return s + z * s * (1 - s) * GELU_K * (1 + 3 * 0.044715 * z * z)
    if name == "sigmoid":
        s = sigmoid(z)
        return s * (1 - s)
    return np.ones_like(z)


def projection(x, weight, bias=None, act=None, residual=None):
    """(y, pre): x (rows, G, K), weight (G, N, K), bias (G, N), residual (rows, G, N)."""
    pre = np.einsum("mgk,gnk->mgn", x, weight)
    if bias is not None:
        pre = pre + bias
    y = activation(pre, act)
    return (y if residual is None else y + residual), pre


def projection_grads(dpre, x, weight):
    """(dx, dweight) of the stored dpre (rows, G, N)."""
    return np.einsum("mgn,gnk->mgk", dpre, weight), np.einsum("mgn,mgk->gnk", dpre, x)


def clip(grads, max_norm, eps=1e-6):
    """(norm, clipped)."""
    norm = np.sqrt(sum((g.astype(np.float64) ** 2).sum() for g in grads))
    return norm, [g * min(1.0, max_norm / (norm + eps)) for g in grads]
