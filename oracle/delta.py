"""fp64 references of the gated delta rule and of the block norms, token by
token and row by row from their definitions (include/ssm_scan.h), sharing
nothing with the library's chunked evaluation.

Arrays are numpy; every input is widened to fp64 first. Shapes as the
library's: q, k (B, L, G, N), v (B, L, H, P), dt, beta (B, L, H), states
(B, H, P, N).
"""
from __future__ import annotations

import numpy as np


def _sigmoid(x):
    return np.where(x >= 0, 1.0 / (1.0 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1.0 + np.exp(-np.abs(x))))


def _terms(q, k, dt, beta, A, H, scale, dt_bias, dt_softplus, beta_sigmoid, qk_norm, qk_eps):
    """Per head: unit and scaled q, unit k, decay, strength, and the inner derivatives."""
    G, N = q.shape[2:]
    raw = dt + (0.0 if dt_bias is None else dt_bias)
    step = np.logaddexp(raw, 0.0) if dt_softplus else raw
    w = _sigmoid(beta) if beta_sigmoid else beta
    nq = np.sqrt((q * q).sum(-1, keepdims=True) + qk_eps) if qk_norm else np.ones(q.shape[:3] + (1,))
    nk = np.sqrt((k * k).sum(-1, keepdims=True) + qk_eps) if qk_norm else np.ones(k.shape[:3] + (1,))
    head = np.arange(H) // (H // G)
    sc = N ** -0.5 if scale is None else scale
    return dict(q=(q / nq)[:, :, head] * sc, k=(k / nk)[:, :, head], a=np.exp(step * A), w=w, step=step, sc=sc, nq=nq, nk=nk,
                dstep=_sigmoid(raw) if dt_softplus else np.ones_like(raw),
                dw=w * (1.0 - w) if beta_sigmoid else np.ones_like(w))


def delta_rule(q, k, v, dt, beta, A, h0=None, dy=None, dh_last=None, scale=None, dt_bias=None, dt_softplus=False,
               beta_sigmoid=False, qk_norm=False, qk_eps=1e-6):
    """(y, h_last), and with ``dy`` a third result: the dict of gradients (and
    ``dA_abs``, ``ddt_bias_abs``: the sums of their terms' magnitudes)."""
    q, k, v, dt, beta, A = (np.asarray(t, np.float64) for t in (q, k, v, dt, beta, A))
    B, L, H, P = v.shape
    G, N = q.shape[2:]
    t = _terms(q, k, dt, beta, A, H, scale, None if dt_bias is None else np.asarray(dt_bias, np.float64), dt_softplus,
               beta_sigmoid, qk_norm, qk_eps)
    S = np.zeros((B, H, P, N)) if h0 is None else np.asarray(h0, np.float64).copy()
    y = np.zeros((B, L, H, P))
    states = [S]
    for i in range(L):
        kt, qt = t["k"][:, i], t["q"][:, i]
        S = t["a"][:, i, :, None, None] * S
        u = t["w"][:, i, :, None] * (v[:, i] - np.matmul(S, kt[..., None])[..., 0])
        S = S + u[..., None] * kt[:, :, None, :]
        y[:, i] = np.matmul(S, qt[..., None])[..., 0]
        states.append(S)
    if dy is None:
        return y, S
    dy = np.asarray(dy, np.float64)
    D = np.zeros_like(S) if dh_last is None else np.asarray(dh_last, np.float64).copy()
    dq, dk, dv = np.zeros(t["q"].shape), np.zeros(t["k"].shape), np.zeros_like(v)
    dlog, db = np.zeros((B, L, H)), np.zeros((B, L, H))
    for i in range(L - 1, -1, -1):
        kt, qt, a, w = t["k"][:, i], t["q"][:, i], t["a"][:, i, :, None, None], t["w"][:, i, :, None]
        dq[:, i] = np.matmul(np.swapaxes(states[i + 1], -1, -2), dy[:, i, :, :, None])[..., 0]
        D = D + dy[:, i, :, :, None] * qt[:, :, None, :]
        old = a * states[i]
        miss = v[:, i] - np.matmul(old, kt[..., None])[..., 0]
        Dk = np.matmul(D, kt[..., None])[..., 0]
        db[:, i] = (Dk * miss).sum(-1)
        dv[:, i] = w * Dk
        dk[:, i] = (np.matmul(np.swapaxes(D, -1, -2), (w * miss)[..., None])
                    - np.matmul(np.swapaxes(old, -1, -2), (w * Dk)[..., None]))[..., 0]
        D = D - (w * Dk)[..., None] * kt[:, :, None, :]
        dlog[:, i] = (D * old).sum((-1, -2))
        D = a * D
    dq = dq.reshape(B, L, G, H // G, N).sum(3) * t["sc"]
    dk = dk.reshape(B, L, G, H // G, N).sum(3)
    if qk_norm:
        dq = dq / t["nq"] - q * (q * dq).sum(-1, keepdims=True) / t["nq"] ** 3
        dk = dk / t["nk"] - k * (k * dk).sum(-1, keepdims=True) / t["nk"] ** 3
    ddt = dlog * A * t["dstep"]
    return y, S, dict(dq=dq, dk=dk, dv=dv, ddt=ddt, dbeta=db * t["dw"], dA=(dlog * t["step"]).sum((0, 1)),
                      ddt_bias=ddt.sum((0, 1)), dh0=D, dA_abs=np.abs(dlog * t["step"]).sum((0, 1)),
                      ddt_bias_abs=np.abs(ddt).sum((0, 1)))


def prenorm(x, weight, residual=None, scale=None, eps=1e-5, dy=None, dr=None, store=None):
    """(y, r) of r = residual + scale x, y = r / rms(r) weight, and with ``dy``
    the gradients. ``store`` rounds r to its stored type (default: no rounding)."""
    x, weight = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    s = 1.0 if scale is None else np.asarray(scale, np.float64)
    r = s * x if residual is None else np.asarray(residual, np.float64) + s * x
    if store is not None:
        r = store(r)
    inv = 1.0 / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    n = r * inv
    if dy is None:
        return n * weight, r
    dy = np.asarray(dy, np.float64)
    wy = dy * weight
    d = inv * (wy - n * (n * wy).mean(-1, keepdims=True)) + (0.0 if dr is None else np.asarray(dr, np.float64))
    axes = tuple(range(x.ndim - 1))
    return n * weight, r, dict(dx=d * s, dresidual=d, dweight=(dy * n).sum(axes), dscale=(d * x).sum(axes),
                               dweight_abs=np.abs(dy * n).sum(axes), dscale_abs=np.abs(d * x).sum(axes))


def gated_norm(x, z, weight, eps=1e-5, gate_first=False, dy=None):
    """y of the norm over the last axis, gated by silu(z) before or behind it,
    and with ``dy`` (y, gradients). weight: (groups, dim) or (dim,)."""
    x, weight = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    gate = dgate = None
    if z is not None:
        z = np.asarray(z, np.float64)
        sg = _sigmoid(z)
        gate, dgate = z * sg, sg * (1.0 + z * (1.0 - sg))
    f = x * gate if gate is not None and gate_first else x
    inv = 1.0 / np.sqrt((f * f).mean(-1, keepdims=True) + eps)
    n = f * inv
    behind = gate if gate is not None and not gate_first else 1.0
    y = n * weight * behind
    if dy is None:
        return y
    up = np.asarray(dy, np.float64) * behind
    wy = up * weight
    df = inv * (wy - n * (n * wy).mean(-1, keepdims=True))
    axes = tuple(range(x.ndim - weight.ndim))
    # the size of the two terms whose difference df is
    size = inv * (np.abs(wy) + np.abs(n * (n * wy).mean(-1, keepdims=True)))
    g = dict(dx=df * gate if gate is not None and gate_first else df, dweight=(up * n).sum(axes),
             dweight_abs=np.abs(up * n).sum(axes), dx_terms=size * np.abs(gate) if gate is not None and gate_first else size)
    if gate is not None:
        g["dz_terms"] = np.abs(size * x * dgate) if gate_first else np.abs(np.asarray(dy, np.float64) * n * weight * dgate)
        g["dz"] = (df * x if gate_first else np.asarray(dy, np.float64) * n * weight) * dgate
    return y, g
