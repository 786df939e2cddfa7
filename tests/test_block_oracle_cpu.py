"""The fp64 formulas of oracle/block.py: gradients against differences."""
import numpy as np
import pytest

from oracle import block


def diff(f, x, d=1e-6):
    """Gradient of the scalar f at x by central differences."""
    g = np.empty_like(x)
    for k in np.ndindex(x.shape):
        p, q = x.copy(), x.copy()
        p[k] += d
        q[k] -= d
        g[k] = (f(p) - f(q)) / (2 * d)
    return g


@pytest.mark.parametrize("gate,reset", [(False, False), (True, False), (True, True)])
def test_recurrence_gradients(gate, reset):
    rng = np.random.default_rng(0)
    B, L, D = 2, 5, 3
    ins = dict(x=rng.normal(size=(B, L, D)), rgate=rng.normal(size=(B, L, D)), igate=rng.normal(size=(B, L, D)),
               lam=rng.normal(size=D) - 2, h0=rng.normal(size=(B, D)))
    if gate:
        ins["gate"] = rng.normal(size=(B, L, D))
    opts = dict(reset=rng.random((B, L)) < 0.4) if reset else {}
    dy, dh = rng.normal(size=(B, L, D)), rng.normal(size=(B, D))

    def loss(**k):
        y, h = block.gated_recurrence(**dict(ins, **k), **opts)
        return (y * dy).sum() + (h * dh).sum()
    got = block.gated_recurrence(**ins, **opts, dy=dy, dh_last=dh)[2]
    for n, v in ins.items():
        assert np.allclose(got["d" + n], diff(lambda t: loss(**{n: t}), v), rtol=1e-6, atol=1e-8), n


def test_recurrence_with_open_gate():
    """rgate of minus infinity: the state stays, and no gradient is NaN."""
    one = np.ones((1, 3, 1))
    rg = one.copy()
    rg[0, 1] = -np.inf
    with np.errstate(over="ignore"):
        y, h, g = block.gated_recurrence(one, rg, one, np.zeros(1), dy=one)
    assert y[0, 1] == y[0, 0] and all(np.isfinite(v).all() for v in g.values())


@pytest.mark.parametrize("act", [None, "silu", "gelu", "sigmoid"])
def test_projection_gradients(act):
    rng = np.random.default_rng(1)
    x, w, b = rng.normal(size=(4, 2, 3)), rng.normal(size=(2, 5, 3)), rng.normal(size=(2, 5))
    dy = rng.normal(size=(4, 2, 5))
    loss = lambda x=x, w=w, b=b: (block.projection(x, w, b, act)[0] * dy).sum()
    dpre = dy * block.activation_grad(block.projection(x, w, b)[1], act)
    dx, dw = block.projection_grads(dpre, x, w)
    assert np.allclose(dx, diff(lambda t: loss(x=t), x), atol=1e-7)
    assert np.allclose(dw, diff(lambda t: loss(w=t), w), atol=1e-7)
    assert np.allclose(dpre.sum(0), diff(lambda t: loss(b=t), b), atol=1e-7)


def test_clip():
    norm, out = block.clip([np.array([3.0]), np.array([4.0, 0.0])], 1.0, eps=0.0)
    assert norm == 5 and np.allclose(out[1], [0.8, 0])
    assert np.array_equal(block.clip([np.array([0.3])], 1.0)[1][0], [0.3])
