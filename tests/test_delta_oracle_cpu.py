"""The fp64 references of the gated delta rule and the block norms against
differences of their own forward, and the delta rule against closed forms."""
import numpy as np
import pytest

from oracle import delta


def rule_inputs(rng, B=2, L=5, G=1, H=2, P=3, N=4):
    return dict(q=rng.standard_normal((B, L, G, N)), k=rng.standard_normal((B, L, G, N)),
                v=rng.standard_normal((B, L, H, P)), dt=rng.standard_normal((B, L, H)), beta=rng.standard_normal((B, L, H)),
                A=-rng.uniform(0.5, 2.0, H), h0=rng.standard_normal((B, H, P, N)), dt_bias=rng.standard_normal(H))


def slope(f, x, at, h=1e-5):
    keep = x[at]
    x[at] = keep + h
    up = f()
    x[at] = keep - h
    down = f()
    x[at] = keep
    return (up - down) / (2 * h)


@pytest.mark.parametrize("norm", [False, True])
def test_rule_gradients_against_differences(norm):
    rng = np.random.default_rng(1)
    x = rule_inputs(rng)
    opts = dict(dt_softplus=True, beta_sigmoid=True, qk_norm=norm, qk_eps=0.1, scale=0.7)
    dy, dh = rng.standard_normal(x["v"].shape), rng.standard_normal(x["h0"].shape)

    def loss():
        y, h = delta.delta_rule(**x, **opts)
        return (y * dy).sum() + (h * dh).sum()
    g = delta.delta_rule(**x, **opts, dy=dy, dh_last=dh)[2]
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("dt", "ddt"), ("beta", "dbeta"), ("A", "dA"),
                       ("h0", "dh0"), ("dt_bias", "ddt_bias")):
        for _ in range(4):
            at = tuple(rng.integers(0, n) for n in x[name].shape)
            # central differences with h = 1e-5: h^2 truncation and 1e-16 / h rounding, both near 1e-10
            assert abs(slope(loss, x[name], at) - g[grad][at]) <= 1e-7 * (1 + abs(g[grad][at])), (name, at)


def test_rule_closed_forms():
    """Strength 1 and a unit key make the state answer that key with the value
    written last; strength 0 leaves only the decay."""
    rng = np.random.default_rng(2)
    x = rule_inputs(rng, L=1, P=4, N=6)
    x["k"] /= np.linalg.norm(x["k"], axis=-1, keepdims=True)
    x["q"] = x["k"]
    y, _ = delta.delta_rule(**dict(x, beta=np.ones_like(x["beta"])), scale=1.0)
    assert np.allclose(y, x["v"], atol=1e-13)
    _, h = delta.delta_rule(**dict(x, beta=np.zeros_like(x["beta"])))
    a = np.exp((x["dt"] + x["dt_bias"])[:, 0] * x["A"])
    assert np.allclose(h, a[..., None, None] * x["h0"], atol=1e-13)


@pytest.mark.parametrize("gate_first", [False, True])
def test_gated_norm_against_differences(gate_first):
    rng = np.random.default_rng(3)
    x, z, w = rng.standard_normal((3, 2, 5)), rng.standard_normal((3, 2, 5)), rng.standard_normal((2, 5))
    dy = rng.standard_normal(x.shape)

    def loss():
        return (delta.gated_norm(x, z, w, 0.1, gate_first) * dy).sum()
    g = delta.gated_norm(x, z, w, 0.1, gate_first, dy=dy)[1]
    for t, grad in ((x, "dx"), (z, "dz"), (w, "dweight")):
        for _ in range(5):
            at = tuple(rng.integers(0, n) for n in t.shape)
            assert abs(slope(loss, t, at) - g[grad][at]) <= 1e-7 * (1 + abs(g[grad][at])), grad


def test_prenorm_against_differences():
    rng = np.random.default_rng(4)
    x, res, w, s = rng.standard_normal((3, 7)), rng.standard_normal((3, 7)), rng.standard_normal(7), rng.standard_normal(7)
    dy, dr = rng.standard_normal(x.shape), rng.standard_normal(x.shape)

    def loss():
        y, r = delta.prenorm(x, w, res, s, 0.1)
        return (y * dy).sum() + (r * dr).sum()
    g = delta.prenorm(x, w, res, s, 0.1, dy=dy, dr=dr)[2]
    for t, grad in ((x, "dx"), (res, "dresidual"), (w, "dweight"), (s, "dscale")):
        for _ in range(5):
            at = tuple(rng.integers(0, n) for n in t.shape)
            assert abs(slope(loss, t, at) - g[grad][at]) <= 1e-7 * (1 + abs(g[grad][at])), grad
