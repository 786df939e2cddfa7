"""GPU: the gated delta rule (sequence, gradients, one token) against the fp64
reference, token by token, through the public binding.

Tolerances, all relative to max(|reference|, rms of the reference):
* bf16 outputs: one rounding, 2^-8, and 2^-12 for what precedes it.
* fp32 states: sums of up to 64 tokens and 128 + 64 products each, every term
  and partial sum within half a step of fp32: 256 * 2^-24.
* dA, ddt_bias: the same, relative to the sum of their terms' magnitudes.
"""
import numpy as np
import pytest

from gpu_util import say, torch_cuda
from oracle import delta

pytestmark = pytest.mark.gpu

TOL_BF = 2.0 ** -8 + 2.0 ** -12
TOL_32 = 256 * 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    torch = torch_cuda()
    import selective_state_space_78_amd as ssm
    ssm.lib()
    return torch, ssm


def err(got, ref):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape and np.isfinite(got).all()
    if got.size == 0:
        return 0.0
    rms = float(np.sqrt(np.mean(ref * ref)))
    return float(np.max(np.abs(got - ref) / np.maximum(np.maximum(np.abs(ref), rms), 1e-30)))


def np64(t):
    return t.detach().double().cpu().numpy()


def inputs(torch, seed, B, L, G, H, P, N, strided=False, h0=True, bias=True, unit=False, grads=False, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    bf = torch.bfloat16
    q, k, v = rnd(B, L, G, N), rnd(B, L, G, N) + 0.3, rnd(B, L, H, P)
    if unit:
        k = k / k.norm(dim=-1, keepdim=True)
        q = q / q.norm(dim=-1, keepdim=True)
    q, k, v, dt, beta = q.to(bf), k.to(bf), v.to(bf), (spread * rnd(B, L, H)).to(bf), rnd(B, L, H).to(bf)
    if strided:
        row = torch.cat([q.reshape(B, L, G * N), k.reshape(B, L, G * N), v.reshape(B, L, H * P), dt, beta,
                         rnd(B, L, (-2 * H) % 8 + 8).to(bf)], -1)
        cut = np.cumsum([0, G * N, G * N, H * P, H, H])
        q, k = (row[..., a:b].unflatten(-1, (G, N)) for a, b in ((cut[0], cut[1]), (cut[1], cut[2])))
        v = row[..., cut[2]:cut[3]].unflatten(-1, (H, P))
        dt, beta = row[..., cut[3]:cut[4]], row[..., cut[4]:cut[5]]
    x = dict(q=q, k=k, v=v, dt=dt, beta=beta, A=-(0.05 + 2.0 * torch.rand(H, generator=g, device="cuda")))
    x["h0"] = rnd(B, H, P, N) if h0 else None
    x["dt_bias"] = rnd(H) - 2.0 if bias else None
    if grads:
        x["dy"], x["dh_last"] = rnd(B, L, H, P).to(bf), rnd(B, H, P, N)
    return x


OPTS = dict(dt_softplus=True, beta_sigmoid=True, qk_norm=True)


def reference(x, **opts):
    return delta.delta_rule(**{n: None if t is None else np64(t) for n, t in x.items()}, **opts)


def check_fwd(torch, ssm, x, **opts):
    y, h = ssm.ssm_gdr_fwd(**x, **opts)
    torch.cuda.synchronize()
    yr, hr = reference(x, **opts)
    ey, eh = err(np64(y), yr), err(np64(h), hr)
    say("  y %.2e, h_last %.2e" % (ey, eh))
    assert ey <= TOL_BF and eh <= TOL_32, (ey, eh)
    return y, h


def check_grads(torch, ssm, x, saved=True, **opts):
    ins = {n: t for n, t in x.items() if n not in ("dy", "dh_last")}
    if saved:
        _, _, ws = ssm.ssm_gdr_fwd_save(**ins, **opts)
        g = ssm.ssm_gdr_bwd_saved(**x, saved=ws, **opts)
    else:
        g = ssm.ssm_gdr_bwd(**x, **opts)
    torch.cuda.synchronize()
    ref = reference(x, **opts)[2]
    e = {n: err(np64(g[n]), ref[n]) for n in ("dq", "dk", "dv", "ddt", "dbeta", "dh0")}
    for n in ("dA", "ddt_bias"):
        if g[n] is not None:
            e[n] = float(np.max(np.abs(np64(g[n]) - ref[n]) / np.maximum(ref[n + "_abs"], 1e-30)))
    say("  " + ", ".join("%s %.2e" % p for p in e.items()))
    for n, v in e.items():
        assert v <= (TOL_BF if n in ("dq", "dk", "dv", "ddt", "dbeta") else TOL_32), (n, v)
    return g


SHAPES = [   # B, L, G, H, P, N: one token to several chunks, ragged ends, every split of columns
    (1, 1, 1, 1, 16, 64), (2, 2, 1, 2, 48, 128), (1, 63, 2, 2, 64, 64), (2, 64, 1, 3, 80, 128), (1, 65, 3, 3, 96, 64),
    (2, 130, 2, 4, 128, 128), (1, 200, 1, 1, 256, 128), (3, 77, 2, 6, 112, 64), (1, 257, 1, 5, 160, 64)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("strided", [False, True])
def test_forward(env, shape, strided):
    torch, ssm = env
    say("gdr forward", shape, "strided" if strided else "dense")
    check_fwd(torch, ssm, inputs(torch, sum(shape), *shape, strided=strided), **OPTS)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("strided", [False, True])
def test_gradients(env, shape, strided):
    torch, ssm = env
    say("gdr gradients", shape, "strided" if strided else "dense")
    check_grads(torch, ssm, inputs(torch, sum(shape), *shape, strided=strided, grads=True), **OPTS)


@pytest.mark.parametrize("softplus,sigmoid,norm", [(False, False, False), (True, False, False), (False, True, True)])
def test_options(env, softplus, sigmoid, norm):
    """Steps and strengths as given, without initial state, bias or a gradient
    of the last state; another readout scale."""
    torch, ssm = env
    x = inputs(torch, 5, 2, 100, 2, 4, 64, 64, h0=False, bias=softplus, unit=not norm, grads=True)
    x["dh_last"] = None
    if not softplus:
        x["dt"] = x["dt"].abs()
    if not sigmoid:
        x["beta"] = (x["beta"].abs() * 0.3).clamp(max=1.0)
    opts = dict(dt_softplus=softplus, beta_sigmoid=sigmoid, qk_norm=norm, scale=0.3)
    say("gdr options", opts)
    check_fwd(torch, ssm, {n: t for n, t in x.items() if n not in ("dy", "dh_last")}, **opts)
    check_grads(torch, ssm, x, saved=False, **opts)


@pytest.mark.parametrize("shape", [(2, 300, 2, 4, 128, 128), (2, 300, 2, 4, 128, 64), (1, 200, 160, 160, 128, 128)])
def test_y_rounded_once(env, shape):
    """y is the exact value rounded to bf16, but where what fp32 arithmetic leaves
    carries it over a border between two roundings: an error e before the rounding
    does so for a share |e| / step of the elements, and moves each by a step. Sums of
    up to 256 products, each rounded by half a step of fp32 in a direction of its own,
    leave sqrt(256) half steps of the rms."""
    torch, ssm = env
    x = inputs(torch, sum(shape), *shape, h0=False)
    y, _ = ssm.ssm_gdr_fwd(**x, **OPTS)
    torch.cuda.synchronize()
    ref = reference(x, **OPTS)[0]
    want = torch.from_numpy(ref).to(torch.bfloat16).double().numpy()
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(ref), 1e-30))) - 7)
    size = 16 * 2.0 ** -24 * np.sqrt(np.mean(ref * ref))
    moved = np64(y) - want
    share = float((moved * moved).sum() / (size * step).sum())
    say("gdr rounding of y", shape, "%d of %d elements, %.3f of the bound" % ((moved != 0).sum(), moved.size, share))
    assert share <= 1


def test_bias_without_softplus(env):
    """A step that is dt + bias as given (here also negative: a growing state),
    and dh0 written over dh_last."""
    torch, ssm = env
    x = inputs(torch, 15, 1, 80, 1, 2, 32, 128, unit=True, grads=True)
    x["dt"] = (0.02 * x["dt"]).to(torch.bfloat16)
    x["dt_bias"] = torch.tensor([0.05, -0.01], device="cuda")
    opts = dict(beta_sigmoid=True)
    g = check_grads(torch, ssm, x, **opts)
    dh = x["dh_last"].clone()
    h = ssm.ssm_gdr_bwd(**dict(x, dh_last=dh), out=dict(dh0=dh), **opts)
    torch.cuda.synchronize()
    assert h["dh0"].data_ptr() == dh.data_ptr()
    for n in g:
        assert torch.equal(g[n], h[n]), n


@pytest.mark.parametrize("softplus", [False, True])
@pytest.mark.parametrize("shape", [(2, 150, 3, 6, 64, 64), (1, 200, 6, 6, 96, 128)])
def test_gradients_of_strong_decays(env, shape, softplus):
    """Decays per token from exp(-0.5) to exp(-44), a head each: the gradients of the
    step, its bias and the rate keep their digits relative to that head's own terms,
    each of which has the token's decay as a factor. Then the same with
    mild tokens between strong ones."""
    torch, ssm = env
    B, L, G, H, P, N = shape
    x = inputs(torch, sum(shape), *shape, bias=softplus, grads=True)
    x["dt"] = 1.0 + 0.1 * x["dt"].float()
    if softplus:
        x["dt"], x["dt_bias"] = x["dt"] - 0.5, torch.full((H,), 0.5, device="cuda")
    x["dt"] = x["dt"].to(torch.bfloat16)
    x["A"] = -torch.tensor([0.5, 4.0, 8.0, 16.0, 28.0, 44.0], device="cuda")
    opts = dict(OPTS, dt_softplus=softplus)

    def check(what):
        g = ssm.ssm_gdr_bwd(**x, **opts)
        torch.cuda.synchronize()
        ref = reference(x, **opts)[2]
        bad = []
        for h in range(H):
            e = dict(ddt=err(np64(g["ddt"])[..., h], ref["ddt"][..., h]))
            for n in ("dA", "ddt_bias")[:1 + softplus]:
                e[n] = float(abs(np64(g[n])[h] - ref[n][h]) / ref[n + "_abs"][h])
            say("  %s, rate %.1f: " % (what, float(x["A"][h])), ", ".join("%s %.2e" % p for p in e.items()))
            bad += [(h, n, v) for n, v in e.items() if not v <= (TOL_BF if n == "ddt" else TOL_32)]
        assert not bad, bad
    check("every token")
    # one token in nine decays strongly
    mild = torch.arange(L, device="cuda") % 9 != 4
    x["dt"][:, mild] = -6.0 if softplus else 1.0 / 512
    check("one in nine")


def test_no_lean_with_rows_of_one_sign(env):
    """The gradients are linear in dy and dh_last: those of the negative are the
    negative, but for the matrix cores' rounding downwards. With keys and queries
    behind a SiLU that must not gather in the decay's gradients: what a pair of
    gradients adds up to is as often above zero as below it, so over 64 heads its mean
    is within 4 standard errors of zero (all but one draw in 16000), and the
    sums are within twice this file's tolerance of sums."""
    torch, ssm = env
    x = inputs(torch, 17, 8, 2048, 64, 64, 64, 128, h0=False, grads=True)
    for n in "qk":
        x[n] = torch.nn.functional.silu(1.5 * x[n].float()).to(torch.bfloat16)
    g = ssm.ssm_gdr_bwd(**x, **OPTS)
    m = ssm.ssm_gdr_bwd(**dict(x, dy=-x["dy"], dh_last=-x["dh_last"]), **OPTS)
    torch.cuda.synchronize()
    for n in ("dA", "ddt_bias"):
        a, d = np64(g[n]), np64(g[n]) + np64(m[n])
        z = d.mean() / (d.std() / 8)
        say("  %s: sums %.2e of the gradients, mean %.2f standard errors" % (n, np.linalg.norm(d) / np.linalg.norm(a), z))
        assert abs(z) <= 4 and np.linalg.norm(d) <= 2 * TOL_32 * np.linalg.norm(a), n


def test_step_of_a_long_sequence(env):
    """Tokens taken out of a (batch, L, ...) tensor: batch rows L rows apart, here
    further than 2^24 elements."""
    torch, ssm = env
    L, G, H, P, N = 9000, 16, 16, 128, 128
    far = torch.empty((2, L, G * N), dtype=torch.bfloat16, device="cuda")
    x = inputs(torch, 16, 2, 1, G, H, P, N)
    cut = []
    for n, w in (("q", (G, N)), ("k", (G, N)), ("v", (H, P))):
        far[:, 7] = x[n].flatten(-2)[:, 0]
        cut.append(far.clone()[:, 7].unflatten(-1, w))
    assert cut[0].stride(0) > 1 << 24
    h = x["h0"].clone()
    y = ssm.ssm_gdr_state_update(*cut, x["dt"][:, 0], x["beta"][:, 0], x["A"], h, dt_bias=x["dt_bias"], **OPTS)
    torch.cuda.synchronize()
    yr, hr = reference(x, **OPTS)
    assert err(np64(y), yr[:, 0]) <= TOL_BF and err(np64(h), hr) <= TOL_32


def test_repeated_keys(env):
    """Every key the same and every strength 1: the chunk's triangular system at
    its least regular (its entries do not decay away from the diagonal)."""
    torch, ssm = env
    x = inputs(torch, 6, 1, 150, 1, 2, 32, 64, unit=True, grads=True)
    x["k"] = x["k"][:, :1].expand_as(x["k"]).contiguous()
    x["beta"] = torch.ones_like(x["beta"])
    x["A"] = torch.tensor([-1e-4, 0.0], device="cuda")
    say("gdr repeated keys")
    check_fwd(torch, ssm, {n: t for n, t in x.items() if n not in ("dy", "dh_last")}, dt_softplus=True)
    check_grads(torch, ssm, x, dt_softplus=True)


def test_resets_and_idle_tokens(env):
    """Tokens that forget everything (a decay of exp(-1e4)), tokens that write
    nothing (strength 0), and zero keys and queries under unit lengths."""
    torch, ssm = env
    x = inputs(torch, 7, 2, 140, 1, 2, 48, 128, bias=False, grads=True)
    x["dt"] = x["dt"].abs() * 0.1
    x["dt"][:, 30] = 1e4
    x["dt"][:, 101:104] = 300.0
    x["beta"] = x["beta"].abs().clamp(max=1.0)
    x["beta"][:, 40:60] = 0.0
    x["k"][:, 70] = 0.0
    x["q"][:, 71] = 0.0
    x["A"] = torch.tensor([-1.0, -0.5], device="cuda")
    opts = dict(qk_norm=True, qk_eps=1e-3)
    say("gdr resets")
    check_fwd(torch, ssm, {n: t for n, t in x.items() if n not in ("dy", "dh_last")}, **opts)
    check_grads(torch, ssm, x, **opts)


@pytest.mark.parametrize("shape", [(1, 66, 200, 200, 80, 64), (2, 70, 9, 45, 112, 128), (1, 65, 64, 128, 144, 128)])
def test_many_heads(env, shape):
    """Heads enough for every launch shape of the kernels that walk the chunks:
    8 columns' waves per workgroup with a ragged end, 4, and 8 in two parts."""
    torch, ssm = env
    say("gdr many heads", shape)
    x = inputs(torch, sum(shape), *shape, grads=True)
    check_fwd(torch, ssm, {n: t for n, t in x.items() if n not in ("dy", "dh_last")}, **OPTS)
    check_grads(torch, ssm, x, saved=False, **OPTS)


def test_resets_of_any_size(env):
    """Steps from 100 to the largest bf16 and an infinite one: the state is
    forgotten, and the tokens behind keep their own decays."""
    torch, ssm = env
    x = inputs(torch, 17, 1, 100, 1, 2, 32, 64, bias=False, grads=True)
    x["dt"] = x["dt"].abs() * 0.1
    big = torch.tensor([100.0, 1e8, 1e20, 3e38, float("inf")], device="cuda").to(torch.bfloat16)
    x["dt"][0, [5, 20, 40, 41, 80]] = big[:, None]
    x["beta"] = x["beta"].abs().clamp(max=1.0)
    x["A"] = torch.tensor([-1.0, -16.0], device="cuda")
    opts = dict(qk_norm=True)
    y, h = ssm.ssm_gdr_fwd(**{n: t for n, t in x.items() if n not in ("dy", "dh_last")}, **opts)
    g = ssm.ssm_gdr_bwd(**x, **opts)
    torch.cuda.synchronize()
    # the reference with steps long enough to forget all, short enough to square
    ref = dict(x, dt=torch.where(x["dt"] > 50, torch.full_like(x["dt"], 1e5), x["dt"]))
    yr, hr, gr = reference(ref, **opts)
    assert err(np64(y), yr) <= TOL_BF and err(np64(h), hr) <= TOL_32
    for n in ("dq", "dk", "dv", "ddt", "dbeta"):
        assert err(np64(g[n]), gr[n]) <= TOL_BF, n
    # no term of dA comes from a reset
    assert float(np.max(np.abs(np64(g["dA"]) - gr["dA"]) / gr["dA_abs"])) <= TOL_32


def test_non_finite_tokens(env):
    """A NaN or an infinity stays out of the chunks before its own."""
    torch, ssm = env
    x = inputs(torch, 18, 1, 200, 1, 2, 32, 64)
    y, _ = ssm.ssm_gdr_fwd(**x, **OPTS)
    for name, value in (("v", float("nan")), ("k", float("inf")), ("beta", float("nan"))):
        bad = dict(x, **{name: x[name].clone()})
        bad[name][0, 150] = value
        z, h = ssm.ssm_gdr_fwd(**bad, **OPTS)
        torch.cuda.synchronize()
        assert torch.equal(z[:, :128], y[:, :128]) and bool(z[:, 150:].isnan().any()), name


NOT_FINITE = [("dt", float("nan")), ("beta", float("nan")), ("k", float("nan")), ("q", float("nan")), ("v", float("nan")),
              ("A", float("nan")), ("dt_bias", float("nan")), ("dt of A = 0", float("inf")), ("k", float("inf")),
              ("v", float("-inf")), ("h0", float("nan")), ("dy", float("nan")), ("dh_last", float("inf"))]


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("name,value", NOT_FINITE)
def test_what_a_non_finite_value_reaches(env, name, value, norm):
    """One value of head 1 (of token 150, in the third of five chunks): whatever is
    not finite by the formulas is not finite here, in both directions and in the
    one-token step; chunks before it, other heads and batch rows keep every bit."""
    torch, ssm = env
    x = inputs(torch, 19, 2, 300, 3, 3, 32, 64, unit=not norm, grads=True)
    if name == "dt of A = 0":
        x["A"][1] = 0.0
    bad = {n: t.clone() for n, t in x.items()}
    if name in ("A", "dt_bias"):
        bad[name][1] = value
    elif name in ("h0", "dh_last"):
        bad[name][0, 1, 3, 7] = value
    elif name in ("dt of A = 0", "beta", "dt"):
        bad[name.split()[0]][0, 150, 1] = value
    else:
        bad[name][0, 150, 1, 5] = value
    opts = dict(OPTS, qk_norm=norm)
    ins = lambda d: {n: t for n, t in d.items() if n not in ("dy", "dh_last")}
    y0, h0, _ = ssm.ssm_gdr_fwd_save(**ins(x), **opts)
    y, h, ws = ssm.ssm_gdr_fwd_save(**ins(bad), **opts)
    g0, g = ssm.ssm_gdr_bwd(**x, **opts), ssm.ssm_gdr_bwd_saved(**bad, saved=ws, **opts)
    torch.cuda.synchronize()
    with np.errstate(all="ignore"):
        yr, hr, gr = reference(bad, **opts)
    every = [("y", y, y0, yr, 2), ("h_last", h, h0, hr, 1)]
    every += [(n, g[n], g0[n], gr[n], {"dA": 0, "ddt_bias": 0, "dh0": 1}.get(n, 2)) for n in g]
    for n, got, clean, ref, dim in every:
        assert not (np.isfinite(np64(got)) & ~np.isfinite(ref)).any(), n
        for head in (0, 2):
            assert torch.equal(got.select(dim, head), clean.select(dim, head)), (n, head)
    if name not in ("A", "dt_bias", "h0"):
        assert torch.equal(y[:, :128], y0[:, :128])
    if name not in ("A", "dt_bias"):
        for n, got, clean, _, dim in every:
            assert dim == 0 or torch.equal(got[1], clean[1]), n
    if name in ("dy", "dh_last"):
        assert torch.equal(y, y0) and torch.equal(h, h0)
        return
    tok = {n: (t[:, 150:151] if n in ("q", "k", "v", "dt", "beta") else t) for n, t in ins(bad).items()}
    state = bad["h0"].clone()
    yt = ssm.ssm_gdr_state_update(*(tok[n][:, 0] for n in ("q", "k", "v", "dt", "beta")), bad["A"], state,
                                  dt_bias=bad["dt_bias"], **opts)
    torch.cuda.synchronize()
    with np.errstate(all="ignore"):
        yr, hr = reference(tok, **opts)
    assert not (np.isfinite(np64(yt)) & ~np.isfinite(yr[:, 0])).any() and not (np.isfinite(np64(state)) & ~np.isfinite(hr)).any()


def test_infinite_rate(env):
    """A = -inf makes every token a reset, also where the last chunk is ragged."""
    torch, ssm = env
    x = inputs(torch, 20, 1, 70, 1, 2, 32, 64)
    x["A"][1] = float("-inf")
    check_fwd(torch, ssm, x, **OPTS)


def test_split_and_resume(env):
    """Two calls, the second continuing the first's state in place, equal one
    over the whole, also where the cut is inside a chunk."""
    torch, ssm = env
    x = inputs(torch, 8, 2, 150, 1, 2, 64, 128)
    y, h = ssm.ssm_gdr_fwd(**x, **OPTS)
    for cut in (64, 101):
        def part(a, b):
            return {n: (t[:, a:b].contiguous() if n in ("q", "k", "v", "dt", "beta") else t) for n, t in x.items()}
        y1, state = ssm.ssm_gdr_fwd(**part(0, cut), **OPTS)
        y2, _ = ssm.ssm_gdr_fwd(**dict(part(cut, 150), h0=state), h_last=state, **OPTS)
        torch.cuda.synchronize()
        ey, eh = err(np64(torch.cat([y1, y2], 1)), np64(y)), err(np64(state), np64(h))
        say("gdr split at %d: y %.2e, h %.2e" % (cut, ey, eh))
        # each side within its own rounding of the exact value
        assert ey <= 2 * TOL_BF and eh <= 2 * TOL_32


@pytest.mark.parametrize("shape", [(1, 16, 32, 128, 128), (3, 2, 6, 48, 64), (2, 1, 3, 256, 128), (70, 1, 1, 16, 64)])
@pytest.mark.parametrize("strided", [False, True])
def test_steps(env, shape, strided):
    """Three tokens one at a time, the state in place and once to a second
    buffer, against the reference, and the layer of length one."""
    torch, ssm = env
    B, G, H, P, N = shape
    x = inputs(torch, sum(shape), B, 3, G, H, P, N, strided=strided)
    yr, hr = reference(x, **OPTS)
    h = x["h0"].clone()
    for t in range(3):
        tok = [x[n][:, t] for n in ("q", "k", "v", "dt", "beta")]
        if t == 1:
            out = torch.full_like(h, float("nan"))
            keep = h.clone()
            y = ssm.ssm_gdr_state_update(*tok, x["A"], h, h_out=out, dt_bias=x["dt_bias"], **OPTS)
            torch.cuda.synchronize()
            assert torch.equal(h, keep)
            h = out
        else:
            y = ssm.ssm_gdr_state_update(*tok, x["A"], h, dt_bias=x["dt_bias"], **OPTS)
        torch.cuda.synchronize()
        assert err(np64(y), yr[:, t]) <= TOL_BF, t
    e = err(np64(h), hr)
    say("gdr steps", shape, "h %.2e" % e)
    assert e <= TOL_32


def test_empty(env):
    torch, ssm = env
    x = inputs(torch, 9, 2, 0, 1, 2, 32, 64, grads=True)
    ins = {n: t for n, t in x.items() if n not in ("dy", "dh_last")}
    y, h = ssm.ssm_gdr_fwd(**ins, **OPTS)
    assert y.shape == (2, 0, 2, 32) and torch.equal(h, x["h0"])
    g = ssm.ssm_gdr_bwd(**x, **OPTS)
    assert torch.equal(g["dh0"], x["dh_last"]) and not g["dA"].any() and not g["ddt_bias"].any()
    _, h = ssm.ssm_gdr_fwd(**dict(ins, h0=None), **OPTS)
    assert not h.any()
    z = inputs(torch, 9, 0, 5, 1, 2, 32, 64, grads=True)
    g = ssm.ssm_gdr_bwd(**z, **OPTS)
    assert g["dq"].numel() == 0 and not g["dA"].any()


def test_neighbours_untouched(env):
    """What lies around the outputs keeps its values, at a ragged end and a
    head size that ends inside a workgroup's columns."""
    torch, ssm = env
    B, L, G, H, P, N = 1, 70, 1, 2, 48, 64
    x = inputs(torch, 10, B, L, G, H, P, N, grads=True)

    def guarded(shape, dtype):
        n = int(np.prod(shape))
        buf = torch.full((n + 512,), 7.0, dtype=dtype, device="cuda")
        return buf, buf[256:256 + n].view(shape)
    spec = dict(dq=((B, L, G, N), torch.bfloat16), dk=((B, L, G, N), torch.bfloat16), dv=((B, L, H, P), torch.bfloat16),
                ddt=((B, L, H), torch.bfloat16), dbeta=((B, L, H), torch.bfloat16), dA=((H,), torch.float32),
                ddt_bias=((H,), torch.float32), dh0=((B, H, P, N), torch.float32))
    bufs = {n: guarded(*s) for n, s in spec.items()}
    by, y = guarded((B, L, H, P), torch.bfloat16)
    bh, h = guarded((B, H, P, N), torch.float32)
    ins = {n: t for n, t in x.items() if n not in ("dy", "dh_last")}
    need = ssm.ssm_gdr_bwd_workspace_size(B, L, H, P, G, N)
    bw = torch.full((need + 512,), 9, dtype=torch.uint8, device="cuda")
    ws = bw[256:256 + need]
    _, _, saved = ssm.ssm_gdr_fwd_save(**ins, y=y, h_last=h, workspace=ws, **OPTS)
    ssm.ssm_gdr_bwd_saved(**x, saved=saved, out={n: v for n, (_, v) in bufs.items()}, **OPTS)
    torch.cuda.synchronize()
    for n, b in list((n, b) for n, (b, _) in bufs.items()) + [("y", by), ("h", bh)]:
        assert bool((b[:256] == 7).all()) and bool((b[-256:] == 7).all()), n
    assert bool((bw[:256] == 9).all()) and bool((bw[-256:] == 9).all())


def test_same_bits_and_recomputation(env):
    """Runs repeat bit for bit, the saved and the recomputing backward agree bit
    for bit, and a saved workspace serves twice."""
    torch, ssm = env
    x = inputs(torch, 11, 2, 200, 2, 4, 96, 128, grads=True)
    ins = {n: t for n, t in x.items() if n not in ("dy", "dh_last")}
    a = ssm.ssm_gdr_bwd(**x, **OPTS)
    y, h, ws = ssm.ssm_gdr_fwd_save(**ins, **OPTS)
    y2, h2 = ssm.ssm_gdr_fwd(**ins, **OPTS)
    assert torch.equal(y, y2) and torch.equal(h, h2)
    for _ in range(2):
        b = ssm.ssm_gdr_bwd_saved(**x, saved=ws, **OPTS)
        for n in a:
            assert torch.equal(a[n], b[n]), n


def test_streams_and_graph(env):
    """On a stream of its own, and captured: the replays, with new inputs and
    eager work between them, equal the eager results."""
    torch, ssm = env
    x = inputs(torch, 12, 1, 130, 1, 2, 64, 64, grads=True)
    ins = {n: t for n, t in x.items() if n not in ("dy", "dh_last")}
    ws = torch.empty(ssm.ssm_gdr_bwd_workspace_size(1, 130, 2, 64, 1, 64), dtype=torch.uint8, device="cuda")

    def step():
        y, h, _ = ssm.ssm_gdr_fwd_save(**ins, workspace=ws, **OPTS)
        return (y, h, *[g for g in ssm.ssm_gdr_bwd_saved(**x, saved=ws, **OPTS).values()])
    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    # a stream handed over, on which the call allocates its workspace itself
    y, h, ws2 = ssm.ssm_gdr_fwd_save(**ins, stream=s, **OPTS)
    other = ssm.ssm_gdr_bwd_saved(**x, saved=ws2, stream=s, **OPTS)
    s.synchronize()
    for a, b in zip(want, (y, h, *other.values())):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for k in range(4):
        x["v"].copy_(torch.randn_like(x["v"]))
        x["dy"].copy_(torch.randn_like(x["dy"]))
        graph.replay()
        kept = [t.clone() for t in got]
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(want, kept):
            assert torch.equal(a, b), k


def test_keys_without_values_are_refused(env):
    """dstate 0 is refused as any other unsupported dstate (not by a division)."""
    torch, ssm = env
    x = inputs(torch, 21, 2, 10, 1, 2, 32, 64)
    x["q"], x["k"], x["h0"] = x["q"][..., :0].contiguous(), x["k"][..., :0].contiguous(), x["h0"][..., :0].contiguous()
    with pytest.raises(ssm.SsmError) as e:
        ssm.ssm_gdr_fwd(**x)
    assert e.value.status == -4


def test_refusals(env):
    torch, ssm = env
    x = inputs(torch, 13, 2, 10, 1, 2, 32, 64)
    with pytest.raises(ssm.SsmError) as e:
        ssm.ssm_gdr_fwd(**{n: (t.float() if n in ("q", "k", "v", "dt", "beta") else t) for n, t in x.items()})
    assert e.value.status == -4
    off = torch.empty(x["q"].numel() + 4, dtype=x["q"].dtype, device="cuda")[4:].view(x["q"].shape)
    with pytest.raises(ssm.SsmError) as e:
        ssm.ssm_gdr_fwd(**dict(x, q=off))                                                     # 8-byte aligned
    assert e.value.status == -8
    with pytest.raises(TypeError):
        ssm.ssm_gdr_fwd(**dict(x, k=x["k"].float()))
    with pytest.raises(ValueError):
        ssm.ssm_gdr_fwd(**dict(x, k=x["k"][:, :9]))
    with pytest.raises(ValueError):
        ssm.ssm_gdr_fwd(**dict(x, q=x["q"].transpose(0, 1).contiguous().transpose(0, 1)))   # batch rows interleaved
    with pytest.raises(ValueError):
        ssm.ssm_gdr_fwd(**dict(x, k=x["k"][:, :1].expand_as(x["k"])))                        # rows overlap
    with pytest.raises(ValueError):
        ssm.ssm_gdr_fwd(**dict(x, A=x["A"].cpu()))
    with pytest.raises(ValueError):
        ssm.ssm_gdr_fwd(**{n: t.cpu() for n, t in x.items()})
    with pytest.raises(ValueError):
        ssm.ssm_gdr_state_update(**{n: t.cpu()[:, 0] for n, t in x.items() if n in ("q", "k", "v", "dt", "beta")},
                                 A=x["A"].cpu(), h=x["h0"].cpu())
    with pytest.raises(ValueError):
        ssm.ssm_gdr_fwd(**x, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        ssm.ssm_gdr_bwd_saved(**x, dy=x["v"], saved=None)
