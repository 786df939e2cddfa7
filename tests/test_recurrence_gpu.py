"""GPU: the gated linear recurrence, its gradients and its one-token step against
the fp64 formulas.

Tolerances, in half steps of fp32, u = 2^-24, with gate inputs |v| <= 6:
sigmoid: the exponent v log2(e) is off by 2 |v| u, exp2 and reciprocal by a step (2 u)
each, 1 + e by u: (2 |v| + 5) u <= 17 u of itself. s = rate softplus(lam) r: 6 u more,
23 u. a = 1 - em with em off by 26 u of itself and em <= s: for s up to 1/2 13 u + u;
beyond, exp2 is off by s (23 + 2) u + 2 u of itself and a s <= 0.37: 12 u. So a is off
by 14 u. m: half of em's 26 u and the square root's: 17 u of itself; b = m i x: 36 u.
The state then has E_t = a E_{t-1} + A u |h_{t-1}| + C u |b_t| + 2 u |h_t|; composing
runs' maps rounds each token's product once or twice more. A = 16, C = 38 hold all.
Back in time the same with g: E_t = a_{t+1} E_{t+1} + 16 u |g_{t+1}| + 4 u |up_t| + 2 u |g_t|.
Outputs are products of these with factors off by: m i 34 u, 1 - i and 1 - r (from e, or
1 - i where i <= 1/2) 34 u, s 23 u, s / m 23 + 17 u: each term's sum is below 100 u of
its size. A bf16 output is rounded once, 2^-8 of itself at most half a step (2^-9 + the
fp32 error): 2^-8 covers it.
"""
import numpy as np
import pytest

from gpu_util import say, torch_cuda
from oracle import block

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    torch = torch_cuda()
    import selective_state_space_78_amd as ssm
    ssm.lib()
    return torch, ssm


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def inputs(torch, B, L, D, dtype, gate=False, h0=False, reset=False, strided=False, seed=0, lead=None):
    g = torch.Generator(device="cuda").manual_seed(seed * 1000 + B * 37 + L * 11 + D)
    lead = (B, L) if lead is None else lead
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    cut = [(1.5 * rnd(*lead, D)).clamp(-6, 6).to(dtype) for _ in range(4)]
    if strided:
        row = torch.cat(cut, -1)
        cut = list(torch.split(row, D, -1))
    # decays of 0.2 to 0.9995 with the gate open, and one channel of none
    lam = torch.log(torch.expm1(torch.exp(torch.empty(D, device="cuda").uniform_(-7.6, 0.5, generator=g)) / 8))
    s = dict(x=cut[0], rgate=cut[1], igate=cut[2], lam=lam, gate=cut[3] if gate else None,
             h0=rnd(B, D) if h0 else None, reset=torch.rand(lead, generator=g, device="cuda") < 0.05 if reset else None)
    s["dy"], s["dh_last"] = rnd(*lead, D).to(dtype), rnd(B, D)
    return s


def reference(s, **opts):
    """The fp64 results, and how far each may be off in fp32."""
    n = {k: (v.cpu().numpy() if k == "reset" and v is not None else np64(v)) for k, v in s.items()}
    y, h, g = block.gated_recurrence(**n, **opts)
    a, m, r, i, e = block.recurrence_parts(n["x"], n["rgate"], n["igate"], n["lam"], n["reset"])
    B, L, D = n["x"].shape
    b = np.abs(m * i * n["x"])
    st = np.abs(g["h"])
    E = np.zeros((B, L + 1, D))
    for t in range(L):
        E[:, t + 1] = a[:, t] * E[:, t] + U * (16 * st[:, t] * (a[:, t] > 0) + 38 * b[:, t] + 2 * st[:, t + 1])
    up = np.abs(n["dy"] if n["gate"] is None else n["dy"] * n["gate"])
    G = np.abs(g["g"])
    F, back = np.zeros((B, L + 1, D)), np.concatenate([G[:, 1:], np.abs(n["dh_last"])[:, None]], 1)
    nexta = np.concatenate([a[:, 1:], np.ones((B, 1, D))], 1)
    for t in range(L - 1, -1, -1):
        F[:, t] = nexta[:, t] * F[:, t + 1] + U * (16 * back[:, t] * (nexta[:, t] > 0) + 4 * up[:, t] + 2 * G[:, t])
    F = F[:, :L]
    with np.errstate(divide="ignore", invalid="ignore"):
        ratio = np.where(m > 0, e / m, 0.0)
    keep = (a > 0)
    terms = keep * a * (a * np.abs(i * n["x"]) * ratio + e * st[:, :-1])
    soft = keep * (a * np.abs(i * n["x"]) * ratio + e * st[:, :-1])
    dw = 100 * U * terms + 14 * U * soft + a * e * E[:, :-1]
    off = dict(y=E[:, 1:] * (1 if n["gate"] is None else np.abs(n["gate"])) + 2 * U * np.abs(y), h_last=E[:, -1],
               dx=F * m * i + 100 * U * G * m * i, digate=F * b * (1 - i) + 100 * U * G * b * (1 - i),
               drgate=(1 - r) * (F * terms + G * dw + 40 * U * G * terms), dh0=a[:, 0] * F[:, 0] + 16 * U * G[:, 0],
               dgate=np.abs(n["dy"]) * E[:, 1:] + 4 * U * np.abs(n["dy"] * st[:, 1:]))
    # the sum over tokens: up to 24 additions in fp32, the rest in 64 bits; its factor 12 u
    each = G * np.abs(g["w"])
    ratio = block.sigmoid(n["lam"]) / block.softplus(n["lam"])
    off["dlam"] = ratio * ((F * terms + G * dw).sum((0, 1)) + 40 * U * each.sum((0, 1)))
    return dict(g, y=y, h_last=h), off


def check(got, ref, off):
    worst = {}
    for k, v in got.items():
        if v is None:
            continue
        r, o = ref[k], off[k]
        if v.dtype.itemsize == 2:
            o = o + 2.0 ** -8 * np.abs(r)
        d = np.abs(np64(v) - r)
        assert np.isfinite(np64(v)).all(), k
        worst[k] = float((d / np.maximum(o, 1e-37)).max()) if d.size else 0.0
    assert all(w <= 1 for w in worst.values()), worst
    return worst


def outputs(ssm, s, **opts):
    ins, kw = (s["x"], s["rgate"], s["igate"], s["lam"]), dict(h0=s["h0"], gate=s["gate"], reset=s["reset"], **opts)
    y, h, saved = ssm.ssm_glr_fwd_save(*ins, **kw)
    g = ssm.ssm_glr_bwd_saved(*ins, s["dy"], saved, dh_last=s["dh_last"], **kw)
    return dict(g, y=y, h_last=h)


# one token; a stream, a kept state, a chunk of each type and their borders; more chunks than are looked back over
LENGTHS = [1, 2, 8, 9, 17, 127, 128, 129, 255, 256, 257, 513, 2600]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("L", LENGTHS)
def test_lengths(env, L, dtype):
    torch, ssm = env
    for k, D in enumerate((64, 70, 33)):
        s = inputs(torch, 2, L, D, getattr(torch, dtype), gate=k != 1, h0=k != 2, reset=k == 1, strided=k == 0)
        got = outputs(ssm, s)
        torch.cuda.synchronize()
        say(dtype, L, D, check(got, *reference(s)))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("D", [1, 2, 3, 31, 32, 63, 65, 128, 200])
def test_widths(env, D, dtype):
    torch, ssm = env
    s = inputs(torch, 3, 300, D, getattr(torch, dtype), gate=True, h0=True, reset=True, strided=D % 2 == 1)
    got = outputs(ssm, s)
    torch.cuda.synchronize()
    say(dtype, D, check(got, *reference(s)))


def test_many_chunks_at_once(env):
    """Some 1300 workgroups that look back over one another, twice with the same results."""
    torch, ssm = env
    s = inputs(torch, 1, 10240, 1024, torch.bfloat16, h0=True)
    one, two = outputs(ssm, s), outputs(ssm, s)
    torch.cuda.synchronize()
    say(check(one, *reference(s)))
    for k in one:
        assert one[k] is None or torch.equal(one[k], two[k]), k


def test_forms_give_the_same(env):
    """The recomputing backward, the forward without keeping, given outputs, a state in place, unaligned tensors."""
    torch, ssm = env
    s = inputs(torch, 2, 700, 96, torch.bfloat16, gate=True, h0=True)
    base = outputs(ssm, s)
    ins, kw = (s["x"], s["rgate"], s["igate"], s["lam"]), dict(gate=s["gate"])
    g = ssm.ssm_glr_bwd(*ins, s["dy"], h0=s["h0"], dh_last=s["dh_last"], **kw)
    y, h = ssm.ssm_glr_fwd(*ins, h0=s["h0"], **kw)
    state = s["h0"].clone()
    y2, h2 = ssm.ssm_glr_fwd(*ins, h0=state, h_last=state, **kw)
    dstate = s["dh_last"].clone()
    g2 = ssm.ssm_glr_bwd(*ins, s["dy"], h0=s["h0"], dh_last=dstate, out=dict(dh0=dstate), **kw)
    torch.cuda.synchronize()
    assert h2 is state and g2["dh0"] is dstate
    for k, v in dict(g, y=y, h_last=h).items():
        assert torch.equal(v, base[k]), k
    for k, v in dict(g2, y=y2, h_last=h2).items():
        assert torch.equal(v, base[k]), k
    # one element off a pair's address: single channels, whose tiles and sums are the same operations
    off = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)
    odd = outputs(ssm, dict(s, x=off(s["x"]), dy=off(s["dy"])))
    torch.cuda.synchronize()
    for k, v in odd.items():
        assert torch.equal(v, base[k]), k


def test_split_resume(env):
    """A sequence in two calls, the state handed over, gives the tolerances of one."""
    torch, ssm = env
    s = inputs(torch, 2, 500, 64, torch.float32, h0=True)
    cut = lambda a, b: {k: (v[:, a:b].contiguous() if v is not None and v.dim() == 3 else v) for k, v in s.items()}
    p, q = cut(0, 333), cut(333, 500)
    y1, h1 = ssm.ssm_glr_fwd(p["x"], p["rgate"], p["igate"], s["lam"], h0=s["h0"])
    y2, h2 = ssm.ssm_glr_fwd(q["x"], q["rgate"], q["igate"], s["lam"], h0=h1)
    check(dict(y=torch.cat([y1, y2], 1), h_last=h2), *reference(s))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("B,D", [(1, 1), (1, 64), (5, 70), (256, 514), (300, 2000)])
def test_step(env, B, D, dtype):
    torch, ssm = env
    s = inputs(torch, B, 1, D, getattr(torch, dtype), gate=D != 70, h0=True, reset=D == 70, strided=D == 514, lead=(B,))
    ins, kw = (s["x"], s["rgate"], s["igate"], s["lam"]), dict(gate=s["gate"], reset=s["reset"])
    out = torch.empty_like(s["h0"])
    y = ssm.ssm_glr_state_update(*ins, s["h0"], h_out=out, **kw)
    h = s["h0"].clone()
    y2 = ssm.ssm_glr_state_update(*ins, h, **kw)
    torch.cuda.synchronize()
    assert torch.equal(h, out) and torch.equal(y, y2)
    one = {k: (v[:, None] if v is not None and k not in ("lam", "h0", "dh_last") else v) for k, v in s.items()}
    ref, off = reference(one)
    check(dict(y=y[:, None], h_last=h), ref, off)


def test_padding_and_infinities(env):
    """Tokens with rgate of minus infinity leave the state; a reset hides what came before; the rest stays apart."""
    torch, ssm = env
    s = inputs(torch, 3, 400, 64, torch.float32, h0=True)
    full = outputs(ssm, s)
    pad = {k: (v.clone() if v is not None else None) for k, v in s.items()}
    pad["rgate"][1, 150:] = -float("inf")
    pad["dy"][1, 150:] = 0
    got = outputs(ssm, pad)
    cut = {k: (v[1:2, :150].contiguous() if v is not None and v.dim() == 3 else v[1:2] if v is not None and k != "lam" else v)
           for k, v in s.items()}
    short = outputs(ssm, cut)
    torch.cuda.synchronize()
    for k in ("y", "dx", "drgate", "digate"):
        assert torch.isfinite(got[k]).all()
        assert torch.equal(got[k][0], full[k][0]) and torch.equal(got[k][2], full[k][2]), k
        if k != "y":
            assert not got[k][1, 150:].any(), k
    ref, off = reference(cut)
    # padded runs map h to 1 h + 0, exactly; what the run and the chunk that the padding begins in leave behind is the
    # same state by other roundings: 22 tokens and 16 runs, two roundings each, of what their magnitudes add up to
    a, m, _, i, _ = block.recurrence_parts(*(np64(cut[k]) for k in ("x", "rgate", "igate", "lam")))
    size = np.abs(ref["h"][0, 128])
    most = size
    for t in range(128, 150):
        size = a[0, t] * size + np.abs(m * i * np64(cut["x"]))[0, t]
        most = np.maximum(most, size)
    tail = np64(got["y"][1, 150:])
    assert (np.abs(tail - tail[:1]) <= 2 * 2 * (22 + 16) * U * most).all()
    assert torch.equal(got["y"][1, 256:], got["h_last"][1].expand(144, 64))
    check(dict({k: got[k][1:2, :150] for k in ("y", "dx", "drgate", "digate")}, h_last=got["h_last"][1:2],
               dh0=got["dh0"][1:2]), ref, off)
    check(short, ref, off)
    # a state of NaN and an infinite token, then a reset behind both
    bad = {k: (v.clone() if v is not None else None) for k, v in s.items()}
    bad["reset"] = torch.zeros(3, 400, dtype=torch.bool, device="cuda")
    bad["reset"][0, 200] = True
    bad["h0"][0] = float("nan")
    bad["x"][0, 100, 3] = float("inf")
    got = outputs(ssm, bad)
    torch.cuda.synchronize()
    assert not torch.isfinite(got["y"][0, :200]).any()
    assert torch.isfinite(got["y"][0, 200:]).all() and torch.isfinite(got["h_last"]).all()
    assert torch.isfinite(got["y"][1:]).all() and torch.isfinite(got["dx"]).all() and torch.isfinite(got["digate"][1:]).all()
    # (a reset's input is not scaled: the sequence by itself starts with one too)
    clean = {k: (v[0:1, 200:].contiguous() if v is not None and v.dim() > 1 else v) for k, v in bad.items()}
    clean.update(h0=None, dh_last=s["dh_last"][0:1])
    ref, off = reference(clean)
    check(dict({k: got[k][0:1, 200:] for k in ("y", "dx", "drgate", "digate")}, h_last=got["h_last"][0:1]), ref, off)


def test_extreme_gates(env):
    """Gates of +-100 and rates from nearly none to a state that lasts no token."""
    torch, ssm = env
    s = inputs(torch, 1, 200, 64, torch.float32, h0=True)
    s["rgate"][0, ::3] = 100
    s["rgate"][0, 1::3] = -100
    s["igate"][0, ::2] = -100
    s["lam"][:20] = torch.linspace(-60, 60, 20, device="cuda")
    got = outputs(ssm, s)
    torch.cuda.synchronize()
    assert all(torch.isfinite(v).all() for v in got.values() if v is not None)
    n = {k: np64(v) for k, v in s.items()}
    y, h, g = block.gated_recurrence(**{k: v for k, v in n.items() if v is not None})
    # exp2's argument of 144 is off by 100 of its half steps: 2e-5 of a sigmoid of exp(-100), which is nothing of y
    assert np.allclose(np64(got["y"]), y, rtol=1e-5, atol=1e-5) and np.allclose(np64(got["dx"]), g["dx"], rtol=1e-5, atol=1e-5)


def test_input_gates_in_fp32(env):
    """Where every token starts a sequence y = sigmoid(igate) x: against its own size, to values of 1e-37. The gate's
    exponent is known to twice fp32's digits; exp2 and the reciprocal 2 u each, four products or sums u each: 10 u."""
    torch, ssm = env
    gate = torch.linspace(-86, 86, 4096, device="cuda")
    for D in (64, 1):
        i = gate.view(1, -1, D)
        x = torch.linspace(0.5, 2, 4096, device="cuda").view_as(i)
        reset = torch.ones(i.shape[:2], dtype=torch.bool, device="cuda")
        y, _ = ssm.ssm_glr_fwd(x, x, i, torch.zeros(D, device="cuda"), reset=reset)
        step = ssm.ssm_glr_state_update(x[:, 3], x[:, 3], i[:, 3], torch.zeros(D, device="cuda"), torch.ones(1, D, device="cuda"),
                                        reset=reset[:, 3])
        torch.cuda.synchronize()
        want = block.sigmoid(np64(i)) * np64(x)
        off = np.abs(np64(y) - want) / want
        say("input gates", D, float(off.max() / U))
        assert off.max() <= 10 * U and torch.equal(step, y[:, 3])


@pytest.mark.parametrize("B,D", [(200000, 8), (70001, 33)])
def test_more_batch_rows_than_a_grid_is_high(env, B, D):
    """Rows keep to themselves: a large batch gives what its parts give, to the bit."""
    torch, ssm = env
    s = inputs(torch, B, 2, D, torch.float32, h0=True)
    cut = lambda v, r: v if v is None or v.shape[0] != B else v[r]
    ins = ("x", "rgate", "igate")
    whole = outputs(ssm, s)
    h = s["h0"].clone()
    y = ssm.ssm_glr_state_update(*(s[k][:, 0].contiguous() for k in ins), s["lam"], h)
    for r in (slice(0, 1000), slice(B - 1000, B)):
        part = {k: cut(v, r) for k, v in s.items()}
        got = outputs(ssm, part)
        h1 = part["h0"].clone()
        y1 = ssm.ssm_glr_state_update(*(part[k][:, 0].contiguous() for k in ins), s["lam"], h1)
        torch.cuda.synchronize()
        assert torch.equal(y[r], y1) and torch.equal(h[r], h1)
        for k, v in got.items():
            assert k == "dlam" or v is None or torch.equal(whole[k][r], v), k


@pytest.mark.parametrize("dtype,D,stride", [("float32", 64, 2 ** 24 - 1), ("bfloat16", 66, 2 ** 24 - 2), ("bfloat16", 33, 2 ** 24 - 1)])
def test_rows_as_far_apart_as_can_be(env, dtype, D, stride):
    """A wave's rows span up to 2^31 bytes, in memory that ends with the last row: as dense rows, bit for bit."""
    torch, ssm = env
    B, L, t = 2, 75, getattr(torch, dtype)
    g = torch.Generator(device="cuda").manual_seed(D)
    dense = [torch.randn(B, L, D, generator=g, device="cuda").to(t) for _ in range(3)]
    dy, lam = torch.randn(B, L, D, generator=g, device="cuda").to(t), torch.randn(D, generator=g, device="cuda")
    wide = []
    for v in dense:
        wide.append(torch.empty((B * L - 1) * stride + D, dtype=t, device="cuda").as_strided((B, L, D), (L * stride, stride, 1)))
        wide[-1].copy_(v)
    (y, h), (want, last) = ssm.ssm_glr_fwd(*wide, lam), ssm.ssm_glr_fwd(*dense, lam)
    grads, ref = ssm.ssm_glr_bwd(*wide, lam, dy), ssm.ssm_glr_bwd(*dense, lam, dy)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(h, last)
    assert all(torch.equal(grads[n], ref[n]) for n in ("dx", "drgate", "digate", "dlam", "dh0"))


def test_empty(env):
    torch, ssm = env
    z = lambda *s: torch.zeros(s, device="cuda")
    h0 = torch.randn(2, 8, device="cuda")
    y, h, saved = ssm.ssm_glr_fwd_save(z(2, 0, 8), z(2, 0, 8), z(2, 0, 8), z(8), h0=h0)
    g = ssm.ssm_glr_bwd_saved(z(2, 0, 8), z(2, 0, 8), z(2, 0, 8), z(8), z(2, 0, 8), saved, dh_last=h0)
    y0, hn = ssm.ssm_glr_fwd(z(2, 0, 8), z(2, 0, 8), z(2, 0, 8), z(8))
    torch.cuda.synchronize()
    assert torch.equal(h, h0) and torch.equal(g["dh0"], h0) and not g["dlam"].any() and not hn.any()
    g = ssm.ssm_glr_bwd(z(0, 5, 8), z(0, 5, 8), z(0, 5, 8), z(8), z(0, 5, 8))
    torch.cuda.synchronize()
    assert not g["dlam"].any()
    assert ssm.ssm_glr_state_update(z(0, 8), z(0, 8), z(0, 8), z(8), z(0, 8)).shape == (0, 8)


def test_captured(env):
    """A training pass in a graph, replayed on new inputs with eager work between, two graphs on one workspace."""
    torch, ssm = env
    s = inputs(torch, 2, 600, 64, torch.bfloat16, gate=True, h0=True)
    ins, kw = (s["x"], s["rgate"], s["igate"], s["lam"]), dict(h0=s["h0"], gate=s["gate"])
    ws = torch.empty(ssm.ssm_glr_bwd_workspace_size(2, 600, 64), dtype=torch.uint8, device="cuda")

    def run():
        y, h, saved = ssm.ssm_glr_fwd_save(*ins, workspace=ws, **kw)
        return dict(ssm.ssm_glr_bwd_saved(*ins, s["dy"], saved, dh_last=s["dh_last"], **kw), y=y, h_last=h)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        graphs.append((g, out))
    for k in range(3):
        s["x"].copy_(torch.randn(s["x"].shape, device="cuda"))
        for g, out in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = run()
        torch.cuda.synchronize()
        for g, out in graphs:
            for n in want:
                assert torch.equal(out[n], want[n]), (k, n)
