"""A gated linear recurrence, projections with their epilogues, and the clipping
of gradients by their global norm: cases, plain forms and calls.

What a block with a gated linear recurrence is made of, trained and served, as
the library offers it beside its scan, its delta rule and its norms:

* ``glr_fwd``, ``glr_train``, ``glr_step``: the recurrence over a sequence, its
  training pass (forward and every gradient) and its one-token form on a kept
  state. Per batch row and channel, with r = sigmoid(rgate), i = sigmoid(igate):

      a_t = exp(-RATE softplus(lam) r_t),   a_t = 0 where a sequence starts (reset)
      h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t,   y_t = h_t gate_t

* ``proj_fwd``, ``proj_bwd``: per group of channels (one group: a plain linear
  layer; several: block-diagonal weights, as the gates of the recurrence have),

      pre = x W^T + bias,   y = act(pre) + residual

  and its gradients. With an activation a training forward stores pre, in x's
  type, and the backward starts from what is stored; dpre = dy act'(pre) is
  stored in x's type as well, and dx and dweight are those of the stored dpre.
* ``clip``: the norm over all gradients of a model and
  g <- g min(1, max_norm / (norm + CLIP_EPS)).

With ``own`` false, ``run`` computes the operators from elementary torch
operations in 32 bits; with ``own`` true it calls the library.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_TYPE = {BF16: torch.bfloat16, F32: torch.float32}
RATE = 8.0
CLIP_EPS = 1e-6
TILE = 256      # elements that a tensor of a gradient bucket is padded to


# ------------------------------------------------------------------ the cases
def _glr(op, name, batch, L, dim, dtype=BF16, gate=False, h0=False, reset=False, strided=False):
    return dict(name=name, op=op, batch=batch, L=L, dim=dim, dtype=dtype, gate=gate, h0=h0, reset=reset, strided=strided)


def _proj(op, name, rows, groups, K, N, dtype=BF16, act="none", bias=False, res="none", strided=False, save=False):
    return dict(name=name, op=op, rows=rows, groups=groups, K=K, N=N, dtype=dtype, act=act, bias=bias, res=res,
                strided=strided, save=save)


def _clip(name, layers, dim, inner, state, dtype, packed=False):
    return dict(name=name, op="clip", layers=layers, dim=dim, inner=inner, state=state, dtype=dtype, packed=packed,
                max_norm=1.0)


def listed():
    return [
        # batch, length and channels of the 1.4B-shaped layer
        _glr("glr_fwd", "glr_fwd_layer_b8_l8192", 8, 8192, 4096),
        # one long document: few channels for the chip, the work is along the time
        _glr("glr_fwd", "glr_fwd_long_l131072", 1, 131072, 5120),
        # the 130M-shaped layer in training, gated by the block's other branch, from a state, inputs cut from one row
        _glr("glr_train", "glr_train_b4_l2048", 4, 2048, 1536, gate=True, h0=True, strided=True),
        # packed sequences of odd length and width in full precision
        _glr("glr_train", "glr_train_packed_f32", 3, 1021, 515, dtype=F32, reset=True),
        # the decode batch
        _glr("glr_step", "glr_step_b256", 256, 1, 5120, gate=True, h0=True),
        # into the block: 8 x 2048 tokens, gelu of the gate branch
        _proj("proj_fwd", "proj_in_16384x2048x4096", 16384, 1, 2048, 4096, act="gelu", bias=True, save=True),
        # the recurrence's gates: block-diagonal
        _proj("proj_fwd", "proj_gates_8192x12x128", 8192, 12, 128, 128, bias=True),
        # the gradients behind an activation: 4 x 2048 tokens, 768 to 1536
        _proj("proj_bwd", "proj_bwd_8192x768x1536", 8192, 1, 768, 1536, act="silu", bias=True),
        # odd sizes in full precision
        _proj("proj_bwd", "proj_bwd_odd_f32", 333, 1, 203, 517, dtype=F32, act="gelu", bias=True, res=F32),
        # one user's token out of the block into the 32-bit residual stream: the weight's bytes
        _proj("proj_fwd", "proj_out_one_token", 1, 1, 4096, 2048, res=F32),
        # all gradients of the 1.4B-shaped model: 48 layers, 432 tensors
        _clip("clip_48_layers", 48, 2048, 4096, 16, BF16),
        # one block's gradients: launches
        _clip("clip_one_block_f32", 1, 768, 1536, 16, F32),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["glr_fwd", "glr_fwd", "glr_train", "glr_train", "glr_step", "proj_fwd", "proj_fwd", "proj_bwd",
                     "proj_bwd", "clip"])
    dtype = rng.choice([BF16, BF16, F32])
    if op.startswith("glr"):
        dim = _log_int(rng, 3, 5120) if rng.random() < 0.4 else 64 * _log_int(rng, 1, 80)
        batch = _log_int(rng, 1, 256 if op == "glr_step" else 16)
        L = 1 if op == "glr_step" else _log_int(rng, 1, 65536 if op == "glr_fwd" else 8192)
        most = 2 ** 28 if op == "glr_fwd" else 2 ** 26
        while batch * L * dim > most:
            if batch > 1:
                batch //= 2
            else:
                L //= 2
        return dict(op=op, batch=batch, L=L, dim=dim, dtype=dtype, gate=rng.random() < 0.5, h0=rng.random() < 0.5,
                    reset=rng.random() < 0.4, strided=rng.random() < 0.4)
    if op.startswith("proj"):
        groups = 1 if rng.random() < 0.7 else _log_int(rng, 2, 32)
        size = lambda hi: _log_int(rng, 5, hi) if rng.random() < 0.3 else 16 * _log_int(rng, 1, hi // 16)  # noqa: E731
        K, N = (size(4096 if groups == 1 else 256) for _ in range(2))
        rows = _log_int(rng, 1, 16384)
        most = 2 ** 36 if dtype == BF16 else 2 ** 34
        while rows * groups * K * N > most:
            rows //= 2
        return dict(op=op, rows=rows, groups=groups, K=K, N=N, dtype=dtype,
                    act=rng.choice(["none", "silu", "gelu", "sigmoid"]), bias=rng.random() < 0.5,
                    res=rng.choice(["none", dtype, F32]), strided=rng.random() < 0.3, save=rng.random() < 0.5)
    dim = _log_int(rng, 7, 2048) if rng.random() < 0.5 else 64 * _log_int(rng, 1, 32)
    return dict(op=op, layers=_log_int(rng, 1, 48), dim=dim, inner=2 * dim, state=rng.choice([8, 16, 64]), dtype=dtype,
                packed=rng.random() < 0.5, max_norm=rng.choice([0.5, 1.0, 1e4]))


# ------------------------------------------------------------------- the data
def _cut(parts, strided):
    """The tensors as they are, or cut out of one row that holds them all."""
    if not strided:
        return parts
    row = torch.cat(parts, -1)
    return list(torch.split(row, [p.shape[-1] for p in parts], -1))


def _glr_inputs(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, L, D, t = c["batch"], c["L"], c["dim"], _TYPE[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    # decays a^RATE of 0.9 to 0.999 with the gate open
    a = 0.9 + 0.099 * torch.rand(D, generator=g, device="cuda")
    s = dict(lam=torch.log(torch.expm1(-torch.log(a) / RATE)))
    lead = (B,) if c["op"] == "glr_step" else (B, L)
    s["x"], s["rgate"], s["igate"] = _cut([normal(*lead, D).to(t) for _ in range(3)], c["strided"])
    s["gate"] = normal(*lead, D).to(t) if c["gate"] else None
    s["h0"] = normal(B, D) if c["h0"] or c["op"] == "glr_step" else None
    # documents of some 200 tokens
    s["reset"] = torch.rand(lead, generator=g, device="cuda") < 1 / 200 if c["reset"] else None
    if c["op"] == "glr_train":
        s["dy"] = normal(*lead, D).to(t)
        s["dh_last"] = normal(B, D)
    if c["op"] == "glr_step":
        # the state behind the token goes to the second of two buffers, as a server keeps them that may take a
        # drafted token back
        s["h_out"] = torch.empty_like(s["h0"])
    return s


def _proj_inputs(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    M, G, K, N, t = c["rows"], c["groups"], c["K"], c["N"], _TYPE[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    lead = (M,) if G == 1 else (M, G)
    x = normal(M, G * K).to(t)
    if c["strided"]:
        x = _cut([x, normal(M, 8).to(t)], True)[0]
    s = dict(x=x if G == 1 else x.unflatten(-1, (G, K)),
             weight=(normal(*(() if G == 1 else (G,)), N, K) * K ** -0.5).to(t),
             bias=0.5 * normal(*(() if G == 1 else (G,)), N) if c["bias"] else None,
             residual=normal(*lead, N).to(_TYPE[c["res"]]) if c["res"] != "none" else None)
    if c["op"] == "proj_bwd":
        s["dy"] = normal(*lead, N).to(_TYPE[c["res"]] if c["res"] != "none" else t)
        # what the forward stored
        s["pre"] = normal(*lead, N).to(t) if c["act"] != "none" else None
    return s


def _layer(c):
    """(shape, whether in 32 bits) of the gradients of one layer: projections into
    and out of the block, convolution, the mixer's parameters, the norm."""
    d, e, n = c["dim"], c["inner"], c["state"]
    return [((e, d), False), ((e, d), False), ((d, e), False), ((e, 4), True), ((e,), True), ((e, n), True), ((e,), True),
            ((e,), True), ((d,), True)]


def _clip_inputs(c, seed):
    """Gradients as views of two buckets, one of each type, as a data-parallel
    program keeps them; `packed` without padding between them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    types = (_TYPE[c["dtype"]], torch.float32)
    places, used = [], [0, 0]
    for _ in range(c["layers"]):
        for shape, wide in _layer(c):
            places.append((int(wide), used[wide], shape))
            n = math.prod(shape)
            used[wide] += n if c["packed"] else -(-n // TILE) * TILE
    flat = [torch.zeros(n, device="cuda", dtype=t) for n, t in zip(used, types)]
    for f in flat:
        for at in range(0, f.numel(), 2 ** 28):
            part = f[at:at + 2 ** 28]
            part.copy_(1e-2 * torch.randn(part.shape, generator=g, device="cuda"))
    result = [torch.zeros_like(f) for f in flat]
    view = lambda b: [b[k][at:at + math.prod(shape)].view(shape) for k, at, shape in places]  # noqa: E731
    return dict(grads=view(flat), out=view(result), flat=result)


def prepare(case, seed):
    op = case["op"]
    s = _glr_inputs(case, seed) if op.startswith("glr") else _proj_inputs(case, seed) if op.startswith("proj") else \
        _clip_inputs(case, seed)
    s["case"] = case
    return s


def work(case):
    c = case
    e = 2 if c["dtype"] == BF16 else 4
    if c["op"].startswith("glr"):
        n, bd = c["batch"] * c["L"] * c["dim"], 4 * c["batch"] * c["dim"]
        gate = n * e if c["gate"] else 0
        rest = 4 * c["dim"] + (c["batch"] * c["L"] if c["reset"] else 0)
        fwd = 4 * n * e + gate + rest
        if c["op"] == "glr_step":
            return {"bytes": fwd + 2 * bd, "flops": 30 * n}
        fwd += bd * (2 if c["h0"] else 1)
        if c["op"] == "glr_fwd":
            return {"bytes": fwd, "flops": 30 * n}
        # besides: dy and dh_last read, every gradient written
        return {"bytes": fwd + 4 * n * e + gate + bd * (2 if c["h0"] else 1) + 4 * c["dim"], "flops": 90 * n}
    if c["op"].startswith("proj"):
        M, G, K, N = c["rows"], c["groups"], c["K"], c["N"]
        x, w, y = M * G * K, G * K * N, M * G * N
        r = e if c["res"] == "none" else 2 if c["res"] == BF16 else 4
        bias = 4 * G * N if c["bias"] else 0
        pre = 0 if c["act"] == "none" else y * e
        if c["op"] == "proj_fwd":
            return {"bytes": (x + w) * e + y * r * (1 if c["res"] == "none" else 2) + bias + (pre if c["save"] else 0),
                    "flops": 2 * M * G * K * N + 10 * y}
        # x, weight, dy and pre read, dx, dweight, dbias and dpre written
        return {"bytes": 2 * (x + w) * e + y * r + pre + y * e + bias, "flops": 4 * M * G * K * N + 20 * y}
    n = sum(math.prod(shape) * (4 if wide else e) for shape, wide in _layer(c)) * c["layers"]
    k = sum(math.prod(shape) for shape, _ in _layer(c)) * c["layers"]
    return {"bytes": 2 * n, "flops": 3 * k}


# ---------------------------------------------- the recurrence in its plain form
def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _runs(a, b, h0):
    """h_t = a_t h_{t-1} + b_t over (B, L, D): chunks side by side from nothing,
    their starting states one after another, then both added."""
    B, L, D = a.shape
    C = max(1, int(math.sqrt(L)))
    nc = -(-L // C)
    full = a.new_ones((B, nc * C, D))
    full[:, :L] = a
    a, full = full.unflatten(1, (nc, C)), a.new_zeros((B, nc * C, D))
    full[:, :L] = b
    h = full.unflatten(1, (nc, C))
    P = a.clone()
    for t in range(1, C):
        h[:, :, t] += a[:, :, t] * h[:, :, t - 1]
        P[:, :, t] *= P[:, :, t - 1]
    start = torch.empty((B, nc, D), device=a.device, dtype=a.dtype)
    at = h0
    for k in range(nc):
        start[:, k] = at
        at = P[:, k, -1] * at + h[:, k, -1]
    h += P * start[:, :, None]
    return h.flatten(1, 2)[:, :L]


def _glr_parts(s, w):
    """Decay, input scale and the two gates of every token, with the exponent of the decay."""
    r, i, lam = _sigmoid(s["rgate"].to(w)), _sigmoid(s["igate"].to(w)), s["lam"].to(w)
    rate = RATE * (torch.clamp(lam, min=0) + torch.log1p(torch.exp(-lam.abs())))
    e = rate * r
    a, m = torch.exp(-e), torch.sqrt(-torch.expm1(-2 * e))
    if s["reset"] is not None:
        first = s["reset"][..., None]
        a, m = torch.where(first, 0.0, a), torch.where(first, 1.0, m)
    return a, m, r, i, e


def _glr_plain(s, c):
    w = torch.float32
    t = s["x"].dtype
    a, m, r, i, e = _glr_parts(s, w)
    x = s["x"].to(w)
    h0 = s["h0"].to(w) if s["h0"] is not None else x.new_zeros((c["batch"], c["dim"]))
    gate = s["gate"].to(w) if s["gate"] is not None else None
    if c["op"] == "glr_step":
        h = a * h0 + m * i * x
        return dict(y=(h * gate if gate is not None else h).to(t), h=h)
    h = _runs(a, m * i * x, h0)
    out = dict(y=(h * gate if gate is not None else h).to(t), h_last=h[:, -1].clone())
    if c["op"] == "glr_fwd":
        return out
    dy = s["dy"].to(w)
    if gate is not None:
        out["dgate"] = (dy * h).to(t)
        dy = dy * gate
    dy[:, -1] += s["dh_last"].to(w)
    # the reverse recurrence g_t = dy_t + a_{t+1} g_{t+1}
    after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    g = _runs(after.flip(1), dy.flip(1), torch.zeros_like(h0)).flip(1)
    before = torch.cat([h0[:, None], h[:, :-1]], 1)
    # d/d exponent of decay and scale, times the exponent
    de = g * a * e * (a * i * x / torch.clamp(m, min=1e-30) - before)
    gm = g * m
    out["dx"] = (gm * i).to(t)
    out["digate"] = (gm * x * i * (1 - i)).to(t)
    out["drgate"] = (de * (1 - r)).to(t)
    lam = s["lam"]
    softplus = torch.clamp(lam, min=0) + torch.log1p(torch.exp(-lam.abs()))
    out["dlam"] = (de.sum((0, 1), dtype=torch.float64) * (_sigmoid(lam) / softplus)).to(w)
    if s["h0"] is not None:
        out["dh0"] = a[:, 0] * g[:, 0]
    return out


# --------------------------------------------- the projection in its plain form
def _act(z, act):
    if act == "silu":
        return z * _sigmoid(z)
    if act == "gelu":
        return z * _sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
    return _sigmoid(z) if act == "sigmoid" else z


def _dact(z, act):
    if act == "silu":
        s = _sigmoid(z)
        return s * (1 + z * (1 - s))
    if act == "gelu":
        k = 2 * math.sqrt(2 / math.pi)
        s = _sigmoid(k * (z + 0.044715 * z * z * z))
        return s + z * s * (1 - s) * k * (1 + 3 * 0.044715 * z * z)
    s = _sigmoid(z)
    return s * (1 - s)


def _by_group(t, G, mat=False):
    """(G, rows, width) of (rows, width) or (rows, G, width); weights keep their order."""
    if mat:
        return t if G > 1 else t[None]
    return t.transpose(0, 1).contiguous() if G > 1 else t[None]


def _proj_plain(s, c):
    w, G, t = torch.float32, c["groups"], s["x"].dtype
    back = (lambda v: v.transpose(0, 1).contiguous()) if G > 1 else (lambda v: v[0])
    x, weight = _by_group(s["x"].to(w), G), _by_group(s["weight"].to(w), G, True)
    if c["op"] == "proj_fwd":
        z = back(torch.matmul(x, weight.transpose(1, 2).contiguous()))
        if s["bias"] is not None:
            z = z + s["bias"]
        y = _act(z, c["act"])
        if s["residual"] is not None:
            y = y + s["residual"].to(w)
        out = dict(y=y.to(t if s["residual"] is None else s["residual"].dtype))
        if c["save"] and c["act"] != "none":
            out["pre"] = z.to(t)
        return out
    dz = s["dy"].to(w)
    if c["act"] != "none":
        dz = dz * _dact(s["pre"].to(w), c["act"])
    out = dict(dpre=dz.to(t))
    if s["bias"] is not None:
        out["dbias"] = dz.sum(0, dtype=torch.float64).to(w)
    dz = _by_group(out["dpre"].to(w), G)
    out["dx"] = back(torch.matmul(dz, weight)).to(t)
    dw = torch.matmul(dz.transpose(1, 2).contiguous(), x)
    out["dweight"] = (dw if G > 1 else dw[0]).to(t)
    return out


# ----------------------------------------------- the clipping in its plain form
def _clip_plain(s, c):
    total = torch.zeros((), device="cuda", dtype=torch.float64)
    for g in s["grads"]:
        g = g.to(torch.float32)
        total = total + (g * g).sum(dtype=torch.float64)
    norm = torch.sqrt(total)
    coef = torch.clamp(c["max_norm"] / (norm + CLIP_EPS), max=1.0).to(torch.float32)
    for g, o in zip(s["grads"], s["out"]):
        o.copy_(g.to(torch.float32) * coef)
    return dict(norm=norm.to(torch.float32), narrow=s["flat"][0], wide=s["flat"][1])


# ------------------------------------------------------------------- one pass
def _own_glr(s, c):
    import selective_state_space_78_amd as ssm
    ins = (s["x"], s["rgate"], s["igate"], s["lam"])
    opts = dict(gate=s["gate"], reset=s["reset"], rate=RATE)
    if c["op"] == "glr_step":
        return dict(y=ssm.ssm_glr_state_update(*ins, s["h0"], h_out=s["h_out"], **opts), h=s["h_out"])
    if c["op"] == "glr_fwd":
        y, h_last = ssm.ssm_glr_fwd(*ins, h0=s["h0"], **opts)
        return dict(y=y, h_last=h_last)
    y, h_last, saved = ssm.ssm_glr_fwd_save(*ins, h0=s["h0"], **opts)
    g = ssm.ssm_glr_bwd_saved(*ins, s["dy"], saved, h0=s["h0"], dh_last=s["dh_last"], want_dh0=s["h0"] is not None, **opts)
    if s["gate"] is None and s["dy"].dtype == torch.float32:
        # the plain form adds dh_last to the last token's dy where it is kept: a further pass on the same state goes
        # on from there, on both sides
        s["dy"][:, -1] += s["dh_last"]
    out = dict(y=y, h_last=h_last)
    out.update({n: v for n, v in g.items() if v is not None})
    return out


def _own_proj(s, c):
    import selective_state_space_78_amd as ssm
    act = None if c["act"] == "none" else c["act"]
    ins = (s["x"], s["weight"])
    if c["op"] == "proj_fwd":
        opts = dict(bias=s["bias"], activation=act, residual=s["residual"])
        if c["save"] and act is not None:
            y, pre = ssm.ssm_proj_fwd_save(*ins, **opts)
            return dict(y=y, pre=pre)
        return dict(y=ssm.ssm_proj_fwd(*ins, **opts))
    g = ssm.ssm_proj_bwd(s["dy"], *ins, pre=s["pre"], activation=act, want_dbias=s["bias"] is not None)
    return {n: v for n, v in g.items() if v is not None}


def run(state):
    c = state["case"]
    if c["op"].startswith("glr"):
        return _own_glr(state, c) if own else _glr_plain(state, c)
    if c["op"].startswith("proj"):
        return _own_proj(state, c) if own else _proj_plain(state, c)
    if not own:
        return _clip_plain(state, c)
    import selective_state_space_78_amd as ssm
    norm = ssm.ssm_grad_clip(state["grads"], c["max_norm"], eps=CLIP_EPS, out=state["out"])
    return dict(norm=norm, narrow=state["flat"][0], wide=state["flat"][1])


# --------------------------------------------------- the definitions in 64 bits
def _exact_glr(c, s):
    d = torch.float64
    train = c["op"] == "glr_train"
    x, rg, ig, lam = (s[n].to(d).requires_grad_(train) for n in ("x", "rgate", "igate", "lam"))
    h = s["h0"].to(d) if s["h0"] is not None else torch.zeros((c["batch"], c["dim"]), dtype=d, device="cuda")
    log_a = -RATE * torch.nn.functional.softplus(lam, threshold=60) * torch.sigmoid(rg)
    a, m = torch.exp(log_a), torch.sqrt(-torch.expm1(2 * log_a))
    if s["reset"] is not None:
        keep = 1 - s["reset"][..., None].to(d)
        a, m = a * keep, m * keep + (1 - keep)
    b = m * torch.sigmoid(ig) * x
    gate = s["gate"].to(d) if s["gate"] is not None else 1.0
    if c["op"] == "glr_step":
        h = a * h + b
        return dict(y=h * gate, h=h)
    L = c["L"]
    av, bv = a.detach(), b.detach()
    first, every = h, torch.empty_like(bv)
    for t in range(L):
        h = torch.addcmul(bv[:, t], av[:, t], h)
        every[:, t] = h
    out = dict(y=every * gate, h_last=h)
    if not train:
        return out
    up = s["dy"].to(d) * gate
    D, got = s["dh_last"].to(d), torch.empty_like(bv)
    for t in range(L - 1, -1, -1):
        D = D + up[:, t]
        got[:, t] = D
        D = D * av[:, t]
    before = torch.cat([first[:, None], every[:, :-1]], 1)
    grads = torch.autograd.grad((a * (got * before) + b * got).sum(), (x, rg, ig, lam))
    out.update(zip(("dx", "drgate", "digate", "dlam"), grads))
    if s["gate"] is not None:
        out["dgate"] = s["dy"].to(d) * every
    if s["h0"] is not None:
        out["dh0"] = D
    return out


def _exact_proj(c, s):
    d, t = torch.float64, s["x"].dtype
    G, M, K, N = c["groups"], c["rows"], c["K"], c["N"]
    x, weight = s["x"].reshape(M, G, K).to(d), s["weight"].reshape(G, N, K).to(d)
    lead = (M,) if G == 1 else (M, G)

    def act(v):
        if c["act"] == "silu":
            return torch.nn.functional.silu(v)
        if c["act"] == "gelu":
            return torch.nn.functional.gelu(v, approximate="tanh")
        return torch.sigmoid(v) if c["act"] == "sigmoid" else v

    if c["op"] == "proj_fwd":
        z = torch.stack([torch.mm(x[:, g], weight[g].t()) for g in range(G)], 1)
        if s["bias"] is not None:
            z = z + s["bias"].reshape(G, N).to(d)
        y = act(z).reshape(*lead, N)
        if s["residual"] is not None:
            y = y + s["residual"].to(d)
        return dict(y=y, pre=z.reshape(*lead, N)) if c["save"] and c["act"] != "none" else dict(y=y)
    dz = s["dy"].reshape(M, G, N).to(d)
    if c["act"] != "none":
        leaf = s["pre"].reshape(M, G, N).to(d).requires_grad_()
        dz = torch.autograd.grad((act(leaf) * dz).sum(), leaf)[0]
    out = dict(dpre=dz.reshape(*lead, N))
    if s["bias"] is not None:
        out["dbias"] = dz.sum(0).reshape(s["bias"].shape)
    dz = dz.to(t).to(d)
    out["dx"] = torch.stack([torch.mm(dz[:, g], weight[g]) for g in range(G)], 1).reshape(*lead, K)
    out["dweight"] = torch.stack([torch.mm(dz[:, g].t(), x[:, g]) for g in range(G)]).reshape(s["weight"].shape)
    return out


def _exact_clip(c, s):
    norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(g.double()) for g in s["grads"]]))
    coef = min(1.0, c["max_norm"] / (float(norm) + CLIP_EPS))
    buckets = [f.double() for f in s["flat"]]
    for g, o in zip(s["grads"], s["out"]):
        k = 0 if o.untyped_storage().data_ptr() == s["flat"][0].untyped_storage().data_ptr() else 1
        at = o.storage_offset()
        buckets[k][at:at + o.numel()] = g.reshape(-1).double() * coef
    return dict(norm=norm, narrow=buckets[0], wide=buckets[1])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return _exact_glr(case, s) if op.startswith("glr") else _exact_proj(case, s) if op.startswith("proj") else \
        _exact_clip(case, s)
