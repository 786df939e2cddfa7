"""Refusals of the gated linear recurrence, the projections and the gradient clipping,
on the host: every call below fails its checks before touching a device, so the
addresses it passes are never read. Then the binding's own checks, and where its
memory comes from, with the launches and streams replaced."""
import ctypes
from array import array

import pytest

import selective_state_space_78_amd as ssm
from test_delta_abi_cpu import EALIAS, EALIGN, EDTYPE, ENULL, ESHAPE, EUNSUP, EWS, GB, L, OK, call, fake  # noqa: F401
from test_stream_memory_cpu import tensors, world  # noqa: F401

torch = pytest.importorskip("torch")
BF, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


# ------------------------------------------------------------ the recurrence
def glr(b=2, n=1000, d=64, dtype=ssm.SSM_BF16, rate=8.0, strides=(0, 0, 0, 0)):
    return ssm.GlrDesc(b, n, d, dtype, rate, *strides)


G_FWD = dict(x=1, rgate=2, igate=3, lam=4, h0=5, gate=6, reset=7, y=8, h_last=9)
G_BWD = dict(x=1, rgate=2, igate=3, lam=4, h0=5, gate=6, reset=7, dy=8, dh_last=9, dx=10, drgate=11, digate=12, dgate=13,
             dlam=14, dh0=15)
G_STEP = dict(x=1, rgate=2, igate=3, lam=4, gate=5, reset=6, h=7, h_out=8, y=9)


def glr_calls(L):
    return ((L.ssm_glr_fwd, G_FWD), (L.ssm_glr_fwd_save, G_FWD), (L.ssm_glr_bwd, G_BWD), (L.ssm_glr_bwd_saved, G_BWD))


def test_glr_descriptor(L):
    for fn, args in glr_calls(L):
        assert call(fn, None, args) == ENULL
        for kw, want in ((dict(b=-1), ESHAPE), (dict(n=-1), ESHAPE), (dict(d=0), ESHAPE), (dict(d=1 << 24), ESHAPE),
                         (dict(strides=(63, 0, 0, 0)), ESHAPE), (dict(strides=(0, -1, 0, 0)), ESHAPE),
                         (dict(strides=(0, 0, 1 << 24, 0)), ESHAPE), (dict(strides=(0, 0, 0, 63)), ESHAPE),
                         (dict(dtype=2), EDTYPE), (dict(rate=-1.0), EUNSUP), (dict(rate=NAN), EUNSUP),
                         (dict(rate=INF), EUNSUP), (dict(b=1 << 40, n=1 << 40), ESHAPE), (dict(b=1 << 31, n=1), ESHAPE),
                         (dict(n=1 << 38), ESHAPE),
                         # 2^32 work items: tiles of 32 channels, chunks of 64 tokens
                         (dict(b=1 << 10, n=1 << 16, d=1 << 10), ESHAPE)):
            assert call(fn, glr(**kw), args) == want, kw
    assert call(L.ssm_glr_state_update, glr(n=2), G_STEP, ws=None) == ESHAPE


def test_glr_pointers(L):
    for n in ("x", "rgate", "igate", "lam", "y"):
        assert call(L.ssm_glr_fwd, glr(), G_FWD, **{n: 0}) == ENULL, n
    for n in ("x", "rgate", "igate", "lam", "dy", "dx", "drgate", "digate", "dgate", "dlam"):
        assert call(L.ssm_glr_bwd, glr(), G_BWD, **{n: 0}) == ENULL, n
    for n in ("x", "rgate", "igate", "lam", "h", "h_out", "y"):
        assert call(L.ssm_glr_state_update, glr(n=1), G_STEP, ws=None, **{n: 0}) == ENULL, n
    for n, off in (("x", 1), ("rgate", 1), ("igate", 1), ("gate", 1), ("lam", 2), ("h0", 2), ("h_last", 2), ("y", 1)):
        assert call(L.ssm_glr_fwd, glr(), G_FWD, **{n: G_FWD[n] * GB + off}) == EALIGN, n
    for n, off in (("dy", 1), ("dx", 1), ("drgate", 1), ("digate", 1), ("dgate", 1), ("dlam", 2), ("dh0", 2), ("dh_last", 2)):
        assert call(L.ssm_glr_bwd, glr(), G_BWD, **{n: G_BWD[n] * GB + off}) == EALIGN, n
    for n, off in (("x", 1), ("h", 2), ("h_out", 2), ("lam", 2), ("y", 1)):
        assert call(L.ssm_glr_state_update, glr(n=1), G_STEP, ws=None, **{n: G_STEP[n] * GB + off}) == EALIGN, n


def test_glr_overlaps(L):
    for n in ("x", "rgate", "igate", "lam", "gate", "reset", "h0"):
        assert call(L.ssm_glr_fwd, glr(), G_FWD, y=G_FWD[n] * GB) == EALIAS, n
        if n != "h0":
            assert call(L.ssm_glr_fwd, glr(), G_FWD, h_last=G_FWD[n] * GB) == EALIAS, n
    assert call(L.ssm_glr_fwd, glr(), G_FWD, h_last=5 * GB + 4) == EALIAS         # h0, but not exactly
    assert call(L.ssm_glr_fwd, glr(), G_FWD, y=20 * GB) == EALIAS                 # the workspace
    assert call(L.ssm_glr_fwd, glr(), G_FWD, y=9 * GB) == EALIAS
    out = ("dx", "drgate", "digate", "dgate", "dlam", "dh0")
    for n in out:
        for other in [m for m in G_BWD if m != n and not (n == "dh0" and m == "dh_last")]:
            assert call(L.ssm_glr_bwd, glr(), G_BWD, **{n: G_BWD[other] * GB}) == EALIAS, (n, other)
        assert call(L.ssm_glr_bwd, glr(), G_BWD, **{n: 20 * GB}) == EALIAS, n
    assert call(L.ssm_glr_bwd, glr(), G_BWD, dh0=9 * GB + 4) == EALIAS
    for n in ("x", "rgate", "igate", "lam", "gate", "reset"):
        assert call(L.ssm_glr_state_update, glr(n=1), G_STEP, ws=None, h_out=G_STEP[n] * GB) == EALIAS, n
    assert call(L.ssm_glr_state_update, glr(n=1), G_STEP, ws=None, y=7 * GB) == EALIAS
    assert call(L.ssm_glr_state_update, glr(n=1), G_STEP, ws=None, h_out=7 * GB + 4) == EALIAS


def test_glr_workspace_and_empty(L):
    for fn, args in glr_calls(L):
        assert call(fn, glr(), args, ws=0) == EWS
        assert call(fn, glr(), args, ws_bytes=64) == EWS
        assert call(fn, glr(), args, ws=20 * GB + 128) == EALIGN
    size, back = (lambda **k: L.ssm_glr_workspace_size(ctypes.byref(glr(**k)))), (lambda **k: L.ssm_glr_bwd_workspace_size(ctypes.byref(glr(**k))))
    assert size(n=128) == 0 and size(n=129) > 0 and size(n=0) == 0 and size(b=0) == 0 and size(d=0) == 0
    assert back(n=1) > 0 and back(n=0) == 0 and back() > size()
    assert call(L.ssm_glr_fwd, glr(b=0), G_FWD) == OK
    assert call(L.ssm_glr_fwd, glr(n=0), G_FWD, h_last=5 * GB) == OK              # h0 in place: nothing to do
    assert call(L.ssm_glr_fwd, glr(n=0), G_FWD, h_last=0) == OK
    assert call(L.ssm_glr_bwd, glr(n=0), G_BWD, dlam=0) == ENULL
    assert call(L.ssm_glr_state_update, glr(b=0, n=1), G_STEP, ws=None) == OK


# ------------------------------------------------------------- the projection
def proj(rows=100, g=1, k=64, n=32, dtype=ssm.SSM_BF16, yt=ssm.SSM_BF16, act=0, reserved=0, xs=0):
    return ssm.ProjDesc(rows, g, k, n, dtype, yt, act, reserved, xs)


P_FWD = dict(x=1, weight=2, bias=3, residual=4, pre=5, y=6)
P_BWD = dict(dy=1, x=2, weight=3, pre=4, dpre=5, dx=6, dweight=7, dbias=8)


def test_proj_descriptor(L):
    for fn, args in ((L.ssm_proj_fwd, P_FWD), (L.ssm_proj_bwd, P_BWD)):
        assert call(fn, None, args) == ENULL
        for kw, want in ((dict(rows=-1), ESHAPE), (dict(g=0), ESHAPE), (dict(k=0), ESHAPE), (dict(n=0), ESHAPE),
                         (dict(k=1 << 22), ESHAPE), (dict(g=1 << 12, n=1 << 10), ESHAPE), (dict(xs=63), ESHAPE),
                         (dict(xs=-1), ESHAPE), (dict(xs=1 << 22), ESHAPE), (dict(rows=1 << 31), ESHAPE),
                         (dict(rows=1 << 30, k=1 << 20), ESHAPE), (dict(dtype=3), EDTYPE), (dict(yt=-1), EDTYPE),
                         (dict(dtype=ssm.SSM_F32, yt=ssm.SSM_BF16), EUNSUP), (dict(act=4), EUNSUP), (dict(act=-1), EUNSUP),
                         (dict(reserved=1), EUNSUP)):
            assert call(fn, proj(**kw), args) == want, kw


def test_proj_pointers(L):
    for n in ("x", "weight", "y"):
        assert call(L.ssm_proj_fwd, proj(), P_FWD, **{n: 0}) == ENULL, n
    assert call(L.ssm_proj_bwd, proj(), P_BWD, dy=0) == ENULL
    assert call(L.ssm_proj_bwd, proj(), P_BWD, x=0) == ENULL                      # dweight reads x
    assert call(L.ssm_proj_bwd, proj(), P_BWD, weight=0) == ENULL                 # dx reads the weight
    assert call(L.ssm_proj_bwd, proj(act=1), P_BWD, pre=0) == ENULL
    assert call(L.ssm_proj_bwd, proj(act=1), P_BWD, dpre=0) == ENULL
    assert call(L.ssm_proj_bwd, proj(yt=ssm.SSM_F32), P_BWD, dpre=0) == ENULL
    for n, off in (("x", 1), ("weight", 1), ("bias", 2), ("residual", 1), ("pre", 1), ("y", 1)):
        assert call(L.ssm_proj_fwd, proj(), P_FWD, **{n: P_FWD[n] * GB + off}) == EALIGN, n
    assert call(L.ssm_proj_fwd, proj(yt=ssm.SSM_F32), P_FWD, y=6 * GB + 2) == EALIGN
    for n, off in (("dy", 1), ("x", 1), ("weight", 1), ("dx", 1), ("dweight", 1), ("dbias", 2)):
        assert call(L.ssm_proj_bwd, proj(), P_BWD, **{n: P_BWD[n] * GB + off}) == EALIGN, n
    for n in ("pre", "dpre"):
        assert call(L.ssm_proj_bwd, proj(act=2), P_BWD, **{n: P_BWD[n] * GB + 1}) == EALIGN, n


def test_proj_overlaps_and_workspace(L):
    for n in ("x", "weight", "bias"):
        assert call(L.ssm_proj_fwd, proj(), P_FWD, y=P_FWD[n] * GB) == EALIAS, n
        assert call(L.ssm_proj_fwd, proj(), P_FWD, pre=P_FWD[n] * GB) == EALIAS, n
    assert call(L.ssm_proj_fwd, proj(), P_FWD, y=4 * GB + 2) == EALIAS            # the residual, but not exactly
    assert call(L.ssm_proj_fwd, proj(), P_FWD, pre=4 * GB) == EALIAS and call(L.ssm_proj_fwd, proj(), P_FWD, pre=6 * GB) == EALIAS
    for n in ("dpre", "dx", "dweight", "dbias"):
        for other in [m for m in P_BWD if m != n]:
            assert call(L.ssm_proj_bwd, proj(act=1), P_BWD, **{n: P_BWD[other] * GB}) == EALIAS, (n, other)
        assert call(L.ssm_proj_bwd, proj(act=1), P_BWD, **{n: 20 * GB}) == EALIAS, n
    for kw in (dict(ws=0), dict(ws_bytes=128)):
        assert call(L.ssm_proj_bwd, proj(), P_BWD, **kw) == EWS
    assert call(L.ssm_proj_bwd, proj(), P_BWD, ws=20 * GB + 16) == EALIGN
    long = proj(rows=40, k=1 << 16, n=64)      # few tiles, a long reduction: splits
    size = L.ssm_proj_workspace_size(ctypes.byref(long))
    assert size > 0 and call(L.ssm_proj_fwd, long, P_FWD, ws_bytes=size - 1) == EWS
    assert call(L.ssm_proj_fwd, long, P_FWD, y=20 * GB) == EALIAS
    # few rows: without tiles, unless the weight's rows are long
    few, more = proj(rows=8, k=1 << 12, n=1 << 12), proj(rows=8, k=1 << 16, n=64)
    assert L.ssm_proj_workspace_size(ctypes.byref(few)) == 0
    size = L.ssm_proj_workspace_size(ctypes.byref(more))
    assert size > 0 and call(L.ssm_proj_fwd, more, P_FWD, ws_bytes=size - 1) == EWS
    assert call(L.ssm_proj_fwd, proj(rows=0), P_FWD) == OK


def test_proj_sizes_serve_any_stride(L, world):
    """The binding's sizes without a stride serve x of any, those with one are that descriptor's. A call whose outputs
    overlap gets past the check of its workspace and no further."""
    grown = 0
    for rows, g, k, n in ((4100, 1, 1032, 1030), (4100, 1, 1032, 1031), (4100, 1, 1031, 1030), (4096, 2, 258, 516), (300, 1, 1032, 1030),
                          (8, 1, 4096, 4096), (100000, 1, 6, 4096), (16384, 2, 257, 515)):
        for dtype in (ssm.SSM_BF16, ssm.SSM_F32):
            fwd, bwd = ssm.ssm_proj_workspace_size(rows, k, n, g, dtype), ssm.ssm_proj_bwd_workspace_size(rows, k, n, g, dtype)
            for xs in (0, g * k, g * k + 1, g * k + 6, g * k + 7):
                d = proj(rows, g, k, n, dtype, dtype, xs=xs)
                one, two = L.ssm_proj_workspace_size(ctypes.byref(d)), L.ssm_proj_bwd_workspace_size(ctypes.byref(d))
                assert one <= fwd and two <= bwd, (rows, g, k, n, xs)
                assert one == ssm.ssm_proj_workspace_size(rows, k, n, g, dtype, x_stride=xs)
                assert two == ssm.ssm_proj_bwd_workspace_size(rows, k, n, g, dtype, x_stride=xs)
                grown += one < fwd
                far = dict(zip(P_FWD, (k * GB << 10 for k in (1, 2, 3, 4, 5, 6))))
                assert call(L.ssm_proj_fwd, d, P_FWD, ws=1 << 50, ws_bytes=fwd, **dict(far, y=far["x"])) == EALIAS
                back = dict(zip(P_BWD, (k * GB << 10 for k in range(1, 9))))
                assert call(L.ssm_proj_bwd, d, P_BWD, ws=1 << 50, ws_bytes=bwd, **dict(back, dx=back["x"])) == EALIAS
    assert grown
    x, w = z(4100, 1039, dtype=BF)[:, :1032], z(1030, 1032, dtype=BF)
    room = lambda n: torch.zeros(n, dtype=torch.uint8)
    ssm.ssm_proj_fwd(x, w, workspace=room(ssm.ssm_proj_workspace_size(4100, 1032, 1030)))
    ssm.ssm_proj_bwd(z(4100, 1030, dtype=BF), x, w, workspace=room(ssm.ssm_proj_bwd_workspace_size(4100, 1032, 1030)))


def test_proj_copies_where_they_help(L):
    """Rows shorter than one 16-byte piece go through registers, padded or not: nothing of such a product is copied."""
    fwd = lambda *a, **k: L.ssm_proj_workspace_size(ctypes.byref(proj(*a, **k)))
    bwd = lambda *a, **k: L.ssm_proj_bwd_workspace_size(ctypes.byref(proj(*a, **k)))
    for rows, n in ((100000, 4096), (200000, 2048)):
        for k in (1, 3, 5, 7):
            assert fwd(rows, 1, k, n) == 0, (rows, k, n)
            # no more than the slabs' and the splits' sums, which its even neighbour has as well
            assert bwd(rows, 1, k, n) <= bwd(rows, 1, k + 1, n), (rows, k, n)
        assert fwd(rows, 1, 6, n, xs=9) == 0 and bwd(rows, 1, 6, n, xs=9) == bwd(rows, 1, 6, n)
    for k in (512, 4096):
        for n in (1, 3, 5, 7):
            assert bwd(50000, 1, k, n) <= bwd(50000, 1, k, n + 1), (k, n)
    # rows of a piece and more are copied
    assert fwd(100000, 1, 9, 4096) > 100000 * 32 and bwd(50000, 1, 513, 515) > 50000 * 2 * 1040


# ---------------------------------------------------------------- the clipping
def arrays(n, at=1, size=1000, dtype=ssm.SSM_F32):
    return (array("Q", [(at + k) * GB for k in range(n)]), array("q", [size] * n), array("i", [dtype] * n))


def address(a):
    return a.buffer_info()[0]


def clip(L, p, s, t, o=None, count=None, norm=40 * GB, ws=50 * GB, ws_bytes=1 << 20, max_norm=1.0, eps=1e-6, fn="ssm_grad_clip"):
    count = len(p) if count is None else count
    o = p if o is None else o
    if fn == "ssm_grad_norm":
        return L.ssm_grad_norm(count, address(p), address(s), address(t), norm, ws, ws_bytes, None)
    if fn == "ssm_grad_scale":
        return L.ssm_grad_scale(count, address(p), address(o), address(s), address(t), norm, max_norm, eps, None)
    return L.ssm_grad_clip(count, address(p), address(o), address(s), address(t), max_norm, eps, norm, ws, ws_bytes, None)


def test_grad_arguments(L):
    p, s, t = arrays(3)
    for fn in ("ssm_grad_clip", "ssm_grad_norm", "ssm_grad_scale"):
        assert clip(L, p, s, t, count=-1, fn=fn) == ESHAPE
        assert clip(L, p, s, t, count=(1 << 20) + 1, fn=fn) == ESHAPE
        assert clip(L, p, array("q", [1, -1, 1]), t, fn=fn) == ESHAPE
        assert clip(L, p, array("q", [1, (1 << 35) + 1, 1]), t, fn=fn) == ESHAPE
        assert clip(L, p, s, array("i", [0, 2, 0]), fn=fn) == EDTYPE
        assert clip(L, array("Q", [GB, 0, 3 * GB]), s, t, fn=fn) == ENULL
        assert clip(L, array("Q", [GB, 2 * GB + 2, 3 * GB]), s, t, fn=fn) == EALIGN
        assert clip(L, p, s, t, norm=0, fn=fn) == ENULL
        assert clip(L, p, s, t, norm=40 * GB + 2, fn=fn) == EALIGN
        if fn != "ssm_grad_scale":
            assert clip(L, p, s, t, ws=0, fn=fn) == EWS and clip(L, p, s, t, ws_bytes=16, fn=fn) == EWS
            assert clip(L, p, s, t, ws=50 * GB + 8, fn=fn) == EALIGN
        if fn != "ssm_grad_norm":
            for kw in (dict(max_norm=-1.0), dict(max_norm=NAN), dict(max_norm=INF), dict(eps=-1.0), dict(eps=NAN)):
                assert clip(L, p, s, t, fn=fn, **kw) == EUNSUP, kw
            assert clip(L, p, s, t, o=array("Q", [GB, 0, 3 * GB]), fn=fn) == ENULL
            assert clip(L, p, s, t, o=array("Q", [GB, 2 * GB, 3 * GB + 2]), fn=fn) == EALIGN
    assert L.ssm_grad_clip(2, address(p), None, address(s), address(t), 1.0, 0.0, 40 * GB, 50 * GB, 1 << 20, None) == ENULL
    assert L.ssm_grad_clip(2, None, address(p), address(s), address(t), 1.0, 0.0, 40 * GB, 50 * GB, 1 << 20, None) == ENULL
    assert clip(L, p, s, t, count=0, fn="ssm_grad_scale") == OK
    assert L.ssm_grad_workspace_size(0) == 0 and 0 < L.ssm_grad_workspace_size(128) < L.ssm_grad_workspace_size(129)


def test_grad_overlaps(L):
    p, s, t = arrays(4)
    for fn in ("ssm_grad_clip", "ssm_grad_scale"):
        go = lambda q, o=None: clip(L, array("Q", q), s, t, o=None if o is None else array("Q", o), fn=fn)
        assert go([GB, 2 * GB, 3 * GB, GB]) == EALIAS                    # the same tensor twice
        assert go([GB, 2 * GB, 3 * GB, GB + 3996]) == EALIAS             # its last element
        assert go([GB, 2 * GB, 3 * GB, 4 * GB], [5 * GB, 6 * GB, 7 * GB, 5 * GB]) == EALIAS
        assert go([GB, 2 * GB, 3 * GB, 4 * GB], [5 * GB, 6 * GB, 7 * GB, 2 * GB]) == EALIAS    # another's gradient
        assert go([GB, 2 * GB, 3 * GB, 4 * GB], [GB + 4, 6 * GB, 7 * GB, 8 * GB]) == EALIAS    # its own, moved
        assert clip(L, p, s, t, norm=2 * GB + 8, fn=fn) == EALIAS
        # a large range that holds a small one further on
        assert clip(L, array("Q", [GB, 3 * GB, 2 * GB, 4 * GB]), array("q", [1 << 30, 10, 10, 10]), t, fn=fn) == EALIAS
    assert clip(L, p, s, t, ws=2 * GB) == EALIAS
    assert clip(L, p, s, t, ws=2 * GB, fn="ssm_grad_norm") == EALIAS and clip(L, p, s, t, norm=50 * GB, fn="ssm_grad_norm") == EALIAS


# ----------------------------------------------------------------- the binding
def z(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refusals():
    x, lam = z(2, 5, 8, dtype=BF), z(8)
    step = x[:, 0].contiguous()
    fails = [
        (ValueError, lambda: ssm.ssm_glr_fwd(step, step, step, lam)),
        (ValueError, lambda: ssm.ssm_glr_fwd(x, x[:, :4], x, lam)),
        (TypeError, lambda: ssm.ssm_glr_fwd(x, x.float(), x, lam)),
        (TypeError, lambda: ssm.ssm_glr_fwd(x.half(), x.half(), x.half(), lam)),
        (ValueError, lambda: ssm.ssm_glr_fwd(x, x, x, z(7))),
        (TypeError, lambda: ssm.ssm_glr_fwd(x, x, x, lam.to(BF))),
        (TypeError, lambda: ssm.ssm_glr_fwd(x, x, x, lam, reset=z(2, 5))),
        (ValueError, lambda: ssm.ssm_glr_fwd(x, x, x, lam, reset=z(2, 4).bool())),
        (ValueError, lambda: ssm.ssm_glr_fwd(x, x, x, lam, h0=z(8))),
        (ValueError, lambda: ssm.ssm_glr_fwd(x.transpose(1, 2), x.transpose(1, 2), x.transpose(1, 2), z(5))),
        (ValueError, lambda: ssm.ssm_glr_bwd(x, x, x, lam, x[:, :4])),
        (ValueError, lambda: ssm.ssm_glr_bwd_saved(x, x, x, lam, x, None)),
        (ValueError, lambda: ssm.ssm_glr_state_update(x, x, x, lam, z(2, 8))),
        (ValueError, lambda: ssm.ssm_glr_state_update(step, step, step, lam, z(2, 9))),
        (ValueError, lambda: ssm.ssm_proj_fwd(x, z(4, 7, dtype=BF))),
        (TypeError, lambda: ssm.ssm_proj_fwd(x, z(4, 8))),
        (ValueError, lambda: ssm.ssm_proj_fwd(x, z(8, dtype=BF))),
        (ValueError, lambda: ssm.ssm_proj_fwd(x, z(4, 8, dtype=BF), activation="tanh")),
        (ValueError, lambda: ssm.ssm_proj_fwd(x, z(4, 8, dtype=BF), bias=z(5))),
        (ValueError, lambda: ssm.ssm_proj_fwd(x, z(4, 8, dtype=BF), residual=z(2, 5, 5))),
        (TypeError, lambda: ssm.ssm_proj_fwd(x.float(), z(4, 8), residual=z(2, 5, 4, dtype=BF))),
        (ValueError, lambda: ssm.ssm_proj_fwd(x, z(3, 4, 8, dtype=BF))),
        (ValueError, lambda: ssm.ssm_proj_fwd(x, z(8, 4, dtype=BF).t())),
        (ValueError, lambda: ssm.ssm_proj_bwd(z(2, 5, 4, dtype=BF), x, z(4, 8, dtype=BF), activation="silu")),
        (ValueError, lambda: ssm.ssm_proj_bwd(z(2, 5, 3, dtype=BF), x, z(4, 8, dtype=BF))),
        (ValueError, lambda: ssm.ssm_grad_clip([], 1.0)),
        (TypeError, lambda: ssm.ssm_grad_clip([z(3).half()], 1.0)),
        (ValueError, lambda: ssm.ssm_grad_clip([z(3, 4).t()], 1.0)),
        (ValueError, lambda: ssm.ssm_grad_clip([z(3)], 1.0, out=[])),
        (ValueError, lambda: ssm.ssm_grad_clip([z(3)], 1.0, out=[None])),
        (ValueError, lambda: ssm.ssm_grad_clip([z(3)], 1.0, out=[z(4)])),
        (ValueError, lambda: ssm.ssm_grad_clip([z(3)], 1.0, out=[z(3, dtype=BF)])),
        (ValueError, lambda: ssm.ssm_grad_norm([z(3)], norm=z(2))),
        (ValueError, lambda: ssm.ssm_grad_norm([z(3), torch.zeros(3, device="meta")])),
        # tensors that are not on a GPU
        (ValueError, lambda: ssm.ssm_glr_fwd(x, x, x, lam)),
        (ValueError, lambda: ssm.ssm_proj_fwd(x, z(4, 8, dtype=BF))),
        (ValueError, lambda: ssm.ssm_grad_norm([z(3)])),
    ]
    for k, (kind, f) in enumerate(fails):
        with pytest.raises(kind):
            f()
            print("not refused:", k)


def recurrence():
    x = z(2, 300, 8, dtype=BF)
    return x, x, x, z(8)


def linear(rows=40):
    return z(rows, 4096, dtype=BF), z(64, 4096, dtype=BF)


CALLS = {
    "glr_fwd": lambda **k: ssm.ssm_glr_fwd(*recurrence(), **k),
    "glr_fwd_save": lambda **k: ssm.ssm_glr_fwd_save(*recurrence(), **k),
    "glr_bwd": lambda **k: ssm.ssm_glr_bwd(*recurrence(), recurrence()[0], gate=recurrence()[0], **k),
    "glr_state_update": lambda **k: ssm.ssm_glr_state_update(*(t[:, 0].contiguous() if t.dim() == 3 else t for t in recurrence()),
                                                             z(2, 8), **k),
    "proj_fwd": lambda **k: ssm.ssm_proj_fwd(*linear(), **k),
    "proj_fwd_few": lambda **k: ssm.ssm_proj_fwd(*linear(1), **k),
    "proj_fwd_save": lambda **k: ssm.ssm_proj_fwd_save(*linear(), **k),
    "proj_bwd": lambda **k: ssm.ssm_proj_bwd(z(40, 64, dtype=BF), *linear(), pre=z(40, 64, dtype=BF), activation="silu",
                                             want_dbias=True, **k),
    "grad_norm": lambda **k: ssm.ssm_grad_norm([z(5), z(6)], **k),
    "grad_clip": lambda **k: ssm.ssm_grad_clip([z(5), z(6)], 1.0, **k),
}


@pytest.mark.parametrize("call_", CALLS.values(), ids=list(CALLS))
def test_memory_of_a_stream_handed_over(world, call_):  # noqa: F811
    given = tensors(call_(stream=world.other))
    assert world.made and all(s is world.other for _, s in world.made)
    assert all(any(t is h and s is world.here for h, s in world.held) for t in given)
    # what the call keeps to itself goes back to that stream alone
    assert len(world.held) == len(given)


@pytest.mark.parametrize("call_", CALLS.values(), ids=list(CALLS))
def test_memory_of_the_current_stream(world, call_):  # noqa: F811
    for k in (dict(), dict(stream=world.here)):
        world.made.clear()
        call_(**k)
        assert world.made and all(s is world.here for _, s in world.made) and not world.held
