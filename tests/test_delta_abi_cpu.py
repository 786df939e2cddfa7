"""Refusals of the gated delta rule and the block norms, on the host: every
call below fails its checks before touching a device, so the addresses it
passes are never read."""
import ctypes
import os

import pytest

import selective_state_space_78_amd as ssm

OK, ENULL, ESHAPE, EDTYPE, EUNSUP, EALIAS, EWS, EALIGN = 0, -1, -2, -3, -4, -5, -6, -8
GB = 1 << 30


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(ssm.LIBRARY):
        pytest.skip("library not built")
    return ssm.lib()


def fake(a):
    return ctypes.c_void_p(a) if a else None


def gdr(b=2, L=100, H=4, P=64, G=2, N=64, dtype=ssm.SSM_BF16, sp=0, sg=0, qn=0, scale=1.0, eps=1e-6, strides=(0,) * 5,
        bias=0):
    return ssm.GdrDesc(b, L, H, P, G, N, dtype, sp, sg, qn, scale, eps, *strides, bias or None)


FWD = dict(q=1, k=2, v=3, dt=4, beta=5, A=6, h0=7, y=8, h_last=9)
BWD = dict(q=1, k=2, v=3, dt=4, beta=5, A=6, h0=7, dy=8, dh_last=9, dq=10, dk=11, dv=12, ddt=13, dbeta=14, dA=15,
           ddt_bias=16, dh0=17)
STEP = dict(q=1, k=2, v=3, dt=4, beta=5, A=6, h=7, h_out=8, y=9)


def call(fn, desc, args, ws=20 * GB, ws_bytes=1 << 33, **over):
    at = {n: v * GB for n, v in args.items()}
    at.update(over)
    a = [ctypes.byref(desc) if desc is not None else None] + [fake(v) for v in at.values()]
    if ws is not None:
        a += [fake(ws), ws_bytes]
    return fn(*a, None)


def test_gdr_descriptor(L):
    for fn, args in ((L.ssm_gdr_fwd, FWD), (L.ssm_gdr_fwd_save, FWD), (L.ssm_gdr_bwd, BWD), (L.ssm_gdr_bwd_saved, BWD)):
        assert call(fn, None, args) == ENULL
        for kw, want in ((dict(b=-1), ESHAPE), (dict(L=-1), ESHAPE), (dict(H=0), ESHAPE), (dict(G=0), ESHAPE),
                         (dict(H=4, G=3), ESHAPE), (dict(dtype=9), EDTYPE), (dict(dtype=ssm.SSM_F32), EUNSUP),
                         (dict(P=8), EUNSUP), (dict(P=72), EUNSUP), (dict(P=272), EUNSUP), (dict(N=96), EUNSUP),
                         (dict(sp=2), EUNSUP), (dict(sg=-1), EUNSUP), (dict(qn=2), EUNSUP),
                         (dict(scale=float("nan")), EUNSUP), (dict(scale=float("inf")), EUNSUP),
                         (dict(qn=1, eps=0.0), EUNSUP), (dict(b=1 << 40, L=1 << 40), ESHAPE),
                         (dict(b=1 << 20, L=1 << 20), ESHAPE),
                         (dict(strides=(127, 0, 0, 0, 0)), ESHAPE),    # rows overlap
                         (dict(strides=(0, 0, 1 << 25, 0, 0)), ESHAPE),  # a chunk's rows past 32-bit offsets
                         (dict(strides=(0, 132, 0, 0, 0)), EALIGN)):
            assert call(fn, gdr(**kw), args) == want, kw


def test_gdr_empty(L):
    assert call(L.ssm_gdr_fwd, gdr(b=0), FWD) == OK
    assert call(L.ssm_gdr_fwd, gdr(L=0), FWD, h_last=0) == OK
    assert call(L.ssm_gdr_fwd, gdr(L=0), FWD, h_last=7 * GB) == OK       # h0 in place: nothing to do
    assert L.ssm_gdr_workspace_size(ctypes.byref(gdr(L=0))) == 0
    assert L.ssm_gdr_workspace_size(ctypes.byref(gdr(P=8))) == 0
    small = L.ssm_gdr_workspace_size(ctypes.byref(gdr()))
    assert 0 < small < L.ssm_gdr_bwd_workspace_size(ctypes.byref(gdr()))


def test_gdr_pointers(L):
    for n in ("q", "k", "v", "dt", "beta", "A", "y"):
        assert call(L.ssm_gdr_fwd, gdr(), FWD, **{n: 0}) == ENULL, n
    for n in ("dy", "dq", "dk", "dv", "ddt", "dbeta", "dA"):
        assert call(L.ssm_gdr_bwd, gdr(), BWD, **{n: 0}) == ENULL, n
    assert call(L.ssm_gdr_bwd, gdr(bias=18 * GB), BWD, ddt_bias=0) == ENULL
    for n, off in (("q", 8), ("k", 8), ("v", 8), ("h0", 8), ("y", 8), ("h_last", 4), ("dt", 1), ("A", 2)):
        assert call(L.ssm_gdr_fwd, gdr(), FWD, **{n: FWD[n] * GB + off}) == EALIGN, n
    for n, off in (("dy", 8), ("dq", 2), ("dk", 8), ("dv", 8), ("ddt", 1), ("dA", 2), ("dh0", 4), ("dh_last", 8)):
        assert call(L.ssm_gdr_bwd, gdr(), BWD, **{n: BWD[n] * GB + off}) == EALIGN, n
    assert call(L.ssm_gdr_fwd, gdr(), FWD, ws=0) == EWS
    need = L.ssm_gdr_workspace_size(ctypes.byref(gdr()))
    assert call(L.ssm_gdr_fwd, gdr(), FWD, ws_bytes=need - 1) == EWS
    assert call(L.ssm_gdr_fwd_save, gdr(), FWD, ws_bytes=need) == EWS
    assert call(L.ssm_gdr_bwd, gdr(), BWD, ws_bytes=need) == EWS
    assert call(L.ssm_gdr_fwd, gdr(), FWD, ws=20 * GB + 128) == EALIGN


def test_gdr_overlaps(L):
    for n in ("q", "k", "v", "dt", "beta", "A", "h0", "h_last"):
        assert call(L.ssm_gdr_fwd, gdr(), FWD, y=FWD[n] * GB) == EALIAS, n
    assert call(L.ssm_gdr_fwd, gdr(), FWD, h_last=7 * GB + 256) == EALIAS     # h0, but not exactly
    assert call(L.ssm_gdr_fwd, gdr(), FWD, ws=3 * GB) == EALIAS
    assert call(L.ssm_gdr_fwd, gdr(), FWD, ws=8 * GB) == EALIAS
    # q cut out of wider rows: what lies between its rows counts as its range
    assert call(L.ssm_gdr_fwd, gdr(strides=(1024, 0, 0, 0, 0)), FWD, y=1 * GB + 2048 * 50 + 512) == EALIAS
    for n in ("q", "dy", "dk", "dv", "ddt", "dA", "dh0", "dh_last"):
        assert call(L.ssm_gdr_bwd, gdr(), BWD, dq=BWD[n] * GB) == EALIAS, n
    assert call(L.ssm_gdr_bwd, gdr(), BWD, dh0=9 * GB + 256) == EALIAS
    assert call(L.ssm_gdr_bwd, gdr(), BWD, ws=8 * GB) == EALIAS


def test_gdr_step(L):
    fn = L.ssm_gdr_state_update
    one = dict(ws=None)
    assert call(fn, gdr(L=2), STEP, **one) == ESHAPE
    assert call(fn, gdr(L=1, P=24), STEP, **one) == EUNSUP
    assert call(fn, gdr(L=1, b=0), STEP, **one) == OK
    for n in STEP:
        assert call(fn, gdr(L=1), STEP, **one, **{n: 0}) == ENULL, n
    assert call(fn, gdr(L=1), STEP, **one, h=7 * GB + 8) == EALIGN
    assert call(fn, gdr(L=1), STEP, **one, q=1 * GB + 4) == EALIGN
    assert call(fn, gdr(L=1, strides=(130, 0, 0, 0, 0)), STEP, **one) == EALIGN
    assert call(fn, gdr(L=1), STEP, **one, h_out=7 * GB + 256) == EALIAS
    assert call(fn, gdr(L=1), STEP, **one, y=7 * GB) == EALIAS
    assert call(fn, gdr(L=1), STEP, **one, y=3 * GB) == EALIAS
    # one token's rows may lie as far apart as a long sequence's: the refusal is the null pointer's
    far = gdr(L=1, strides=(1 << 26, 0, 1 << 26, 0, 0))
    assert call(fn, far, STEP, **one, y=0) == ENULL
    assert call(L.ssm_gdr_fwd, far, FWD, y=0) == ESHAPE


def test_launch_limits(L):
    """Sizes whose launch would have 2^32 work items are refused by their shape;
    operands here lie 4 TiB apart."""
    T = 4096
    far = lambda names: {n: (k + 1) * T * GB for k, n in enumerate(names)}
    ws = dict(ws=64 * T * GB, ws_bytes=1 << 42)
    step = lambda **kw: call(L.ssm_gdr_state_update, gdr(L=1, **kw), STEP, ws=None, **far(STEP))
    assert step(b=1 << 22, H=4, P=16) == ESHAPE
    assert step(b=1 << 21, H=4, P=256, N=128, G=4) == ESHAPE
    for d in (pre(rows=1 << 24, dim=4096), pre(rows=1 << 26, dim=1024), pre(rows=1 << 29, dim=64)):
        assert call(L.ssm_prenorm_fwd, d, PRE, ws=None, **far(PRE)) == ESHAPE
    assert call(L.ssm_gated_norm_fwd, gated(rows=1 << 25, groups=16), GAT, ws=None, **far(GAT)) == ESHAPE
    for d in (gated(rows=1, groups=1 << 20, dim=64), gated(rows=1 << 24, groups=1, dim=16384)):
        assert call(L.ssm_gated_norm_bwd, d, GATB, **ws, **far(GATB)) == ESHAPE
    assert call(L.ssm_prenorm_bwd, pre(rows=1 << 24, dim=16384), PREB, **ws, **far(PREB)) == ESHAPE


def test_sequence_launch_limits(L):
    """Sequences whose launches would have 2^32 work items, in the preparation, a walk
    or the gradients: refused by their shape before the first; sizes just below go on
    to the next check (a null pointer's)."""
    T = 4096
    far = lambda names: {n: (k + 1) * T * GB for k, n in enumerate(names)}
    ws = dict(ws=64 * T * GB, ws_bytes=1 << 42)
    fwd = lambda d, **o: call(L.ssm_gdr_fwd, d, FWD, **ws, **dict(far(FWD), **o))
    bwd = lambda fn, d, **o: call(fn, d, BWD, **ws, **dict(far(BWD), **o))
    walk = dict(H=4, G=4, P=256, L=1)
    assert fwd(gdr(b=1 << 20, **walk)) == ESHAPE
    assert fwd(gdr(b=(1 << 20) - 1, **walk), y=0) == ENULL
    prep = dict(b=1, H=1, G=1, P=16)
    assert fwd(gdr(L=(1 << 30) - 63, **prep)) == ESHAPE
    assert fwd(gdr(L=(1 << 30) - 128, **prep), y=0) == ENULL
    assert fwd(gdr(L=1 << 29, N=128, **prep), y=0) == ENULL
    for fn in (L.ssm_gdr_bwd, L.ssm_gdr_bwd_saved):
        assert bwd(fn, gdr(b=1 << 20, **walk)) == ESHAPE
        assert bwd(fn, gdr(L=1 << 29, N=128, **prep)) == ESHAPE
        assert bwd(fn, gdr(L=(1 << 29) - 64, N=128, **prep), dq=0) == ENULL
    assert call(L.ssm_gdr_fwd, gdr(b=1 << 20, **dict(walk, L=0)), FWD, **dict(far(FWD), h_last=0)) == OK


def pre(rows=4, dim=64, dt=ssm.SSM_BF16, rt=ssm.SSM_BF16, eps=1e-5, reserved=0, xs=0):
    return ssm.PrenormDesc(rows, dim, dt, rt, eps, reserved, xs)


PRE = dict(x=1, residual=2, scale=3, weight=4, r=5, y=6)
PREB = dict(dy=1, r=2, dr=3, x=4, scale=5, weight=6, dx=7, dresidual=8, dweight=9, dscale=10)


def test_prenorm(L):
    fwd = lambda d, **o: call(L.ssm_prenorm_fwd, d, PRE, ws=None, **o)
    bwd = lambda d, **o: call(L.ssm_prenorm_bwd, d, PREB, **o)
    for f in (fwd, bwd):
        assert f(None) == ENULL
        for kw, want in ((dict(rows=-1), ESHAPE), (dict(dim=0), ESHAPE), (dict(dim=(1 << 20) + 1), ESHAPE),
                         (dict(xs=63), ESHAPE), (dict(rows=1 << 40), ESHAPE), (dict(dt=4), EDTYPE), (dict(rt=4), EDTYPE),
                         (dict(dt=ssm.SSM_F32), EUNSUP), (dict(eps=-1.0), EUNSUP), (dict(eps=float("nan")), EUNSUP),
                         (dict(reserved=1), EUNSUP)):
            assert f(pre(**kw)) == want, kw
    assert fwd(pre(rows=0)) == OK
    for n in ("x", "weight", "y"):
        assert fwd(pre(), **{n: 0}) == ENULL
    assert fwd(pre(), x=1 * GB + 1) == EALIGN
    assert fwd(pre(rt=ssm.SSM_F32), r=5 * GB + 2) == EALIGN
    for n in ("x", "residual", "scale", "weight", "r"):
        assert fwd(pre(), y=PRE[n] * GB) == EALIAS, n
    assert fwd(pre(), r=2 * GB + 64) == EALIAS
    for n in ("dy", "r", "weight", "dx", "dweight", "dscale", "x"):
        assert bwd(pre(), **{n: 0}) == ENULL, n
    assert bwd(pre(), ws=0) == EWS
    need = L.ssm_prenorm_bwd_workspace_size(ctypes.byref(pre()))
    assert need > 0 and bwd(pre(), ws_bytes=need - 1) == EWS
    assert bwd(pre(), ws=20 * GB + 4) == EALIGN
    for n in ("dy", "r", "dr", "x", "dresidual", "dweight"):
        assert bwd(pre(), dx=PREB[n] * GB) == EALIAS, n
    assert bwd(pre(), ws=1 * GB) == EALIAS


def gated(rows=4, groups=2, dim=64, dt=ssm.SSM_BF16, first=0, shared=0, eps=1e-5, xs=0, zs=0):
    return ssm.GatedNormDesc(rows, groups, dim, dt, first, shared, eps, xs, zs)


GAT = dict(x=1, z=2, weight=3, y=4)
GATB = dict(dy=1, x=2, z=3, weight=4, dx=5, dz=6, dweight=7)


def test_gated_norm(L):
    fwd = lambda d, **o: call(L.ssm_gated_norm_fwd, d, GAT, ws=None, **o)
    bwd = lambda d, **o: call(L.ssm_gated_norm_bwd, d, GATB, **o)
    for f in (fwd, bwd):
        assert f(None) == ENULL
        for kw, want in ((dict(rows=-1), ESHAPE), (dict(groups=0), ESHAPE), (dict(dim=0), ESHAPE),
                         (dict(xs=127), ESHAPE), (dict(zs=1), ESHAPE), (dict(rows=1 << 40), ESHAPE), (dict(dt=5), EDTYPE),
                         (dict(first=2), EUNSUP), (dict(shared=2), EUNSUP), (dict(eps=float("inf")), EUNSUP)):
            assert f(gated(**kw)) == want, kw
    assert fwd(gated(rows=0)) == OK
    for n in ("x", "weight", "y"):
        assert fwd(gated(), **{n: 0}) == ENULL
    assert fwd(gated(), z=2 * GB + 1) == EALIGN
    for n in ("x", "z", "weight"):
        assert fwd(gated(), y=GAT[n] * GB) == EALIAS
    for n in ("dy", "x", "weight", "dx", "dz", "dweight"):
        assert bwd(gated(), **{n: 0}) == ENULL, n
    assert bwd(gated(), ws=0) == EWS
    for n in ("dy", "x", "z", "weight", "dz", "dweight"):
        assert bwd(gated(), dx=GATB[n] * GB) == EALIAS, n
