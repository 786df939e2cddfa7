"""GPU: calls with a stream handed over, while work on the current stream still
uses memory that it has given back, and with results dropped before they are
written."""
import pytest

from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = torch_cuda()
    import selective_state_space_78_amd as ssm
    ssm.lib()
    return torch, ssm


def flat(result):
    if isinstance(result, dict):
        result = result.values()
    elif not isinstance(result, (tuple, list)):
        result = [result]
    return [t for t in result if t is not None]


def calls(torch, ssm):
    bf = torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
    B, L, H, P, N = 2, 200, 4, 64, 64
    q, k, v, dy = (rnd(B, L, H, n).to(bf) for n in (N, N, P, P))
    dt, beta, A = rnd(B, L, H).to(bf), rnd(B, L, H).to(bf), -rnd(H).abs()
    o = dict(dt_softplus=True, beta_sigmoid=True, qk_norm=True)
    h = rnd(B, H, P, N)
    x, z, w, s = rnd(500, 4, 64), rnd(500, 4, 64), rnd(64), rnd(64)
    flat_x, flat_z = x.flatten(0, 1), z.flatten(0, 1)
    out = torch.empty_like(h)
    u, de, zz, dyu = (rnd(B, L, 128) for _ in range(4))
    Bs, Cs, As, D = rnd(B, L, 16), rnd(B, L, 16), -rnd(128, 16).abs(), rnd(128)
    de = 0.1 * de.abs()
    sx, sd, sB, sC = rnd(B, L, H, P).to(bf), rnd(B, L, H).abs().to(bf), rnd(B, L, 1, N).to(bf), rnd(B, L, 1, N).to(bf)
    # (a scan's workspace holds bytes that nothing writes)
    return {
        "scan_fwd": lambda **kw: ssm.ssm_scan_fwd(u, de, As, Bs, Cs, D, zz, **kw),
        "scan_fwd_save": lambda **kw: ssm.ssm_scan_fwd_save(u, de, As, Bs, Cs, D, zz, **kw)[:2],
        "scan_bwd": lambda **kw: ssm.ssm_scan_bwd(u, de, As, Bs, Cs, dyu, D, zz, **kw),
        "ssd_fwd": lambda **kw: ssm.ssm_ssd_fwd(sx, sd, A, sB, sC, **kw),
        "gdr_fwd": lambda **kw: ssm.ssm_gdr_fwd(q, k, v, dt, beta, A, **o, **kw),
        # (the workspace holds bytes that nothing writes)
        "gdr_fwd_save": lambda **kw: ssm.ssm_gdr_fwd_save(q, k, v, dt, beta, A, **o, **kw)[:2],
        "gdr_bwd": lambda **kw: ssm.ssm_gdr_bwd(q, k, v, dt, beta, A, dy, **o, **kw),
        "gdr_state_update": lambda **kw: ssm.ssm_gdr_state_update(q[:, 0], k[:, 0], v[:, 0], dt[:, 0], beta[:, 0], A, h, h_out=out,
                                                                  **o, **kw),
        "prenorm_fwd": lambda **kw: ssm.ssm_prenorm_fwd(flat_x, w, residual=flat_z, scale=s, **kw),
        "prenorm_bwd": lambda **kw: ssm.ssm_prenorm_bwd(flat_z, flat_x, w, x=flat_z, scale=s, **kw),
        "gated_norm_fwd": lambda **kw: ssm.ssm_gated_norm_fwd(x, z, w, **kw),
        "gated_norm_bwd": lambda **kw: ssm.ssm_gated_norm_bwd(z, x, z, w, **kw),
    }


NAMES = ["scan_fwd", "scan_fwd_save", "scan_bwd", "ssd_fwd", "gdr_fwd", "gdr_fwd_save", "gdr_bwd", "gdr_state_update",
         "prenorm_fwd", "prenorm_bwd", "gated_norm_fwd", "gated_norm_bwd"]
WAIT = 10_000_000      # clock cycles: some milliseconds


@pytest.mark.parametrize("name", NAMES)
def test_memory_that_queued_work_still_uses(env, name):
    torch, ssm = env
    call = calls(torch, ssm)[name]
    want = [t.clone() for t in flat(call())]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    # blocks of the results' sizes and of the workspaces', given back while a fill of them is queued
    old = [torch.empty_like(t) for t in want] + [torch.empty(n, dtype=torch.uint8, device="cuda") for n in
                                                 (1 << 16, 1 << 20, 1 << 22, 1 << 24, 1 << 25)]
    torch.cuda._sleep(WAIT)
    for t in old:
        t.fill_(7)
    del old, t
    got = flat(call(stream=s))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", NAMES)
def test_results_dropped_before_they_are_written(env, name):
    torch, ssm = env
    call = calls(torch, ssm)[name]
    want = [t.clone() for t in flat(call())]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(WAIT)
    call(stream=s)
    new = [torch.full_like(t, 5.0) for t in want] * 2
    torch.cuda.synchronize()
    assert all(bool((t == 5.0).all()) for t in new)
