"""GPU: the norm over many gradients and their clipping.

Tolerances: the sum is taken in 64 bits, so the norm is off by its rounding to fp32,
2^-24 of itself (and some 2^-50). The factor is rounded to fp32 once (2^-24), the
product once (2^-24), a bf16 result once more (2^-8 at the most, half a step is 2^-9
to 2^-8 of the value): 3 half steps of fp32, and 2^-8 with bf16.
"""
import numpy as np
import pytest

from gpu_util import torch_cuda
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
    return t.detach().double().cpu().numpy()


def make(torch, sizes, seed=0, scale=0.01):
    """Tensors of both types, at every alignment, in buffers whose other elements are marked."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    kinds = [torch.bfloat16, torch.float32]
    buffers, views = [], []
    for k, n in enumerate(sizes):
        t = kinds[k % 2]
        b = torch.full((n + 24,), 7.0, dtype=t, device="cuda")
        at = (3 * k + k // 2) % 9
        v = b[at:at + n]
        v.copy_(scale * torch.randn(n, generator=g, device="cuda"))
        buffers.append((b, at, n))
        views.append(v)
    return buffers, views


def around(buffers):
    return all(bool((b[:at] == 7).all()) and bool((b[at + n:] == 7).all()) for b, at, n in buffers)


SIZES = {"one": [1], "few": [5, 0, 17, 4096, 1], "border": [8191, 8192, 8193, 8199, 8200, 16384, 16391, 3, 65536, 7],
         "many": [(37 * k * k) % 5000 for k in range(300)], "long": [3_000_001, 2_999_999, 100]}


@pytest.mark.parametrize("sizes", SIZES.values(), ids=list(SIZES))
@pytest.mark.parametrize("max_norm", [1e-3, 0.7, 1e9])
def test_clip(env, sizes, max_norm):
    torch, ssm = env
    buffers, grads = make(torch, sizes, len(sizes))
    ref, want = block.clip([np64(g) for g in grads], max_norm)
    before = [g.clone() for g in grads]
    other_buffers, other = make(torch, sizes, 99)
    norm = ssm.ssm_grad_clip(grads, max_norm, out=other)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    alone = ssm.ssm_grad_norm(grads)
    same = [b.clone() for b in before]
    ssm.ssm_grad_scale(same, alone, max_norm)
    norm2 = ssm.ssm_grad_clip(grads, max_norm)
    torch.cuda.synchronize()
    assert abs(float(norm) - ref) <= 1.01 * U * ref
    assert torch.equal(norm, norm2) and torch.equal(norm, alone)
    assert around(buffers) and around(other_buffers)
    for g, o, s, w, b in zip(grads, other, same, want, before):
        assert torch.equal(g, o)
        off = (3 * U + (2.0 ** -8 if g.dtype == torch.bfloat16 else 0)) * np.abs(w)
        assert (np.abs(np64(g) - w) <= off).all()
        # the norm rounded to fp32 first: one half step more
        assert (np.abs(np64(s) - w) <= off + U * np.abs(w)).all()
        if max_norm > ref + 1e-6:
            assert torch.equal(g, b)


def test_aligned_differently(env):
    """Source and destination a few elements apart in their alignment."""
    torch, ssm = env
    a = torch.randn(20000, device="cuda").bfloat16()
    out = torch.zeros(20011, device="cuda").bfloat16()
    norm = ssm.ssm_grad_clip([a[5:19000]], 0.5, out=[out[2:18997]])
    torch.cuda.synchronize()
    ref, (want,) = block.clip([np64(a[5:19000])], 0.5)
    assert (np.abs(np64(out[2:18997]) - want) <= (2.0 ** -8 + 3 * U) * np.abs(want)).all() and abs(float(norm) - ref) <= 1.01 * U * ref
    assert not out[:2].any() and not out[18997:].any()


def test_sizes_of_values(env):
    """Values whose squares overflow or vanish in 32 bits; infinities and NaN."""
    torch, ssm = env
    t = lambda *v: torch.tensor(v, device="cuda")
    for v in (1e30, 1e-30):
        g = [t(3 * v, 0.0), t(4 * v)]
        norm = ssm.ssm_grad_clip(g, v, eps=0.0)
        torch.cuda.synchronize()
        assert abs(float(norm) / v - 5) <= 5e-6 and abs(float(g[1]) / v - 0.8) <= 1e-6
    g = [t(1.0, float("inf")), t(2.0)]
    norm = ssm.ssm_grad_clip(g, 1.0)
    torch.cuda.synchronize()
    assert float(norm) == float("inf") and float(g[1]) == 0 and float(g[0][0]) == 0 and bool(g[0][1].isnan())
    g = [t(1.0, float("nan")), t(2.0)]
    norm = ssm.ssm_grad_clip(g, 1.0)
    torch.cuda.synchronize()
    assert bool(norm.isnan()) and bool(g[1].isnan().all())


def test_norm_beyond_fp32(env):
    """Finite gradients whose norm is beyond fp32: it is infinity, and they become 0, by either route; one just inside
    leaves what the formula says."""
    torch, ssm = env
    full = lambda n, v, t: torch.full((n,), v, device="cuda", dtype=t)
    # a few workgroups' sums, some hundred, those of two launches, and so many that a launch of its own adds them
    for sizes in ([2, 1], [3_000_000, 5], [100] * 130, [80_000] * 130):
        for t in (torch.float32, torch.bfloat16):
            grads = [full(n, 3e38, t) for n in sizes]
            out = [torch.ones_like(g) for g in grads]
            norm = ssm.ssm_grad_clip(grads, 1.0, out=out)
            same = [g.clone() for g in grads]
            alone = ssm.ssm_grad_norm(same)
            ssm.ssm_grad_scale(same, alone, 1.0)
            ssm.ssm_grad_clip(grads, 1.0)
            torch.cuda.synchronize()
            assert float(norm) == float("inf") == float(alone)
            for g, o, k in zip(grads, out, same):
                assert not bool(g.any()) and not bool(o.any()) and not bool(k.any()), (sizes, t)
    grads = [full(1, 2e38, torch.float32) for _ in range(2)]
    ref, want = block.clip([np64(g) for g in grads], 1e30)
    norm = ssm.ssm_grad_clip(grads, 1e30)
    torch.cuda.synchronize()
    assert abs(float(norm) - ref) <= 1.01 * U * ref
    for g, w in zip(grads, want):
        assert (np.abs(np64(g) - w) <= 3 * U * np.abs(w)).all()


def test_nothing(env):
    torch, ssm = env
    e = torch.zeros(0, device="cuda")
    assert float(ssm.ssm_grad_clip([e, None, e], 1.0)) == 0
    norm = torch.ones((), device="cuda")
    assert float(ssm.ssm_grad_norm([], norm=norm)) == 0
    ssm.ssm_grad_scale([None], norm, 1.0)
    assert float(ssm.ssm_grad_norm([torch.ones(4, device="cuda")] * 4)) == 4


def test_norm_of_zero(env):
    """Zeros stay zeros, also where the formula's quotient would be 0 / 0."""
    torch, ssm = env
    for max_norm, eps in ((1.0, 1e-6), (1.0, 0.0), (0.0, 1e-6), (0.0, 0.0)):
        g = [torch.zeros(70000, device="cuda"), torch.zeros(5, device="cuda").bfloat16()]
        out = [torch.ones_like(t) for t in g]
        norm = ssm.ssm_grad_clip(g, max_norm, eps=eps, out=out)
        torch.cuda.synchronize()
        assert float(norm) == 0 and not any(bool(t.any()) for t in out), (max_norm, eps)


def test_captured(env):
    """In a graph, replayed on new gradients with eager work between."""
    torch, ssm = env
    _, grads = make(torch, [4097] * 150 + [70000])
    ssm.ssm_grad_clip(grads, 0.5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = ssm.ssm_grad_clip(grads, 0.5)
    for k in range(3):
        for g in grads:
            g.normal_()
        eager = [g.clone() for g in grads]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = ssm.ssm_grad_clip(eager, 0.5)
        torch.cuda.synchronize()
        assert torch.equal(norm, want) and all(torch.equal(a, b) for a, b in zip(grads, eager)), k
