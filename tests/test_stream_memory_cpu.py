"""What a call with a stream handed over allocates belongs to that stream, and what
it returns is held for the current one: on the host, with the library's launches
and torch's streams replaced."""
import os

import pytest

import selective_state_space_78_amd as ssm

torch = pytest.importorskip("torch")
BF, F32 = torch.bfloat16, torch.float32


class Stream:
    def __init__(self, name):
        self.name = name
        self.cuda_stream = 0

    def __eq__(self, other):
        return self is other


class Library:
    """Workspace sizes as they are; every launch succeeds."""

    def __init__(self, real):
        self.real = real

    def __getattr__(self, name):
        return getattr(self.real, name) if "workspace_size" in name else lambda *args: 0


@pytest.fixture
def world(monkeypatch):
    if not os.path.exists(ssm.LIBRARY):
        pytest.skip("library not built")
    w = type("World", (), dict(inside=[], made=[], held=[], here=Stream("current"), other=Stream("handed over")))()
    empty, real = torch.empty, ssm.lib()

    class Under:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            w.inside.append(self.stream)

        def __exit__(self, *_):
            w.inside.pop()

    def made(*args, **kw):
        t = empty(*args, **kw)
        w.made.append((t, w.inside[-1] if w.inside else w.here))
        return t
    monkeypatch.setattr(torch, "empty", made)
    monkeypatch.setattr(torch.cuda, "stream", Under)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: w.here)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: w.held.append((t, s)))
    monkeypatch.setattr(ssm, "_stream", lambda stream, device: 0)
    monkeypatch.setattr(ssm, "lib", lambda: Library(real))
    return w


def rule(L=3):
    lead = (2,) if L is None else (2, L)
    t = lambda *s: torch.zeros(*lead, *s, dtype=BF)
    return t(1, 64), t(1, 64), t(2, 16), t(2), t(2), torch.zeros(2)


def scan():
    t = torch.zeros(2, 40, 16, dtype=BF)
    return t, t, torch.zeros(16, 4), torch.zeros(2, 40, 4, dtype=BF), torch.zeros(2, 40, 4, dtype=BF)


def ssd(L=40):
    lead = (2,) if L is None else (2, L)
    t = lambda *s: torch.zeros(*lead, *s, dtype=BF)
    return t(2, 16), t(2), torch.zeros(2), t(1, 64), t(1, 64)


CALLS = {
    "scan_fwd": lambda **k: ssm.ssm_scan_fwd(*scan(), **k),
    "scan_fwd_tuned": lambda **k: ssm.ssm_scan_fwd(*scan(), tuning=(1, 2), **k),
    "scan_fwd_noalloc": lambda **k: ssm.ssm_scan_fwd_noalloc(*scan(), **k),
    "scan_fwd_save": lambda **k: ssm.ssm_scan_fwd_save(*scan(), **k),
    "scan_bwd": lambda **k: ssm.ssm_scan_bwd(*scan(), scan()[0], D=torch.zeros(16), z=scan()[0], **k),
    "state_update": lambda **k: ssm.ssm_state_update(*(t[:, 0].contiguous() if t.dim() == 3 else t for t in scan()),
                                                     torch.zeros(2, 16, 4), **k),
    "ssd_fwd": lambda **k: ssm.ssm_ssd_fwd(*ssd(), **k),
    "ssd_state_update": lambda **k: ssm.ssm_ssd_state_update(*ssd(None), torch.zeros(2, 2, 16, 64), **k),
    "gdr_fwd": lambda **k: ssm.ssm_gdr_fwd(*rule(), **k),
    "gdr_fwd_save": lambda **k: ssm.ssm_gdr_fwd_save(*rule(), **k),
    "gdr_bwd": lambda **k: ssm.ssm_gdr_bwd(*rule(), rule()[2], dt_bias=torch.zeros(2), **k),
    "gdr_state_update": lambda **k: ssm.ssm_gdr_state_update(*rule(None), torch.zeros(2, 2, 16, 64), **k),
    "prenorm_fwd": lambda **k: ssm.ssm_prenorm_fwd(torch.zeros(4, 8), torch.zeros(8), **k),
    "prenorm_bwd": lambda **k: ssm.ssm_prenorm_bwd(torch.zeros(4, 8), torch.zeros(4, 8), torch.zeros(8), x=torch.zeros(4, 8),
                                                   scale=torch.zeros(8), **k),
    "gated_norm_fwd": lambda **k: ssm.ssm_gated_norm_fwd(torch.zeros(4, 2, 8), torch.zeros(4, 2, 8), torch.zeros(8), **k),
    "gated_norm_bwd": lambda **k: ssm.ssm_gated_norm_bwd(*(torch.zeros(4, 2, 8) for _ in range(3)), torch.zeros(8), **k),
}


def tensors(result):
    if isinstance(result, dict):
        result = result.values()
    elif not isinstance(result, (tuple, list)):
        result = [result]
    return [t for t in result if t is not None]


@pytest.mark.parametrize("call", CALLS.values(), ids=list(CALLS))
def test_memory_of_a_stream_handed_over(world, call):
    given = tensors(call(stream=world.other))
    assert world.made and all(s is world.other for _, s in world.made)
    assert all(any(t is h and s is world.here for h, s in world.held) for t in given)
    # what the call keeps to itself goes back to that stream alone
    assert len(world.held) == len(given)


@pytest.mark.parametrize("call", CALLS.values(), ids=list(CALLS))
def test_memory_of_the_current_stream(world, call):
    for k in (dict(), dict(stream=world.here)):
        world.made.clear()
        call(**k)
        assert world.made and all(s is world.here for _, s in world.made) and not world.held
