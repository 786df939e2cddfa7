"""Python binding of the MI355X selective-scan library (libssm_scan.so).

Argument marshalling only: every step of the scans, the delta rule, the norms
and the decode steps runs in the library's HIP kernels. PyTorch supplies device memory and the current
HIP stream; the library itself is a plain C ABI (include/ssm_scan.h) that
links no torch. There is no fallback: if the library is missing, every call
raises.

Names follow the C ABI: ``ssm_scan_fwd``, ``ssm_scan_fwd_noalloc``, ``ssm_scan_workspace_size``,
``ssm_scan_plan``, ``ssm_scan_bwd``, ``ssm_state_update``, ``ssm_ssd_fwd``,
``ssm_gdr_fwd``, ``ssm_gdr_bwd``, ``ssm_gdr_state_update``, ``ssm_prenorm_fwd``,
``ssm_gated_norm_fwd``, ``ssm_status_string``.

``stream`` runs a call on a stream other than the current one. The caller orders the
two where inputs or results cross; what the call allocates comes out of that stream's
memory.
"""
from __future__ import annotations

import ctypes
import os
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(PKG, "libssm_scan.so")

SSM_F32, SSM_BF16 = 0, 1
SSM_DISC_EULER, SSM_DISC_ZOH = 0, 1
_DISC = {"euler": SSM_DISC_EULER, "zoh": SSM_DISC_ZOH}

# Every symbol include/ssm_scan.h declares.
EXPORTS = ("ssm_scan_workspace_size", "ssm_scan_fwd", "ssm_scan_workspace_size_tuned",
           "ssm_scan_fwd_tuned", "ssm_scan_plan", "ssm_scan_bwd_workspace_size", "ssm_scan_bwd",
           "ssm_scan_fwd_save", "ssm_scan_bwd_saved", "ssm_state_update", "ssm_ssd_fwd", "ssm_ssd_state_update",
           "ssm_scan_fwd_noalloc", "ssm_gdr_workspace_size", "ssm_gdr_bwd_workspace_size", "ssm_gdr_fwd",
           "ssm_gdr_fwd_save", "ssm_gdr_bwd", "ssm_gdr_bwd_saved", "ssm_gdr_state_update", "ssm_prenorm_fwd",
           "ssm_prenorm_bwd", "ssm_prenorm_bwd_workspace_size", "ssm_gated_norm_fwd", "ssm_gated_norm_bwd",
           "ssm_gated_norm_bwd_workspace_size", "ssm_status_string")

# Fixed scratch of ssm_scan_fwd_noalloc per GPU (SSM_NOALLOC_SCRATCH_BYTES).
NOALLOC_SCRATCH_BYTES = 64 << 20


class ScanDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("dtype", ctypes.c_int32), ("disc", ctypes.c_int32),
                ("delta_softplus", ctypes.c_int32), ("conv_width", ctypes.c_int32),
                ("delta_bias", ctypes.c_void_p), ("conv_weight", ctypes.c_void_p), ("conv_bias", ctypes.c_void_p)]


class SsdDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int32),
                ("headdim", ctypes.c_int32), ("ngroups", ctypes.c_int32), ("dstate", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("disc", ctypes.c_int32), ("dt_softplus", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("dt_bias", ctypes.c_void_p)]


class GdrDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int32),
                ("headdim", ctypes.c_int32), ("ngroups", ctypes.c_int32), ("dstate", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("dt_softplus", ctypes.c_int32), ("beta_sigmoid", ctypes.c_int32),
                ("qk_norm", ctypes.c_int32), ("scale", ctypes.c_float), ("qk_eps", ctypes.c_float),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("dt_stride", ctypes.c_int64), ("beta_stride", ctypes.c_int64), ("dt_bias", ctypes.c_void_p)]


class PrenormDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("residual_dtype", ctypes.c_int32), ("eps", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("x_stride", ctypes.c_int64)]


class GatedNormDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("groups", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("gate_first", ctypes.c_int32), ("weight_shared", ctypes.c_int32),
                ("eps", ctypes.c_float), ("x_stride", ctypes.c_int64), ("z_stride", ctypes.c_int64)]


class ScanTuning(ctypes.Structure):
    _fields_ = [("state_groups", ctypes.c_int32), ("segments", ctypes.c_int32)]


class SsmError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__("%s failed: %s (status %d)" % (what, ssm_status_string(status), status))
        self.status = status


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIBRARY):
                raise ImportError("libssm_scan.so is not built (run __graft_entry__.build() or "
                                  "python selective_state_space_78_amd/build.py); there is no fallback")
            L = ctypes.CDLL(LIBRARY)
            vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
            pdesc, ptun = ctypes.POINTER(ScanDesc), ctypes.POINTER(ScanTuning)
            L.ssm_scan_workspace_size.argtypes = [pdesc]
            L.ssm_scan_workspace_size.restype = sz
            L.ssm_scan_workspace_size_tuned.argtypes = [pdesc, ptun]
            L.ssm_scan_workspace_size_tuned.restype = sz
            L.ssm_scan_plan.argtypes = [pdesc, ptun]
            L.ssm_scan_plan.restype = ctypes.c_int
            scan_args = [pdesc, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz]
            L.ssm_scan_fwd.argtypes = scan_args + [vp]
            L.ssm_scan_fwd.restype = ctypes.c_int
            L.ssm_scan_fwd_noalloc.argtypes = scan_args[:-2] + [vp]
            L.ssm_scan_fwd_noalloc.restype = ctypes.c_int
            L.ssm_scan_fwd_tuned.argtypes = scan_args + [ptun, vp]
            L.ssm_scan_fwd_tuned.restype = ctypes.c_int
            L.ssm_scan_bwd_workspace_size.argtypes = [pdesc]
            L.ssm_scan_bwd_workspace_size.restype = sz
            L.ssm_scan_bwd.argtypes = [pdesc] + [vp] * 21 + [vp, sz, vp]
            L.ssm_scan_fwd_save.restype = ctypes.c_int
            L.ssm_scan_fwd_save.argtypes = scan_args + [vp]
            L.ssm_scan_bwd_saved.restype = ctypes.c_int
            L.ssm_scan_bwd_saved.argtypes = [pdesc] + [vp] * 21 + [vp, sz, vp]
            L.ssm_scan_bwd.restype = ctypes.c_int
            L.ssm_state_update.argtypes = [i64, i64, i64, i32, i32, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp,
                                           vp]
            L.ssm_state_update.restype = ctypes.c_int
            L.ssm_ssd_fwd.argtypes = [ctypes.POINTER(SsdDesc)] + [vp] * 11
            L.ssm_ssd_fwd.restype = ctypes.c_int
            L.ssm_ssd_state_update.argtypes = [ctypes.POINTER(SsdDesc)] + [vp] * 10
            L.ssm_ssd_state_update.restype = ctypes.c_int
            pg, pp, pn = ctypes.POINTER(GdrDesc), ctypes.POINTER(PrenormDesc), ctypes.POINTER(GatedNormDesc)
            for name, d in (("ssm_gdr_workspace_size", pg), ("ssm_gdr_bwd_workspace_size", pg),
                            ("ssm_prenorm_bwd_workspace_size", pp), ("ssm_gated_norm_bwd_workspace_size", pn)):
                getattr(L, name).argtypes = [d]
                getattr(L, name).restype = sz
            for name, args in (("ssm_gdr_fwd", [pg] + [vp] * 10 + [sz, vp]),
                               ("ssm_gdr_fwd_save", [pg] + [vp] * 10 + [sz, vp]),
                               ("ssm_gdr_bwd", [pg] + [vp] * 18 + [sz, vp]),
                               ("ssm_gdr_bwd_saved", [pg] + [vp] * 18 + [sz, vp]),
                               ("ssm_gdr_state_update", [pg] + [vp] * 10),
                               ("ssm_prenorm_fwd", [pp] + [vp] * 7),
                               ("ssm_prenorm_bwd", [pp] + [vp] * 11 + [sz, vp]),
                               ("ssm_gated_norm_fwd", [pn] + [vp] * 5),
                               ("ssm_gated_norm_bwd", [pn] + [vp] * 8 + [sz, vp])):
                getattr(L, name).argtypes = args
                getattr(L, name).restype = ctypes.c_int
            L.ssm_status_string.argtypes = [ctypes.c_int]
            L.ssm_status_string.restype = ctypes.c_char_p
            _lib = L
        return _lib


def ssm_status_string(status: int) -> str:
    return lib().ssm_status_string(int(status)).decode()


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return SSM_BF16
    if t.dtype == torch.float32:
        return SSM_F32
    raise TypeError("per-token tensors must be bfloat16 or float32, got %s" % t.dtype)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(t, name, shape=None, dtype=None, device=None):
    if t is None:
        return
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if shape is not None and t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))


def _stream(stream, device):
    if device.type != "cuda":
        raise ValueError("tensors must be on a GPU, got %s" % device)
    if stream is not None:
        return stream.cuda_stream
    import torch
    # the handle alone: a Stream object costs more than a launch of a small kernel
    index = device.index
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if index is None else index)


def _empty(shape, dtype, device, stream, returned=True):
    """A tensor that work on ``stream`` (None: the current one) is to write. Under a
    stream handed over it comes out of that stream's memory: a block of the current
    stream's may still be in use by work queued there, and would go back to it as
    soon as the tensor is dropped, written or not. What the caller gets is held for
    the work that they queue on the current stream as well."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    current = torch.cuda.current_stream(device)
    if stream == current:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(current)
    return t


def _on(device, fn, *args):
    """fn(*args) with the tensors' GPU as the current one."""
    import torch
    if device.index is None or device.index == torch.cuda.current_device():
        return fn(*args)
    with torch.cuda.device(device):
        return fn(*args)


def _tuning(tuning):
    if tuning is None:
        return None
    g, s = tuning
    return ctypes.byref(ScanTuning(int(g), int(s)))


def make_desc(batch, seqlen, dim, dstate, dtype, disc="euler", delta_bias=None, delta_softplus=False,
              conv_weight=None, conv_bias=None) -> ScanDesc:
    """The scan descriptor; ``delta_bias`` (dim,), ``conv_weight`` (dim, W) and
    ``conv_bias`` (dim,) are float32 device tensors or None."""
    ptr = lambda t: None if t is None else t.data_ptr()
    W = 0 if conv_weight is None else int(conv_weight.shape[1])
    return ScanDesc(int(batch), int(seqlen), int(dim), int(dstate), int(dtype), _DISC[disc],
                    int(bool(delta_softplus)), W, ptr(delta_bias), ptr(conv_weight), ptr(conv_bias))


def ssm_scan_workspace_size(batch, seqlen, dim, dstate, dtype=SSM_BF16, disc="euler", tuning=None,
                            delta_bias=None, delta_softplus=False, conv_weight=None, conv_bias=None) -> int:
    """Workspace bytes of ssm_scan_fwd for this shape and these options (the
    convolution prologue adds its u)."""
    desc = make_desc(batch, seqlen, dim, dstate, dtype, disc, delta_bias, delta_softplus, conv_weight, conv_bias)
    if tuning is None:
        return int(lib().ssm_scan_workspace_size(ctypes.byref(desc)))
    return int(lib().ssm_scan_workspace_size_tuned(ctypes.byref(desc), _tuning(tuning)))


def ssm_scan_plan(batch, seqlen, dim, dstate, dtype=SSM_BF16, disc="euler"):
    """(state_groups, segments) the library picks for this shape."""
    desc = make_desc(batch, seqlen, dim, dstate, dtype, disc)
    out = ScanTuning()
    rc = lib().ssm_scan_plan(ctypes.byref(desc), ctypes.byref(out))
    if rc != 0:
        raise SsmError(rc, "ssm_scan_plan")
    return out.state_groups, out.segments


def ssm_scan_fwd(u, delta, A, B, C, D=None, z=None, h0=None, y=None, h_last=None,
                 disc="euler", workspace=None, tuning=None, stream=None, want_h_last=True,
                 delta_bias=None, delta_softplus=False, conv_weight=None, conv_bias=None):
    """Selective scan forward on device tensors.

    u, delta, z: (batch, L, dim); B, C: (batch, L, N) of the same dtype
    (bfloat16 or float32); A: (dim, N) float32; D: (dim,) float32; h0:
    (batch, dim, N) float32. Outputs y (batch, L, dim) and h_last
    (batch, dim, N) are allocated when not given. Returns (y, h_last).
    ``tuning`` is an optional (state_groups, segments) pair. ``delta_bias``
    (dim,) float32 and ``delta_softplus`` form the step in the kernel:
    softplus(delta + bias). With ``conv_weight`` (dim, W <= 4) float32 (and
    ``conv_bias`` (dim,)), ``u`` holds x and the scan input is
    silu(causal depthwise conv1d(x) + bias), formed in the kernel.
    """
    y, h_last, _ = _fwd(u, delta, A, B, C, D, z, h0, y, h_last, disc, workspace, tuning, stream, want_h_last,
                        delta_bias, delta_softplus, conv_weight, conv_bias, save=False)
    return y, h_last


def ssm_scan_fwd_noalloc(u, delta, A, B, C, D=None, z=None, h0=None, y=None, h_last=None,
                         disc="euler", stream=None, want_h_last=True,
                         delta_bias=None, delta_softplus=False, conv_weight=None, conv_bias=None):
    """ssm_scan_fwd without a workspace (the C call of the same name): the
    library's fixed per-GPU scratch serves instead, and the call allocates no
    device memory of its own. Pass ``y`` (and ``h_last``) to allocate nothing
    here either. Problems needing more than NOALLOC_SCRATCH_BYTES of scratch
    raise SsmError (SSM_ERR_SCRATCH)."""
    y, h_last, _ = _fwd(u, delta, A, B, C, D, z, h0, y, h_last, disc, None, None, stream, want_h_last,
                        delta_bias, delta_softplus, conv_weight, conv_bias, save=False, noalloc=True)
    return y, h_last


def ssm_scan_fwd_save(u, delta, A, B, C, D=None, z=None, h0=None, y=None, h_last=None,
                      disc="euler", workspace=None, stream=None, want_h_last=True,
                      delta_bias=None, delta_softplus=False, conv_weight=None, conv_bias=None):
    """ssm_scan_fwd that also keeps the backward's checkpoints (the C call of
    the same name). Returns (y, h_last, saved): ``saved`` is the workspace
    (uint8, ssm_scan_bwd_workspace_size bytes; ``workspace`` if given) to pass
    unchanged to ssm_scan_bwd_saved with the same inputs."""
    return _fwd(u, delta, A, B, C, D, z, h0, y, h_last, disc, workspace, None, stream, want_h_last,
                delta_bias, delta_softplus, conv_weight, conv_bias, save=True)


def _fwd(u, delta, A, B, C, D, z, h0, y, h_last, disc, workspace, tuning, stream, want_h_last,
         delta_bias, delta_softplus, conv_weight, conv_bias, save, noalloc=False):
    import torch
    batch, L, dim = u.shape
    N = A.shape[1]
    dev = u.device
    dt = u.dtype
    code = _dtype_code(u)
    _check(u, "u", device=dev)
    _check(delta, "delta", (batch, L, dim), dt, dev)
    _check(z, "z", (batch, L, dim), dt, dev)
    _check(B, "B", (batch, L, N), dt, dev)
    _check(C, "C", (batch, L, N), dt, dev)
    _check(A, "A", (dim, N), torch.float32, dev)
    _check(D, "D", (dim,), torch.float32, dev)
    _check(h0, "h0", (batch, dim, N), torch.float32, dev)
    if y is None:
        y = _empty((batch, L, dim), dt, dev, stream)
    if h_last is None and want_h_last:
        h_last = _empty((batch, dim, N), torch.float32, dev, stream)
    _check(y, "y", (batch, L, dim), dt, dev)
    _check(h_last, "h_last", (batch, dim, N), torch.float32, dev)
    _check(delta_bias, "delta_bias", (dim,), torch.float32, dev)
    if conv_weight is not None:
        _check(conv_weight, "conv_weight", (dim, conv_weight.shape[1]), torch.float32, dev)
    _check(conv_bias, "conv_bias", (dim,), torch.float32, dev)
    desc = make_desc(batch, L, dim, N, code, disc, delta_bias, delta_softplus, conv_weight, conv_bias)
    L_ = lib()
    if noalloc:
        rc = L_.ssm_scan_fwd_noalloc(ctypes.byref(desc), _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                     _ptr(z), _ptr(h0), _ptr(y), _ptr(h_last), _stream(stream, dev))
        if rc != 0:
            raise SsmError(rc, "ssm_scan_fwd_noalloc")
        return y, h_last, None
    if save:
        need = L_.ssm_scan_bwd_workspace_size(ctypes.byref(desc))
    elif tuning is None:
        need = L_.ssm_scan_workspace_size(ctypes.byref(desc))
    else:
        need = L_.ssm_scan_workspace_size_tuned(ctypes.byref(desc), _tuning(tuning))
    if workspace is None and need > 0:
        workspace = _empty(need, torch.uint8, dev, stream, save)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = [ctypes.byref(desc), _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
            _ptr(h0), _ptr(y), _ptr(h_last), _ptr(workspace), ws_bytes]
    if save:
        name = "ssm_scan_fwd_save"
        rc = L_.ssm_scan_fwd_save(*args, _stream(stream, dev))
    elif tuning is None:
        name = "ssm_scan_fwd"
        rc = L_.ssm_scan_fwd(*args, _stream(stream, dev))
    else:
        name = "ssm_scan_fwd_tuned"
        rc = L_.ssm_scan_fwd_tuned(*args, _tuning(tuning), _stream(stream, dev))
    if rc != 0:
        raise SsmError(rc, name)
    return y, h_last, workspace


def ssm_scan_bwd_workspace_size(batch, L, dim, N, dtype_code, disc="euler", delta_bias=None,
                                delta_softplus=False, conv_weight=None, conv_bias=None) -> int:
    desc = make_desc(batch, L, dim, N, dtype_code, disc, delta_bias, delta_softplus, conv_weight, conv_bias)
    return int(lib().ssm_scan_bwd_workspace_size(ctypes.byref(desc)))


def ssm_scan_bwd_saved(u, delta, A, B, C, dy, saved, D=None, z=None, h0=None, dh_last=None, disc="euler",
                       stream=None, want_dh0=True, out=None, delta_bias=None, delta_softplus=False,
                       conv_weight=None, conv_bias=None):
    """ssm_scan_bwd that reads the checkpoints an ssm_scan_fwd_save call with
    the same inputs left in ``saved`` (its returned workspace) instead of
    recomputing them (the C call of the same name). Arguments and results as
    ssm_scan_bwd."""
    if saved is None:
        raise ValueError("ssm_scan_bwd_saved needs the workspace of an ssm_scan_fwd_save call")
    return ssm_scan_bwd(u, delta, A, B, C, dy, D=D, z=z, h0=h0, dh_last=dh_last, disc=disc, workspace=saved,
                        stream=stream, want_dh0=want_dh0, out=out, delta_bias=delta_bias,
                        delta_softplus=delta_softplus, conv_weight=conv_weight, conv_bias=conv_bias,
                        _saved=True)


def ssm_scan_bwd(u, delta, A, B, C, dy, D=None, z=None, h0=None, dh_last=None, disc="euler",
                 workspace=None, stream=None, want_dh0=True, out=None, delta_bias=None, delta_softplus=False,
                 conv_weight=None, conv_bias=None, _saved=False):
    """Backward of ssm_scan_fwd on device tensors.

    Inputs as ssm_scan_fwd, plus dy (batch, L, dim) of the input dtype and an
    optional dh_last (batch, dim, N) float32. Returns a dict with du, ddelta,
    dz (input dtype, dz only with a gate), dA (dim, N), dB, dC (batch, L, N),
    dD (dim,) (with a skip) and dh0 (batch, dim, N) (when ``want_dh0``), all
    float32 except the per-token ones, and ddelta_bias (dim,) with a
    ``delta_bias``. With ``conv_weight`` (dim, W) (and ``conv_bias``), ``u``
    holds x, du is the gradient of x, and dconv_weight (dim, W), dconv_bias
    (dim,) are added. ``out`` may hold preallocated outputs.
    """
    import torch
    batch, L, dim = u.shape
    N = A.shape[1]
    dev = u.device
    dt = u.dtype
    code = _dtype_code(u)
    _check(u, "u", device=dev)
    _check(delta, "delta", (batch, L, dim), dt, dev)
    _check(z, "z", (batch, L, dim), dt, dev)
    _check(B, "B", (batch, L, N), dt, dev)
    _check(C, "C", (batch, L, N), dt, dev)
    _check(A, "A", (dim, N), torch.float32, dev)
    _check(D, "D", (dim,), torch.float32, dev)
    _check(h0, "h0", (batch, dim, N), torch.float32, dev)
    _check(dy, "dy", (batch, L, dim), dt, dev)
    _check(dh_last, "dh_last", (batch, dim, N), torch.float32, dev)
    o = dict(out or {})
    f32 = torch.float32

    def get(name, shape, dtype, wanted=True):
        if not wanted:
            return None
        if name not in o or o[name] is None:
            o[name] = _empty(shape, dtype, dev, stream)
        _check(o[name], name, shape, dtype, dev)
        return o[name]
    du = get("du", (batch, L, dim), dt)
    dde = get("ddelta", (batch, L, dim), dt)
    dz = get("dz", (batch, L, dim), dt, z is not None)
    dA = get("dA", (dim, N), f32)
    dB = get("dB", (batch, L, N), f32)
    dC = get("dC", (batch, L, N), f32)
    dD = get("dD", (dim,), f32, D is not None)
    dh0 = get("dh0", (batch, dim, N), f32, want_dh0)
    _check(delta_bias, "delta_bias", (dim,), f32, dev)
    ddb = get("ddelta_bias", (dim,), f32, delta_bias is not None)
    W = 0 if conv_weight is None else int(conv_weight.shape[1])
    if conv_weight is not None:
        _check(conv_weight, "conv_weight", (dim, W), f32, dev)
    _check(conv_bias, "conv_bias", (dim,), f32, dev)
    dcw = get("dconv_weight", (dim, W), f32, W > 0)
    dcb = get("dconv_bias", (dim,), f32, W > 0)
    desc = make_desc(batch, L, dim, N, code, disc, delta_bias, delta_softplus, conv_weight, conv_bias)
    L_ = lib()
    need = L_.ssm_scan_bwd_workspace_size(ctypes.byref(desc))
    if workspace is not None and workspace.numel() * workspace.element_size() < need:
        raise ValueError("workspace has %d bytes, ssm_scan_bwd needs %d" % (
            workspace.numel() * workspace.element_size(), need))
    if workspace is None and need > 0:
        workspace = _empty(need, torch.uint8, dev, stream, False)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    name = "ssm_scan_bwd_saved" if _saved else "ssm_scan_bwd"
    rc = getattr(L_, name)(ctypes.byref(desc), _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                           _ptr(h0), _ptr(dy), _ptr(dh_last), _ptr(du), _ptr(dde), _ptr(dA), _ptr(dB), _ptr(dC),
                           _ptr(dD), _ptr(dz), _ptr(dh0), _ptr(ddb), _ptr(dcw), _ptr(dcb), _ptr(workspace), ws_bytes,
                           _stream(stream, dev))
    if rc != 0:
        raise SsmError(rc, name)
    return dict(du=du, ddelta=dde, dz=dz, dA=dA, dB=dB, dC=dC, dD=dD, dh0=dh0, ddelta_bias=ddb,
                dconv_weight=dcw, dconv_bias=dcb)


def ssm_state_update(x, delta, A, B, C, h, D=None, z=None, y=None, disc="euler", stream=None,
                     delta_bias=None, delta_softplus=False):
    """One decode step on device tensors; h (batch, dim, N) float32 is updated in place.

    x, delta, z: (batch, dim); B, C: (batch, N). Returns y (batch, dim).
    """
    import torch
    batch, dim = x.shape
    N = A.shape[1]
    dev = x.device
    dt = x.dtype
    code = _dtype_code(x)
    _check(x, "x", device=dev)
    _check(delta, "delta", (batch, dim), dt, dev)
    _check(z, "z", (batch, dim), dt, dev)
    _check(B, "B", (batch, N), dt, dev)
    _check(C, "C", (batch, N), dt, dev)
    _check(A, "A", (dim, N), torch.float32, dev)
    _check(D, "D", (dim,), torch.float32, dev)
    _check(h, "h", (batch, dim, N), torch.float32, dev)
    if y is None:
        y = _empty((batch, dim), dt, dev, stream)
    _check(y, "y", (batch, dim), dt, dev)
    _check(delta_bias, "delta_bias", (dim,), torch.float32, dev)
    rc = lib().ssm_state_update(batch, dim, N, code, _DISC[disc], _ptr(x), _ptr(delta), _ptr(delta_bias),
                                int(bool(delta_softplus)), _ptr(A),
                                _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(h), _ptr(y), _stream(stream, dev))
    if rc != 0:
        raise SsmError(rc, "ssm_state_update")
    return y


def make_ssd_desc(batch, seqlen, nheads, headdim, ngroups, dstate, dtype=SSM_BF16, disc="euler",
                  dt_bias=None, dt_softplus=False) -> SsdDesc:
    return SsdDesc(int(batch), int(seqlen), int(nheads), int(headdim), int(ngroups), int(dstate), int(dtype),
                   _DISC[disc], int(bool(dt_softplus)), 0, None if dt_bias is None else dt_bias.data_ptr())


def ssm_ssd_fwd(x, dt, A, B, C, D=None, z=None, h0=None, y=None, h_last=None, disc="euler",
                dt_bias=None, dt_softplus=False, want_h_last=True, stream=None):
    """Mamba-2 SSD layer on device tensors.

    x, z: (batch, L, H, P) bfloat16; dt: (batch, L, H) bfloat16; B, C:
    (batch, L, G, N) bfloat16; A, D, dt_bias: (H,) float32; h0: (batch, H, P, N)
    float32. Outputs y (batch, L, H, P) and h_last (batch, H, P, N) are
    allocated when not given. Returns (y, h_last).
    """
    import torch
    batch, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    dev = x.device
    code = _dtype_code(x)
    _check(x, "x", device=dev)
    _check(dt, "dt", (batch, L, H), x.dtype, dev)
    _check(z, "z", (batch, L, H, P), x.dtype, dev)
    _check(B, "B", (batch, L, G, N), x.dtype, dev)
    _check(C, "C", (batch, L, G, N), x.dtype, dev)
    _check(A, "A", (H,), torch.float32, dev)
    _check(D, "D", (H,), torch.float32, dev)
    _check(dt_bias, "dt_bias", (H,), torch.float32, dev)
    _check(h0, "h0", (batch, H, P, N), torch.float32, dev)
    if y is None:
        y = _empty((batch, L, H, P), x.dtype, dev, stream)
    if h_last is None and want_h_last:
        h_last = _empty((batch, H, P, N), torch.float32, dev, stream)
    _check(y, "y", (batch, L, H, P), x.dtype, dev)
    _check(h_last, "h_last", (batch, H, P, N), torch.float32, dev)
    desc = make_ssd_desc(batch, L, H, P, G, N, code, disc, dt_bias, dt_softplus)
    rc = lib().ssm_ssd_fwd(ctypes.byref(desc), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                           _ptr(h0), _ptr(y), _ptr(h_last), _stream(stream, dev))
    if rc != 0:
        raise SsmError(rc, "ssm_ssd_fwd")
    return y, h_last


def ssm_ssd_state_update(x, dt, A, B, C, h, D=None, z=None, y=None, disc="euler", dt_bias=None,
                         dt_softplus=False, stream=None):
    """One SSD decode step on device tensors: x, z (batch, H, P) bfloat16, dt
    (batch, H) bfloat16, B, C (batch, G, N) bfloat16, A, D, dt_bias (H,)
    float32; h (batch, H, P, N) float32 is updated in place. Returns y
    (batch, H, P), allocated when not given."""
    import torch
    batch, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    dev = x.device
    code = _dtype_code(x)
    _check(x, "x", device=dev)
    _check(dt, "dt", (batch, H), x.dtype, dev)
    _check(z, "z", (batch, H, P), x.dtype, dev)
    _check(B, "B", (batch, G, N), x.dtype, dev)
    _check(C, "C", (batch, G, N), x.dtype, dev)
    _check(A, "A", (H,), torch.float32, dev)
    _check(D, "D", (H,), torch.float32, dev)
    _check(dt_bias, "dt_bias", (H,), torch.float32, dev)
    _check(h, "h", (batch, H, P, N), torch.float32, dev)
    if y is None:
        y = _empty((batch, H, P), x.dtype, dev, stream)
    _check(y, "y", (batch, H, P), x.dtype, dev)
    desc = make_ssd_desc(batch, 1, H, P, G, N, code, disc, dt_bias, dt_softplus)
    rc = lib().ssm_ssd_state_update(ctypes.byref(desc), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                    _ptr(z), _ptr(h), _ptr(y), _stream(stream, dev))
    if rc != 0:
        raise SsmError(rc, "ssm_ssd_state_update")
    return y


def _row_stride(t, name, lead, tail, dtype, device):
    """Elements from one row of `t` (the `tail` dimensions, dense) to the next,
    where the rows of the `lead` dimensions follow one another evenly; raises
    for any other layout."""
    if t.shape != lead + tail:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), lead + tail))
    if t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if t.is_contiguous():
        return 0
    width = 1
    for n, st in zip(reversed(tail), reversed(t.stride()[len(lead):])):
        if n != 1 and st != width and t.numel() > 0:
            raise ValueError("the last %d dimension(s) of %s must be dense" % (len(tail), name))
        width *= n
    if t.numel() == 0:
        return 0
    # innermost leading dimension of more than one row gives the stride
    row, rows = None, 1
    for n, st in zip(reversed(lead), reversed(t.stride()[:len(lead)])):
        if n == 1:
            continue
        if row is None:
            row = st
        elif st != row * rows:
            raise ValueError("the rows of %s must be evenly spaced" % name)
        rows *= n
    if row is None or row == width:
        return 0
    if row < width:
        raise ValueError("the rows of %s overlap" % name)
    return row


def _gdr_desc(q, k, v, dt, beta, A, scale, dt_bias, dt_softplus, beta_sigmoid, qk_norm, qk_eps):
    import torch
    code = _dtype_code(v)
    if q.dim() < 2:
        raise ValueError("q must be (..., G, N)")
    lead, (H, P), (G, N) = tuple(v.shape[:-2]), v.shape[-2:], q.shape[-2:]
    dev, t = v.device, v.dtype
    strides = [_row_stride(x, n, lead, tail, t, dev)
               for x, n, tail in ((q, "q", (G, N)), (k, "k", (G, N)), (v, "v", (H, P)), (dt, "dt", (H,)),
                                  (beta, "beta", (H,)))]
    _check(A, "A", (H,), torch.float32, dev)
    _check(dt_bias, "dt_bias", (H,), torch.float32, dev)
    batch, L = lead if len(lead) == 2 else (lead[0], 1)
    return GdrDesc(batch, L, H, P, G, N, code, int(bool(dt_softplus)), int(bool(beta_sigmoid)), int(bool(qk_norm)),
                   float(max(N, 1) ** -0.5 if scale is None else scale), float(qk_eps), *strides,
                   None if dt_bias is None else dt_bias.data_ptr())


def _workspace(workspace, need, device, name, stream, returned=False):
    import torch
    if workspace is None:
        if need == 0:
            return None, 0
        return _empty(need, torch.uint8, device, stream, returned), need
    _check(workspace, "workspace", device=device)
    have = workspace.numel() * workspace.element_size()
    if have < need:
        raise ValueError("workspace has %d bytes, %s needs %d" % (have, name, need))
    return workspace, have


def ssm_gdr_workspace_size(batch, seqlen, nheads, headdim, ngroups, dstate) -> int:
    """Workspace bytes of ssm_gdr_fwd."""
    desc = GdrDesc(batch, seqlen, nheads, headdim, ngroups, dstate, SSM_BF16, 0, 0, 0, 1.0)
    return int(lib().ssm_gdr_workspace_size(ctypes.byref(desc)))


def ssm_gdr_bwd_workspace_size(batch, seqlen, nheads, headdim, ngroups, dstate) -> int:
    """Workspace bytes of ssm_gdr_bwd, ssm_gdr_fwd_save and ssm_gdr_bwd_saved."""
    desc = GdrDesc(batch, seqlen, nheads, headdim, ngroups, dstate, SSM_BF16, 0, 0, 0, 1.0)
    return int(lib().ssm_gdr_bwd_workspace_size(ctypes.byref(desc)))


def ssm_gdr_fwd(q, k, v, dt, beta, A, h0=None, y=None, h_last=None, scale=None, dt_bias=None, dt_softplus=False,
                beta_sigmoid=False, qk_norm=False, qk_eps=1e-6, workspace=None, want_h_last=True, stream=None,
                _save=False):
    """The gated delta rule over a sequence, on device tensors.

    q, k: (batch, L, G, N) bfloat16, N 64 or 128; v: (batch, L, H, P) bfloat16,
    P a multiple of 16 up to 256; dt, beta: (batch, L, H) bfloat16; A, dt_bias:
    (H,) float32; h0: (batch, H, P, N) float32. ``scale`` (of the readout)
    defaults to N ** -0.5. ``dt_softplus`` passes dt + dt_bias through
    softplus, ``beta_sigmoid`` beta through the sigmoid, ``qk_norm`` gives
    queries and keys unit length (``qk_eps`` added to the sum of squares). q,
    k, v, dt and beta may be cut out of wider rows (one projection's output).
    Outputs y (batch, L, H, P) and h_last (batch, H, P, N) are allocated when
    not given. Returns (y, h_last).
    """
    import torch
    if v.dim() != 4:
        raise ValueError("v must be (batch, L, H, P)")
    desc = _gdr_desc(q, k, v, dt, beta, A, scale, dt_bias, dt_softplus, beta_sigmoid, qk_norm, qk_eps)
    batch, L, H, P = v.shape
    N, dev = q.shape[-1], v.device
    _check(h0, "h0", (batch, H, P, N), torch.float32, dev)
    if y is None:
        y = _empty((batch, L, H, P), v.dtype, dev, stream)
    if h_last is None and want_h_last:
        h_last = _empty((batch, H, P, N), torch.float32, dev, stream)
    _check(y, "y", (batch, L, H, P), v.dtype, dev)
    _check(h_last, "h_last", (batch, H, P, N), torch.float32, dev)
    L_ = lib()
    name = "ssm_gdr_fwd_save" if _save else "ssm_gdr_fwd"
    size = L_.ssm_gdr_bwd_workspace_size if _save else L_.ssm_gdr_workspace_size
    workspace, ws_bytes = _workspace(workspace, size(ctypes.byref(desc)), dev, name, stream, _save)
    rc = _on(dev, getattr(L_, name), ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(dt), _ptr(beta), _ptr(A), _ptr(h0),
                           _ptr(y), _ptr(h_last), _ptr(workspace), ws_bytes, _stream(stream, dev))
    if rc != 0:
        raise SsmError(rc, name)
    return (y, h_last, workspace) if _save else (y, h_last)


def ssm_gdr_fwd_save(q, k, v, dt, beta, A, h0=None, y=None, h_last=None, scale=None, dt_bias=None,
                     dt_softplus=False, beta_sigmoid=False, qk_norm=False, qk_eps=1e-6, workspace=None,
                     want_h_last=True, stream=None):
    """ssm_gdr_fwd that also keeps what the backward would first recompute.
    Returns (y, h_last, saved): ``saved`` is the workspace (uint8,
    ssm_gdr_bwd_workspace_size bytes; ``workspace`` if given) to pass unchanged
    to ssm_gdr_bwd_saved with the same inputs."""
    return ssm_gdr_fwd(q, k, v, dt, beta, A, h0, y, h_last, scale, dt_bias, dt_softplus, beta_sigmoid, qk_norm,
                       qk_eps, workspace, want_h_last, stream, _save=True)


def ssm_gdr_bwd(q, k, v, dt, beta, A, dy, h0=None, dh_last=None, scale=None, dt_bias=None, dt_softplus=False,
                beta_sigmoid=False, qk_norm=False, qk_eps=1e-6, workspace=None, want_dh0=True, out=None, stream=None,
                _saved=False):
    """Backward of ssm_gdr_fwd on device tensors.

    Inputs as ssm_gdr_fwd, plus dy (batch, L, H, P) bfloat16 and an optional
    dh_last (batch, H, P, N) float32. Returns a dict with dq, dk, dv, ddt, dbeta
    (bfloat16, of the inputs' shapes), dA (H,), ddt_bias (H,) (with a
    ``dt_bias``) and dh0 (batch, H, P, N) (when ``want_dh0``), float32. ``out``
    may hold preallocated outputs.
    """
    import torch
    if v.dim() != 4:
        raise ValueError("v must be (batch, L, H, P)")
    desc = _gdr_desc(q, k, v, dt, beta, A, scale, dt_bias, dt_softplus, beta_sigmoid, qk_norm, qk_eps)
    batch, L, H, P = v.shape
    G, N = q.shape[-2:]
    dev, t, f32 = v.device, v.dtype, torch.float32
    _check(h0, "h0", (batch, H, P, N), f32, dev)
    _check(dy, "dy", (batch, L, H, P), t, dev)
    _check(dh_last, "dh_last", (batch, H, P, N), f32, dev)
    o = dict(out or {})

    def get(name, shape, dtype, wanted=True):
        if not wanted:
            return None
        if o.get(name) is None:
            o[name] = _empty(shape, dtype, dev, stream)
        _check(o[name], name, shape, dtype, dev)
        return o[name]
    g = dict(dq=get("dq", (batch, L, G, N), t), dk=get("dk", (batch, L, G, N), t), dv=get("dv", (batch, L, H, P), t),
             ddt=get("ddt", (batch, L, H), t), dbeta=get("dbeta", (batch, L, H), t), dA=get("dA", (H,), f32),
             ddt_bias=get("ddt_bias", (H,), f32, dt_bias is not None),
             dh0=get("dh0", (batch, H, P, N), f32, want_dh0))
    L_ = lib()
    name = "ssm_gdr_bwd_saved" if _saved else "ssm_gdr_bwd"
    workspace, ws_bytes = _workspace(workspace, L_.ssm_gdr_bwd_workspace_size(ctypes.byref(desc)), dev, name, stream)
    rc = _on(dev, getattr(L_, name), ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(dt), _ptr(beta), _ptr(A), _ptr(h0),
                           _ptr(dy), _ptr(dh_last), _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["ddt"]),
                           _ptr(g["dbeta"]), _ptr(g["dA"]), _ptr(g["ddt_bias"]), _ptr(g["dh0"]), _ptr(workspace),
                           ws_bytes, _stream(stream, dev))
    if rc != 0:
        raise SsmError(rc, name)
    return g


def ssm_gdr_bwd_saved(q, k, v, dt, beta, A, dy, saved, h0=None, dh_last=None, scale=None, dt_bias=None,
                      dt_softplus=False, beta_sigmoid=False, qk_norm=False, qk_eps=1e-6, want_dh0=True, out=None,
                      stream=None):
    """ssm_gdr_bwd that reads what an ssm_gdr_fwd_save call with the same inputs
    left in ``saved`` (its returned workspace). Arguments and results as
    ssm_gdr_bwd."""
    if saved is None and v.numel() > 0:
        raise ValueError("ssm_gdr_bwd_saved needs the workspace of an ssm_gdr_fwd_save call")
    return ssm_gdr_bwd(q, k, v, dt, beta, A, dy, h0, dh_last, scale, dt_bias, dt_softplus, beta_sigmoid, qk_norm,
                       qk_eps, saved, want_dh0, out, stream, _saved=True)


def ssm_gdr_state_update(q, k, v, dt, beta, A, h, y=None, h_out=None, scale=None, dt_bias=None, dt_softplus=False,
                         beta_sigmoid=False, qk_norm=False, qk_eps=1e-6, stream=None):
    """One token of the gated delta rule: q, k (batch, G, N), v (batch, H, P),
    dt, beta (batch, H) bfloat16; A, dt_bias (H,) float32; options as
    ssm_gdr_fwd. h (batch, H, P, N) float32 is updated in place, or left and
    the new state written to ``h_out``. Returns y (batch, H, P), allocated when
    not given."""
    import torch
    if v.dim() != 3:
        raise ValueError("v must be (batch, H, P)")
    desc = _gdr_desc(q, k, v, dt, beta, A, scale, dt_bias, dt_softplus, beta_sigmoid, qk_norm, qk_eps)
    batch, H, P = v.shape
    N, dev = q.shape[-1], v.device
    _check(h, "h", (batch, H, P, N), torch.float32, dev)
    if h_out is None:
        h_out = h
    _check(h_out, "h_out", (batch, H, P, N), torch.float32, dev)
    if y is None:
        y = _empty((batch, H, P), v.dtype, dev, stream)
    _check(y, "y", (batch, H, P), v.dtype, dev)
    rc = _on(dev, lib().ssm_gdr_state_update, ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(dt), _ptr(beta), _ptr(A),
                                    _ptr(h), _ptr(h_out), _ptr(y), _stream(stream, dev))
    if rc != 0:
        raise SsmError(rc, "ssm_gdr_state_update")
    return y


def ssm_prenorm_fwd(x, weight, residual=None, scale=None, eps=1e-5, y=None, r=None, want_r=True, stream=None):
    """The residual add and RMS norm before a block, on device tensors:
    r = residual + scale * x, y = r / sqrt(mean(r^2) + eps) * weight.

    x: (..., dim) bfloat16 or float32 (rows evenly spaced); residual: the same
    shape, of x's dtype or float32; weight, scale: (dim,) float32. r has
    residual's dtype (x's without one) and y is the norm of r as stored.
    ``r`` may be the residual itself. Returns (y, r); r is None with
    ``want_r`` false.
    """
    import torch
    dim, lead, dev = x.shape[-1], tuple(x.shape[:-1]), x.device
    code = _dtype_code(x)
    xs = _row_stride(x, "x", lead, (dim,), x.dtype, dev)
    rt = x.dtype if residual is None else residual.dtype
    if rt not in (x.dtype, torch.float32):
        raise TypeError("residual must be float32 or of x's dtype, got %s" % rt)
    _check(residual, "residual", x.shape, rt, dev)
    _check(weight, "weight", (dim,), torch.float32, dev)
    _check(scale, "scale", (dim,), torch.float32, dev)
    if y is None:
        y = _empty(x.shape, x.dtype, dev, stream)
    if r is None and want_r:
        r = _empty(x.shape, rt, dev, stream)
    _check(y, "y", x.shape, x.dtype, dev)
    _check(r, "r", x.shape, rt, dev)
    desc = PrenormDesc(x.numel() // dim if dim else 0, dim, code, SSM_F32 if rt == torch.float32 else SSM_BF16,
                       float(eps), 0, xs)
    rc = _on(dev, lib().ssm_prenorm_fwd, ctypes.byref(desc), _ptr(x), _ptr(residual), _ptr(scale), _ptr(weight), _ptr(r),
                               _ptr(y), _stream(stream, dev))
    if rc != 0:
        raise SsmError(rc, "ssm_prenorm_fwd")
    return y, r


def ssm_prenorm_bwd(dy, r, weight, dr=None, x=None, scale=None, eps=1e-5, want_dresidual=True, out=None,
                    workspace=None, stream=None):
    """Backward of ssm_prenorm_fwd. r: what the forward returned; dr: its
    gradient (of r's dtype) or None; x (the forward's) is needed with a
    ``scale``. Returns a dict with dx (dy's dtype), dresidual (r's dtype, when
    wanted), dweight and dscale (with a scale), float32. ``out`` may hold
    preallocated outputs (dresidual may be dr itself)."""
    import torch
    dim, dev = dy.shape[-1], dy.device
    code = _dtype_code(dy)
    rt = r.dtype
    if rt not in (dy.dtype, torch.float32):
        raise TypeError("r must be float32 or of dy's dtype, got %s" % rt)
    _check(dy, "dy", device=dev)
    _check(r, "r", dy.shape, rt, dev)
    _check(dr, "dr", dy.shape, rt, dev)
    _check(weight, "weight", (dim,), torch.float32, dev)
    _check(scale, "scale", (dim,), torch.float32, dev)
    if scale is not None and x is None:
        raise ValueError("the gradient of scale needs x")
    xs = 0 if scale is None else _row_stride(x, "x", tuple(dy.shape[:-1]), (dim,), dy.dtype, dev)
    o = dict(out or {})

    def get(name, shape, dtype, wanted=True):
        if not wanted:
            return None
        if o.get(name) is None:
            o[name] = _empty(shape, dtype, dev, stream)
        _check(o[name], name, shape, dtype, dev)
        return o[name]
    g = dict(dx=get("dx", dy.shape, dy.dtype), dresidual=get("dresidual", dy.shape, rt, want_dresidual),
             dweight=get("dweight", (dim,), torch.float32), dscale=get("dscale", (dim,), torch.float32, scale is not None))
    desc = PrenormDesc(dy.numel() // dim if dim else 0, dim, code, SSM_F32 if rt == torch.float32 else SSM_BF16,
                       float(eps), 0, xs)
    L_ = lib()
    workspace, ws_bytes = _workspace(workspace, L_.ssm_prenorm_bwd_workspace_size(ctypes.byref(desc)), dev,
                                     "ssm_prenorm_bwd", stream)
    rc = _on(dev, L_.ssm_prenorm_bwd, ctypes.byref(desc), _ptr(dy), _ptr(r), _ptr(dr), _ptr(x if scale is not None else None),
                            _ptr(scale), _ptr(weight), _ptr(g["dx"]), _ptr(g["dresidual"]), _ptr(g["dweight"]),
                            _ptr(g["dscale"]), _ptr(workspace), ws_bytes, _stream(stream, dev))
    if rc != 0:
        raise SsmError(rc, "ssm_prenorm_bwd")
    return g


def _gated_desc(x, z, weight, eps, gate_first):
    import torch
    if x.dim() < 2:
        raise ValueError("x must be (..., groups, dim)")
    groups, dim = x.shape[-2:]
    lead, dev = tuple(x.shape[:-2]), x.device
    code = _dtype_code(x)
    xs = _row_stride(x, "x", lead, (groups, dim), x.dtype, dev)
    zs = 0 if z is None else _row_stride(z, "z", lead, (groups, dim), x.dtype, dev)
    shared = weight.dim() == 1
    _check(weight, "weight", (dim,) if shared else (groups, dim), torch.float32, dev)
    width = groups * dim
    return GatedNormDesc(x.numel() // width if width else 0, groups, dim, code, int(bool(gate_first)), int(shared),
                         float(eps), xs, zs)


def ssm_gated_norm_fwd(x, z, weight, eps=1e-5, gate_first=False, y=None, stream=None):
    """The gated RMS norm behind a mixer, on device tensors. Per row and group:
    y = x / sqrt(mean(x^2) + eps) * weight * silu(z), or with ``gate_first``
    the norm of x * silu(z) times weight.

    x, z: (..., groups, dim) bfloat16 or float32 (rows evenly spaced: z may be
    cut out of a projection's output); z None: no gate. weight: (groups, dim)
    or (dim,) for every group, float32. Returns y, allocated when not given.
    """
    desc = _gated_desc(x, z, weight, eps, gate_first)
    if y is None:
        y = _empty(x.shape, x.dtype, x.device, stream)
    _check(y, "y", x.shape, x.dtype, x.device)
    rc = _on(x.device, lib().ssm_gated_norm_fwd, ctypes.byref(desc), _ptr(x), _ptr(z), _ptr(weight), _ptr(y),
                                  _stream(stream, x.device))
    if rc != 0:
        raise SsmError(rc, "ssm_gated_norm_fwd")
    return y


def ssm_gated_norm_bwd(dy, x, z, weight, eps=1e-5, gate_first=False, out=None, workspace=None, stream=None):
    """Backward of ssm_gated_norm_fwd. Returns a dict with dx, dz (x's dtype, dz
    with a gate) and dweight (float32, of weight's shape). ``out`` may hold
    preallocated outputs."""
    import torch
    desc = _gated_desc(x, z, weight, eps, gate_first)
    dev = x.device
    _check(dy, "dy", x.shape, x.dtype, dev)
    o = dict(out or {})

    def get(name, shape, dtype, wanted=True):
        if not wanted:
            return None
        if o.get(name) is None:
            o[name] = _empty(shape, dtype, dev, stream)
        _check(o[name], name, shape, dtype, dev)
        return o[name]
    g = dict(dx=get("dx", x.shape, x.dtype), dz=get("dz", x.shape, x.dtype, z is not None),
             dweight=get("dweight", tuple(weight.shape), torch.float32))
    L_ = lib()
    workspace, ws_bytes = _workspace(workspace, L_.ssm_gated_norm_bwd_workspace_size(ctypes.byref(desc)), dev,
                                     "ssm_gated_norm_bwd", stream)
    rc = _on(dev, L_.ssm_gated_norm_bwd, ctypes.byref(desc), _ptr(dy), _ptr(x), _ptr(z), _ptr(weight), _ptr(g["dx"]),
                               _ptr(g["dz"]), _ptr(g["dweight"]), _ptr(workspace), ws_bytes, _stream(stream, dev))
    if rc != 0:
        raise SsmError(rc, "ssm_gated_norm_bwd")
    return g
