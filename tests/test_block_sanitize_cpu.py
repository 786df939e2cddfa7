"""The host code of the gated linear recurrence, the projections and the clipping of
gradients under AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU alone:
its units are compiled for the host only and linked with a driver
(tests/sanitize/block_driver.cpp) that stands in for the HIP runtime, checks the shape
of every launch, and makes seeded random calls over sizes at which something changes
or overflows."""
from __future__ import annotations

import os
import re

import pytest

from test_sanitize_cpu import CSRC, HERE, HOST_SAN, ROOT, RUN_ENV, _need, _run


def test_host_code_under_sanitizers(tmp_path):
    hipcc, nm = _need("hipcc"), _need("nm")
    flags = ["--offload-arch=gfx950", "--offload-host-only", "-O1", "-g", "-std=c++17", "-fPIC", *HOST_SAN,
             "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    objects, link = [], []
    for name in ("glr", "grad", "proj"):
        obj = tmp_path / (name + ".o")
        r = _run([hipcc, *flags, "-c", "-o", obj, os.path.join(CSRC, name + ".hip")], timeout=600)
        assert r.returncode == 0, r.stderr[-4000:]
        objects.append(obj)
        # the device code that a host-only object expects at its side, and nobody looks at here
        link += ["-Wl,--defsym=%s=0" % s for s in set(re.findall(r"U (__hip_fatbin_\w+)", _run([nm, obj]).stdout))]
    drv, exe = tmp_path / "block_driver.o", tmp_path / "block_san"
    r = _run([hipcc, *flags, "-x", "hip", "-c", "-o", drv, os.path.join(HERE, "block_driver.cpp")])
    assert r.returncode == 0, r.stderr[-4000:]
    cxx = os.path.join(os.path.dirname(os.path.realpath(hipcc)), "..", "lib", "llvm", "bin", "clang++")
    if not os.path.exists(cxx):
        pytest.skip("no clang++ beside hipcc")
    r = _run([cxx, "-fsanitize=" + ",".join(("address", "undefined")), "-o", exe, drv, *objects, *link])
    assert r.returncode == 0, r.stderr[-4000:]
    r = _run([exe], env=RUN_ENV)
    assert r.returncode == 0, (r.stdout + r.stderr)[-6000:]
    assert "all calls clean" in r.stdout
