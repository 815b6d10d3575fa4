"""The host side of the attention-layer entry points under AddressSanitizer and
UndefinedBehaviorSanitizer (host code only), driven by tests/sanitize/layer_driver.c through
workspace queries and rejected calls over shapes up to and past the limits."""
import os
import shutil
import tempfile
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_oracle_sanitized import CSRC, HIPCC, ROOT, SAN, _clean, _env, _run

SOURCES = ["jb_api", "jb_layer", "jb_attn", "jb_rope", "jb_gen", "jb_prefill", "jb_fwd", "jb_decode", "jb_proj",
           "jb_backward"]


@pytest.mark.skipif(not os.path.exists(HIPCC) or shutil.which("nm") is None, reason="hipcc not available")
def test_layer_host_code_under_asan_ubsan():
    host_san = [f for s in SAN for f in ("-Xarch_host", s)]
    common = [HIPCC, "--offload-arch=gfx950", "-O1", "-Xarch_host", "-g", "-fno-omit-frame-pointer",
              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-fno-sanitize-recover=all", *host_san]
    with tempfile.TemporaryDirectory() as d:
        def obj(name):
            o = os.path.join(d, name + ".o")
            _run([*common, "-std=c++17", "-fPIC", "-c", os.path.join(CSRC, name + ".hip"), "-o", o])
            return o
        with ThreadPoolExecutor(min(len(SOURCES), os.cpu_count() or 1)) as ex:
            objs = list(ex.map(obj, SOURCES))
        drv, exe = os.path.join(d, "layer_driver.o"), os.path.join(d, "layer_driver")
        _run(["/opt/rocm/llvm/bin/clang", "-std=c11", "-O1", "-g", "-fno-omit-frame-pointer", *SAN,
              "-fno-sanitize-recover=all", "-c", os.path.join(ROOT, "tests", "sanitize", "layer_driver.c"), "-o", drv])
        _run([*common, "-o", exe, drv, *objs, "-Wl,-rpath,/opt/rocm/lib"])
        r = _run([exe], env=_env(), timeout=300)
        _clean(r)
        if r.stdout.startswith("skipped"):
            pytest.skip(r.stdout.strip())
        assert "checks passed" in r.stdout, r.stdout
