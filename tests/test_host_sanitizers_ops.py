"""The host code of the calls around the linears under AddressSanitizer and
UndefinedBehaviorSanitizer, driven by tests/host_check/ops_check.cpp (no GPU
visible, nothing launched)."""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_host_sanitizers import CSRC, FLAGS, HIPCC, ROOT, SAN


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
def test_ops_host_code_under_asan_and_ubsan(tmp_path):
    srcs = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".hip", ".cpp")))
    srcs.append(os.path.join(ROOT, "tests", "host_check", "ops_check.cpp"))

    def one(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        r = subprocess.run([HIPCC, "-x", "hip", *FLAGS, *SAN, "-c", src, "-o", obj], capture_output=True, text=True)
        assert r.returncode == 0, f"{src}: {r.stderr[-2000:]}"
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(one, srcs))
    exe = str(tmp_path / "ops_check")
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", *SAN, *objs, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    sys.stdout.write(r.stdout[-4000:])
    if r.returncode == 77:
        pytest.skip("the driver runs only where no GPU is visible")
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "OK (0 failed checks)" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
