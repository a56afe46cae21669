"""The host code of the calls that train around the linears: launch shapes up to the
documented sizes (the runtime's launch entry replaced, nothing runs), and the whole under
AddressSanitizer and UndefinedBehaviorSanitizer (no GPU visible)."""
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_host_sanitizers import CSRC, FLAGS, HIPCC, ROOT, SAN

PKG = os.path.join(ROOT, "orthogonal_equivalence_cayley_amd")


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
def test_launches_stay_countable(tmp_path):
    obj, exe = str(tmp_path / "check.o"), str(tmp_path / "check")
    src = os.path.join(ROOT, "tests", "host_check", "train_launch_check.cpp")
    for cmd in ([HIPCC, "-x", "hip", *FLAGS, "-c", src, "-o", obj],
                [HIPCC, "--offload-arch=gfx950", "-rdynamic", obj, "-L", PKG, "-l:libpoetx.so", f"-Wl,-rpath,{PKG}",
                 "-o", exe]):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert "OK (0 failed checks)" in r.stdout


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
def test_host_code_under_asan_and_ubsan(tmp_path):
    srcs = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".hip", ".cpp")))
    srcs.append(os.path.join(ROOT, "tests", "host_check", "train_ops_check.cpp"))

    def one(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        r = subprocess.run([HIPCC, "-x", "hip", *FLAGS, *SAN, "-c", src, "-o", obj], capture_output=True, text=True)
        assert r.returncode == 0, f"{src}: {r.stderr[-2000:]}"
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(one, srcs))
    exe = str(tmp_path / "train_ops_check")
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", *SAN, *objs, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    if r.returncode == 77:
        pytest.skip("the driver runs only where no GPU is visible")
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "OK (0 failed checks)" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
