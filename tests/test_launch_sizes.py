"""Launch shapes of the calls around the linears up to their documented sizes
(T < 2^31, m and dim up to 2^24): tests/host_check/launch_check.cpp drives the
built library with the runtime's launch entry replaced, so nothing runs and no
GPU is needed."""
import os
import subprocess

import pytest

from test_host_sanitizers import FLAGS, HIPCC, ROOT

PKG = os.path.join(ROOT, "orthogonal_equivalence_cayley_amd")


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
def test_launches_stay_countable(tmp_path):
    obj, exe = str(tmp_path / "launch_check.o"), str(tmp_path / "launch_check")
    src = os.path.join(ROOT, "tests", "host_check", "launch_check.cpp")
    for cmd in ([HIPCC, "-x", "hip", *FLAGS, "-c", src, "-o", obj],
                [HIPCC, "--offload-arch=gfx950", "-rdynamic", obj, "-L", PKG, "-l:libpoetx.so", f"-Wl,-rpath,{PKG}",
                 "-o", exe]):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert "OK (0 failed checks)" in r.stdout
