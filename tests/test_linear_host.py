"""The projections' argument checks under sanitizers (host code, no GPU): linear_api.cpp with launchers that only count."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"), reason="needs g++ and the ROCm headers")
def test_argument_checks_under_sanitizers(tmp_path):
    src, exe = os.path.join(ROOT, "state_space_recurrence_amd", "csrc"), str(tmp_path / "linear_api_checks")
    cmd = ["g++", "-std=c++17", "-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
           "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
           "-I" + src, os.path.join(src, "linear_api.cpp"), os.path.join(ROOT, "tests", "sanitize", "linear_api_checks.cpp"),
           "-o", exe]
    for c in (cmd, [exe]):
        r = subprocess.run(c, capture_output=True, text=True, timeout=300, env={**os.environ, "ASAN_OPTIONS": "detect_leaks=0"})
        assert r.returncode == 0, f"{' '.join(c)}\n{r.stdout}\n{r.stderr}"
    assert "0 failed" in r.stdout
