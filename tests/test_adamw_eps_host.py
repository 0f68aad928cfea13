"""The eps that an AdamW step takes, on the CPU: with 8-bit states the divisor
must stay below 2^126, so eps is at most 2^125 there."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "bucketed_gradient_all_amd", "csrc")
NATIVE = os.path.join(ROOT, "tests", "native")


def test_eps_by_the_size_of_the_states(tmp_path):
    if shutil.which("g++") is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime_api.h"):
        pytest.skip("needs g++ and the ROCm headers")
    exe = tmp_path / "adamw_eps_checks"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-static-libasan", "-static-libubsan", "-D__HIP_PLATFORM_AMD__",
           "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", NATIVE,
           os.path.join(CSRC, "adamw.cpp"), os.path.join(NATIVE, "adamw_eps_checks.cpp"),
           "-Wl,--wrap=_Znwm,--wrap=_Znam,--wrap=_ZnwmRKSt9nothrow_t,--wrap=_ZnamRKSt9nothrow_t", "-o", str(exe)]
    subprocess.run(cmd, check=True, timeout=600)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "adamw_eps_checks ok" in r.stdout
