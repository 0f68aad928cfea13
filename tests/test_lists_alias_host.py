"""Gradient lists in unsafe places, on the CPU: calls that would write over what
they read, and lists made on another device than their reducer's. The host
sources run under AddressSanitizer and UndefinedBehaviorSanitizer with
stand-ins for the HIP runtime and the kernel launchers."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "bucketed_gradient_all_amd", "csrc")
NATIVE = os.path.join(ROOT, "tests", "native")


def run_native(tmp_path, name, sources, extra=()):
    """Builds tests/native/<name>.cpp with the library's host sources and runs it."""
    if shutil.which("g++") is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime_api.h"):
        pytest.skip("needs g++ and the ROCm headers")
    exe = tmp_path / name
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-static-libasan", "-static-libubsan", "-D__HIP_PLATFORM_AMD__",
           "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", NATIVE,
           *(os.path.join(CSRC, s) for s in sources), os.path.join(NATIVE, "fake_hip.cpp"),
           os.path.join(NATIVE, name + ".cpp"),
           "-Wl,--wrap=_Znwm,--wrap=_Znam,--wrap=_ZnwmRKSt9nothrow_t,--wrap=_ZnamRKSt9nothrow_t", *extra, "-o", str(exe)]
    subprocess.run(cmd, check=True, timeout=600)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=600, env=env)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert f"{name} ok" in r.stdout


def test_a_norm_or_a_scratch_over_what_a_call_reads_is_refused(tmp_path):
    run_native(tmp_path, "list_alias_checks", ["reducer.cpp", "grad_list.cpp"])


def test_the_list_of_a_reducer_is_made_on_its_device(tmp_path):
    run_native(tmp_path, "list_device_checks", ["reducer.cpp", "grad_list.cpp"], ["-Wl,--wrap=hipGetDevice"])
