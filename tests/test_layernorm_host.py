"""The layer norm on the CPU: every refusal that comes before a device is
touched, workspace sizes, and the host source under AddressSanitizer and
UndefinedBehaviorSanitizer with stand-ins for the HIP runtime and the launchers."""
import ctypes
import math
import os
import shutil
import subprocess

import pytest

import bucketed_gradient_all_amd as ddp
from conftest import ROOT

CSRC = os.path.join(ROOT, "bucketed_gradient_all_amd", "csrc")
NATIVE = os.path.join(ROOT, "tests", "native")

# addresses that no call on the CPU ever reads
X, ADD, W, B, Z, Y, MEAN, RSTD, DX, DW, DB, WS = (0x10000000 * (k + 1) for k in range(12))
BIG = 1 << 40


def _desc(width=64, **kw):
    return ddp.LayerNormDesc(width, **kw)


def _forward(d, n=4, **kw):
    a = {"x": X, "weight": W, "bias": B, "y": Y, "add": ADD, "z": Z, "mean": MEAN, "rstd": RSTD, **kw}
    ddp.ddp_layernorm(d, n, a["x"], a["weight"], a["bias"], a["y"], 0, add=a["add"], z=a["z"], mean=a["mean"],
                      rstd=a["rstd"])


def _backward(d, n=4, accumulate=True, ws_bytes=BIG, **kw):
    a = {"dy": Y, "z": Z, "weight": W, "mean": MEAN, "rstd": RSTD, "dx": DX, "dweight": DW, "dbias": DB, "dz": ADD,
         "ws": WS, **kw}
    ddp.ddp_layernorm_grad(d, n, a["dy"], a["z"], a["weight"], a["mean"], a["rstd"], a["dx"], a["dweight"], a["dbias"],
                           accumulate, a["ws"], ws_bytes, 0, dz=a["dz"])


def _refused(fn, text):
    with pytest.raises(ddp.DDPError) as e:
        fn()
    assert e.value.code == ddp.DDP_ERR_INVALID, e.value
    assert text in e.value.msg, e.value.msg


@pytest.mark.parametrize("width,kw,text", [
    (-1, {}, "width"), ((1 << 26) + 1, {}, "width"),
    (64, {"kind": 2}, "unknown kind"), (64, {"kind": -1}, "unknown kind"),
    (64, {"x_dtype": 3, "y_dtype": 0}, "element type"), (64, {"y_dtype": -1}, "element type"),
    (64, {"weight_dtype": 5}, "element type"), (64, {"grad_dtype": 3}, "element type"),
    (64, {"x_dtype": 1, "y_dtype": 0}, "y_dtype must be"), (64, {"x_dtype": 1, "y_dtype": 2}, "y_dtype must be"),
    (64, {"eps": -1e-5}, "eps"), (64, {"eps": math.inf}, "eps"), (64, {"eps": math.nan}, "eps"),
    (64, {"x_stride": -1}, "strides"), (64, {"add_stride": (1 << 31) + 1}, "strides"),
    (64, {"z_stride": -64}, "strides"), (64, {"y_stride": 1 << 40}, "strides"),
])
def test_descs_are_checked(width, kw, text):
    d = _desc(width, **kw)
    _refused(lambda: _forward(d), text)
    _refused(lambda: ddp.ddp_layernorm_grad_workspace_bytes(d, 4), text)
    _refused(lambda: _backward(d), text)


@pytest.mark.parametrize("n", [-1, 1 << 31])
def test_row_counts_are_checked(n):
    _refused(lambda: _forward(_desc(), n), "n_rows")
    _refused(lambda: ddp.ddp_layernorm_grad_workspace_bytes(_desc(), n), "n_rows")
    _refused(lambda: _backward(_desc(), n), "n_rows")


def test_offsets_past_64_bits_are_refused():
    for name in ("x_stride", "add_stride", "z_stride", "y_stride"):
        d = _desc(**{name: 1 << 31})
        _refused(lambda: _forward(d, (1 << 31) - 1), "too large")
        _refused(lambda: _backward(d, (1 << 31) - 1), "too large")


@pytest.mark.parametrize("kw,text", [
    ({"x": 0}, "x is NULL"), ({"y": 0}, "y is NULL"), ({"x": X + 2}, "x is misaligned"), ({"y": Y + 1}, "y is misaligned"),
    ({"add": ADD + 2}, "add is misaligned"), ({"z": Z + 2}, "z is misaligned"), ({"weight": W + 2}, "weight is misaligned"),
    ({"bias": B + 3}, "bias is misaligned"), ({"mean": MEAN + 2}, "mean is misaligned"),
    ({"rstd": RSTD + 1}, "rstd is misaligned"), ({"add": 0}, "z is given without add"),
    ({"y": Z}, "overlap"), ({"mean": RSTD}, "overlap"), ({"mean": X + 256}, "mean and x overlap"),
    ({"rstd": W}, "rstd and weight overlap"), ({"y": B}, "y and bias overlap"), ({"y": X + 4}, "y and x overlap"),
    ({"z": X + 128}, "z and x overlap"), ({"z": ADD - 4}, "z and add overlap"), ({"y": X, "z": X}, "overlap"),
])
def test_forward_pointers_are_checked(kw, text):
    _refused(lambda: _forward(_desc(), **kw), text)


@pytest.mark.parametrize("kw,text", [
    ({"dy": 0}, "dy is NULL"), ({"z": 0}, "z is NULL"), ({"mean": 0}, "mean is NULL"), ({"rstd": 0}, "rstd is NULL"),
    ({"dy": Y + 2}, "dy is misaligned"), ({"z": Z + 2}, "z is misaligned"), ({"dz": ADD + 2}, "dz is misaligned"),
    ({"dx": DX + 2}, "dx is misaligned"), ({"dweight": DW + 2}, "dweight is misaligned"),
    ({"dbias": DB + 1}, "dbias is misaligned"), ({"weight": W + 2}, "weight is misaligned"),
    ({"rstd": RSTD + 2}, "rstd is misaligned"),
    ({"ws": 0}, "workspace missing"), ({"ws": WS + 64}, "workspace missing"),
    ({"dx": Z}, "dx and z overlap"), ({"dx": Y + 256}, "dx and dy overlap"), ({"dx": ADD + 4}, "dx and dz overlap"),
    ({"dweight": DB}, "overlap"), ({"dweight": W}, "dweight and weight overlap"), ({"dbias": DX + 64}, "overlap"),
    ({"dweight": MEAN}, "dweight and mean overlap"), ({"ws": Z}, "workspace and z overlap"),
    ({"ws": DX}, "overlap"), ({"ws": DW}, "overlap"), ({"ws": RSTD}, "workspace and rstd overlap"),
])
def test_backward_pointers_are_checked(kw, text):
    _refused(lambda: _backward(_desc(), **kw), text)


def test_a_workspace_that_is_too_small_is_refused():
    need = ddp.ddp_layernorm_grad_workspace_bytes(_desc(), 4)
    _refused(lambda: _backward(_desc(), ws_bytes=need - 1), "workspace missing")


def test_strides_below_the_width_are_refused_for_outputs():
    for kw in ({"x_stride": 63}, {"y_stride": 63}, {"y_stride": 0}, {"z_stride": 63}):
        _refused(lambda: _forward(_desc(**kw)), "at least the width")
    _refused(lambda: _backward(_desc(x_stride=63)), "at least the width")


def test_rows_that_interleave():
    """Of one stride: apart where their columns are; of two: taken to meet."""
    wide = {"x_stride": 256, "y_stride": 256}
    for off, meets in ((64 * 4, False), (64 * 4 - 4, True), (192 * 4, False), (193 * 4, True), (256 * 4, True)):
        if meets:
            _refused(lambda: _forward(_desc(**wide), y=X + off, add=0, z=0), "y and x overlap")
    _refused(lambda: _forward(_desc(x_stride=256, y_stride=128), y=X + 256, add=0, z=0), "y and x overlap")
    # the same address with another stride or another element size is not the same place
    _refused(lambda: _forward(_desc(x_stride=64, y_stride=128), y=X, add=0, z=0), "y and x overlap")
    _refused(lambda: _forward(_desc(y_dtype=1), y=X, add=0, z=0), "y and x overlap")
    _refused(lambda: _backward(_desc(y_stride=0), dx=Y), "dx and dy overlap")


def test_calls_with_nothing_to_do_touch_no_device():
    zeros = dict.fromkeys(("x", "weight", "bias", "y", "add", "z", "mean", "rstd"), 0)
    _forward(_desc(), 0, **zeros)
    _forward(_desc(0), 5, **zeros)
    none = dict.fromkeys(("dy", "z", "weight", "mean", "rstd", "dx", "dweight", "dbias", "dz", "ws"), 0)
    _backward(_desc(), 0, **none)
    _backward(_desc(0), 5, False, **none)
    _backward(_desc(), 5, **{**none, "dy": Y, "z": Z, "rstd": RSTD})
    _backward(_desc(), 0, True, **{**none, "dweight": DW})


@pytest.mark.parametrize("width,x", [(1, 0), (64, 1), (512, 0), (2048, 1), (20000, 2), (1 << 20, 0)])
def test_workspace_serves_every_shorter_call(width, x):
    last = 0
    for n in [0, 1, 3, 4, 5, 100, 511, 512, 513, 2047, 2048, 2049, 100000, (1 << 31) - 1]:
        size = ddp.ddp_layernorm_grad_workspace_bytes(_desc(width, x_dtype=x), n)
        assert size >= last
        last = size
    assert last <= 512 * 8 * width + 512


def test_null_descs_are_refused():
    L = ddp.lib()
    assert L.ddp_layernorm(None, 1, X, None, None, None, None, Y, None, None, None) == ddp.DDP_ERR_INVALID
    assert L.ddp_layernorm_grad_workspace_bytes(None, 1) == 0
    assert L.ddp_layernorm_grad(None, 1, Y, Z, None, None, None, RSTD, DX, None, None, 0, None, 0,
                                None) == ddp.DDP_ERR_INVALID


def _gcc(tmp_path, name, source, *flags):
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    src, out = tmp_path / (name + ".c"), tmp_path / name
    src.write_text(source)
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), *flags, str(src), "-o", str(out)], check=True, timeout=120)
    return str(out)


def test_the_header_is_c(tmp_path):
    """A C program that names every type and entry point of the layer norm compiles."""
    _gcc(tmp_path, "use.o", """#include "ddp.h"
int use(void) {
    ddp_layernorm_desc d = {0};
    size_t n = ddp_layernorm_grad_workspace_bytes(&d, 1);
    d.kind = DDP_RMS_NORM;
    return ddp_layernorm(&d, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0) + DDP_LAYER_NORM
        + ddp_layernorm_grad(&d, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 1, 0, n, 0);
}
""", "-std=c99", "-Wall", "-Werror", "-pedantic", "-c")


def test_the_struct_matches_the_header(tmp_path):
    exe = _gcc(tmp_path, "sizes", """#include "ddp.h"
#include <stdio.h>
int main(void) {
    printf("%zu %zu %zu\\n", sizeof(ddp_layernorm_desc), offsetof(ddp_layernorm_desc, eps),
           offsetof(ddp_layernorm_desc, grad_dtype));
    return 0;
}
""")
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    T = ddp.ddp_layernorm_desc
    assert got == [ctypes.sizeof(T), T.eps.offset, T.grad_dtype.offset]


def test_host_source_under_sanitizers(tmp_path):
    if shutil.which("g++") is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime_api.h"):
        pytest.skip("needs g++ and the ROCm headers")
    exe = tmp_path / "layernorm_host_checks"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-static-libasan", "-static-libubsan", "-D__HIP_PLATFORM_AMD__",
           "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", NATIVE,
           os.path.join(CSRC, "layernorm.cpp"), os.path.join(NATIVE, "layernorm_host_checks.cpp"),
           "-Wl,--wrap=_Znwm,--wrap=_Znam,--wrap=_ZnwmRKSt9nothrow_t,--wrap=_ZnamRKSt9nothrow_t", "-o", str(exe)]
    subprocess.run(cmd, check=True, timeout=600)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=600, env=env)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "layernorm_host_checks ok" in r.stdout
