"""The AdamW step on the CPU: workspace sizes, every refusal that comes before a
device is touched, the binding's own checks, and the host source under
AddressSanitizer and UndefinedBehaviorSanitizer with stand-ins for the HIP
runtime and the kernel's launcher."""
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
G, P, M, V, C, MS, VS, WS = (0x10000000 * (k + 1) for k in range(8))


def _desc(numel=(64,), **kw):
    n = len(numel)
    at = {"grad_ptrs": G, "param_ptrs": P, "m_ptrs": M, "v_ptrs": V}
    args = {k: [a + 4096 * i for i in range(n)] for k, a in at.items()}
    args.update({"workspace": WS, "workspace_bytes": 1 << 30}, **kw)
    return ddp.AdamWDesc(list(numel), **args)


def _small(numel=(64,), **kw):
    n = len(numel)
    return _desc(numel, **{"state": ddp.DDP_STATE_8BIT, "m_scale_ptrs": [MS + 256 * i for i in range(n)],
                           "v_scale_ptrs": [VS + 256 * i for i in range(n)], **kw})


def _refused(fn, text):
    with pytest.raises(ddp.DDPError) as e:
        fn()
    assert e.value.code == ddp.DDP_ERR_INVALID, e.value
    assert text in e.value.msg, e.value.msg


def test_workspace_grows_with_the_list():
    size = ddp.ddp_adamw_workspace_bytes
    assert 0 < size(_desc([])) < size(_desc([100])) < size(_desc([100] * 50))
    assert size(_desc([1 << 30])) >= 4 * (1 << 30) // 2048
    assert size(_small([100])) == size(_desc([100]))


@pytest.mark.parametrize("numel,kw,text", [
    ([-1], {}, "bad size"),
    ([1 << 60], {}, "bad size"),
    ([1 << 50], {}, "too many elements"),
    ([4], {"grad_dtype": [7]}, "unknown type"),
    ([4], {"param_dtype": [-1]}, "unknown type"),
    ([4], {"state": 2}, "unknown state"),
    ([4], {"copy_ptrs": [C]}, "go together"),
    ([4], {"copy_dtype": [1]}, "go together"),
    ([4], {"weight_decay": [-0.1]}, "weight decay"),
    ([4], {"weight_decay": math.inf}, "weight decay"),
    ([4], {"weight_decay": math.nan}, "weight decay"),
])
def test_sizes_types_and_decays_are_checked(numel, kw, text):
    desc = _desc(numel, **kw)
    _refused(lambda: ddp.ddp_adamw_workspace_bytes(desc), text)
    _refused(lambda: ddp.ddp_adamw_create(desc), text)


@pytest.mark.parametrize("make,kw,text", [
    (_desc, {"workspace": 0}, "workspace missing"),
    (_desc, {"workspace": WS + 8}, "workspace missing"),
    (_desc, {"grad_ptrs": [0]}, "tensor 0's gradient is NULL"),
    (_desc, {"param_ptrs": [0]}, "tensor 0's parameter is NULL"),
    (_desc, {"m_ptrs": [0]}, "tensor 0's m is NULL"),
    (_desc, {"v_ptrs": [0]}, "tensor 0's v is NULL"),
    (_desc, {"grad_ptrs": [G + 2]}, "gradient is misaligned"),
    (_desc, {"grad_ptrs": [G + 1], "grad_dtype": [1]}, "gradient is misaligned"),
    (_desc, {"param_ptrs": [P + 2]}, "parameter is misaligned"),
    (_desc, {"param_ptrs": [P + 1], "param_dtype": [2]}, "parameter is misaligned"),
    (_desc, {"m_ptrs": [M + 2]}, "m is misaligned"),
    (_desc, {"v_ptrs": [V + 1]}, "v is misaligned"),
    (_desc, {"copy_ptrs": [C + 1], "copy_dtype": [1]}, "copy is misaligned"),
    (_desc, {"copy_ptrs": [C], "copy_dtype": [0]}, "copy must be"),
    (_desc, {"copy_ptrs": [C], "copy_dtype": [3]}, "copy must be"),
    (_desc, {"copy_ptrs": [C], "copy_dtype": [1], "param_dtype": [1]}, "copy must be"),
    (_desc, {"m_ptrs": None}, "grads, params, m or v is NULL"),
    (_desc, {"m_scale_ptrs": [MS], "v_scale_ptrs": [VS]}, "go with 8-bit states"),
    (_desc, {"v_scale_ptrs": [VS]}, "go with 8-bit states"),
    (_small, {"m_scale_ptrs": None}, "go with 8-bit states"),
    (_small, {"v_scale_ptrs": None}, "go with 8-bit states"),
    (_small, {"m_scale_ptrs": [0]}, "m_scale is NULL"),
    (_small, {"v_scale_ptrs": [VS + 2]}, "v_scale is misaligned"),
])
def test_pointers_are_checked(make, kw, text):
    _refused(lambda: ddp.ddp_adamw_create(make([64], **kw)), text)


def test_a_workspace_that_is_too_small_is_refused():
    need = ddp.ddp_adamw_workspace_bytes(_desc())
    _refused(lambda: ddp.ddp_adamw_create(_desc(workspace_bytes=need - 1)), "workspace missing")


@pytest.mark.parametrize("make,kw,text", [
    (_desc, {"param_ptrs": [G]}, "overlap"),
    (_desc, {"param_ptrs": [G + 252]}, "overlap"),
    (_desc, {"m_ptrs": [V]}, "m and tensor 0's v overlap"),
    (_desc, {"m_ptrs": [P - 252]}, "overlap"),
    (_desc, {"copy_ptrs": [G + 128], "copy_dtype": [1]}, "overlap"),
    (_desc, {"workspace": G}, "the workspace"),
    (_desc, {"workspace": V}, "the workspace"),
    (_small, {"m_ptrs": [V + 63]}, "overlap"),
    (_small, {"m_scale_ptrs": [VS]}, "m_scale and tensor 0's v_scale overlap"),
    (_small, {"v_scale_ptrs": [M + 60]}, "overlap"),
])
def test_ranges_that_overlap_are_refused(make, kw, text):
    _refused(lambda: ddp.ddp_adamw_create(make([64], **kw)), text)


def test_tensors_that_share_memory_are_refused():
    _refused(lambda: ddp.ddp_adamw_create(_desc([64, 64], param_ptrs=[P, P])), "overlap")
    _refused(lambda: ddp.ddp_adamw_create(_desc([64, 64], grad_ptrs=[G, G + 128], m_ptrs=[M, G + 380])), "overlap")
    _refused(lambda: ddp.ddp_adamw_create(_desc([64, 64], grad_ptrs=[G, G], m_ptrs=[M, G])), "overlap")
    _refused(lambda: ddp.ddp_adamw_create(_desc([6400, 64], grad_ptrs=[G, G + 64], m_ptrs=[M + 65536, G + 20000])), "overlap")
    _refused(lambda: ddp.ddp_adamw_create(_small([129, 64], m_scale_ptrs=[MS, MS + 4])), "overlap")


def test_the_binding_checks_lengths():
    for kw in ({"grad_ptrs": [G, G]}, {"param_dtype": [0, 0]}, {"copy_ptrs": [C], "copy_dtype": []},
               {"weight_decay": [0.1, 0.1]}, {"m_scale_ptrs": []}):
        with pytest.raises(ValueError):
            _desc([4], **kw)


def test_null_arguments_are_refused():
    L = ddp.lib()
    assert L.ddp_adamw_workspace_bytes(None) == 0
    assert L.ddp_adamw_create(None, None) == ddp.DDP_ERR_INVALID
    assert L.ddp_adamw_step(None, None, None) == ddp.DDP_ERR_INVALID
    assert L.ddp_adamw_destroy(None) == ddp.DDP_OK


def test_the_header_is_c(tmp_path):
    """A C program that names every type and entry point of the step compiles."""
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    src = tmp_path / "use.c"
    src.write_text("""#include "ddp.h"
int use(void) {
    ddp_adamw_desc d = {0}; ddp_adamw_args a = {0}; ddp_adamw *o = 0;
    size_t n = ddp_adamw_workspace_bytes(&d) + DDP_STATE_BLOCK;
    d.state = DDP_STATE_8BIT; d.workspace_bytes = n;
    return ddp_adamw_create(&d, &o) + ddp_adamw_step(o, &a, 0) + ddp_adamw_destroy(o) + DDP_STATE_F32;
}
""")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), "-c", str(src),
                    "-o", str(tmp_path / "use.o")], check=True, timeout=120)


def test_the_structs_match_the_header(tmp_path):
    """Sizes and last offsets of the binding's structures are the header's."""
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    src = tmp_path / "sizes.c"
    src.write_text("""#include "ddp.h"
#include <stdio.h>
int main(void) {
    printf("%zu %zu %zu %zu\\n", sizeof(ddp_adamw_desc), offsetof(ddp_adamw_desc, workspace_bytes),
           sizeof(ddp_adamw_args), offsetof(ddp_adamw_args, skip_nonfinite));
    return 0;
}
""")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True, timeout=120)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    import ctypes
    assert got == [ctypes.sizeof(ddp.ddp_adamw_desc), ddp.ddp_adamw_desc.workspace_bytes.offset,
                   ctypes.sizeof(ddp.ddp_adamw_args), ddp.ddp_adamw_args.skip_nonfinite.offset]


def test_host_source_under_sanitizers(tmp_path):
    if shutil.which("g++") is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime_api.h"):
        pytest.skip("needs g++ and the ROCm headers")
    exe = tmp_path / "adamw_host_checks"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-static-libasan", "-static-libubsan", "-D__HIP_PLATFORM_AMD__",
           "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", NATIVE,
           os.path.join(CSRC, "adamw.cpp"), os.path.join(NATIVE, "adamw_host_checks.cpp"),
           "-Wl,--wrap=_Znwm,--wrap=_Znam,--wrap=_ZnwmRKSt9nothrow_t,--wrap=_ZnamRKSt9nothrow_t", "-o", str(exe)]
    subprocess.run(cmd, check=True, timeout=600)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=600, env=env)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "adamw_host_checks ok" in r.stdout


class _Allocation:
    device = "cuda:0"

    def data_ptr(self):
        return 0x100

    def numel(self):
        return 64


@pytest.mark.parametrize("streams,waits", [((), False), ((0x7000,), False), ((0x7000, 0x9000), True), ((0,), True)])
@pytest.mark.parametrize("destroy", [False, True])
def test_tables_of_a_dropped_list_wait_for_other_streams(monkeypatch, streams, waits, destroy):
    """As the gradient lists' do: memory used on its own stream alone is freed
    at once, any other waits for the device."""
    import gc
    import types

    import torch
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=0x7000))
    monkeypatch.setattr(ddp, "_parked", [])
    o, tables = ddp.AdamW(0), _Allocation()
    o.own(tables)
    for s in streams:
        _refused(lambda: ddp.ddp_adamw_step(o, 1e-3, 1, s), "NULL argument")   # notes the stream first
    if destroy:
        ddp.ddp_adamw_destroy(o)
        ddp.ddp_adamw_destroy(o)
    else:
        del o
        gc.collect()
    assert ddp._parked == ([tables] if waits else [])
