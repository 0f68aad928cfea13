"""Gradient lists and embedding operators on the CPU: workspace sizes, every
refusal that comes before a device is touched, the binding's own checks, and
the host sources under AddressSanitizer and UndefinedBehaviorSanitizer with
stand-ins for the HIP runtime and the kernel launchers."""
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
A, B, WS = 0x10000000, 0x20000000, 0x70000000


def _create(numel, ptrs, ws=WS, ws_bytes=1 << 30, **kw):
    return ddp.ddp_grads_create(ddp.GradsDesc(numel, ptrs, workspace=ws, workspace_bytes=ws_bytes, **kw))


def _refused(fn, text):
    with pytest.raises(ddp.DDPError) as e:
        fn()
    assert e.value.code == ddp.DDP_ERR_INVALID, e.value
    assert text in e.value.msg, e.value.msg


def test_list_workspace_grows_with_the_list():
    one = ddp.ddp_grads_workspace_bytes(ddp.GradsDesc([100], [[A]]))
    assert one >= 32 + 4
    copies = ddp.ddp_grads_workspace_bytes(ddp.GradsDesc([100], [[A], [B]]))
    many = ddp.ddp_grads_workspace_bytes(ddp.GradsDesc([100] * 50, [[A] * 50]))
    large = ddp.ddp_grads_workspace_bytes(ddp.GradsDesc([1 << 30], [[A]]))
    assert one < copies < many and large >= 4 * (1 << 30) // 8192
    assert ddp.ddp_grads_workspace_bytes(ddp.GradsDesc([], [[]])) > 0


@pytest.mark.parametrize("numel,kw,text", [
    ([-1], {}, "bad size"),
    ([1 << 60], {}, "bad size"),
    ([1 << 50], {}, "too many elements"),
    ([4], {"dtype": [7]}, "unknown type"),
    ([4], {"dtype": [-1]}, "unknown type"),
    ([4], {"out_ptrs": [[B]], "out_dtype": [3]}, "unknown type"),
    ([4], {"out_dtype": [0]}, "out_dtype is given without out"),
])
def test_list_sizes_and_types_are_checked(numel, kw, text):
    desc = ddp.GradsDesc(numel, [[A]], **kw)
    _refused(lambda: ddp.ddp_grads_workspace_bytes(desc), text)
    _refused(lambda: _create(numel, [[A]], **kw), text)


def test_list_workspace_and_pointers_are_checked():
    need = ddp.ddp_grads_workspace_bytes(ddp.GradsDesc([64], [[A]]))
    _refused(lambda: _create([64], [[A]], ws=0), "workspace missing")
    _refused(lambda: _create([64], [[A]], ws=WS + 8), "workspace missing")
    _refused(lambda: _create([64], [[A]], ws_bytes=need - 1), "workspace missing")
    _refused(lambda: _create([64], [[0]]), "NULL pointer")
    _refused(lambda: _create([64], [[A + 2]]), "misaligned")
    _refused(lambda: _create([64], [[A + 1]], dtype=[ddp.DDP_BF16]), "misaligned")
    _refused(lambda: _create([64], [[A]], out_ptrs=[[0]]), "NULL pointer")
    _refused(lambda: _create([64], [[A]], out_ptrs=[[B + 2]]), "misaligned")


def test_a_workspace_that_overlaps_a_tensor_is_refused():
    """Its upload would overwrite the gradient."""
    need = ddp.ddp_grads_workspace_bytes(ddp.GradsDesc([64], [[A]]))
    for ws in (A, A + 240, A - need // 16 * 16 + 16):
        _refused(lambda: _create([64], [[A]], ws=ws), "the workspace and gradient 0 overlap")
    _refused(lambda: _create([64], [[A]], out_ptrs=[[B]], ws=B), "the workspace and gradient 0 overlap")
    _refused(lambda: _create([64, 64], [[B, A]], ws=A), "the workspace and gradient 1 overlap")


def test_list_tensors_that_overlap_are_refused():
    _refused(lambda: _create([64, 64], [[A, A]]), "overlap")
    _refused(lambda: _create([64, 64], [[A, A + 252]]), "overlap")
    _refused(lambda: _create([64], [[A], [A]]), "overlap")
    _refused(lambda: _create([64], [[A]], out_ptrs=[[A]]), "overlap")
    _refused(lambda: _create([64], [[A], [B]], out_ptrs=[[B], [A + 4096]]), "overlap")
    _refused(lambda: _create([64], [[A]], out_ptrs=[[A + 128]], out_dtype=[ddp.DDP_BF16]), "overlap")


def test_list_binding_checks_lengths():
    with pytest.raises(ValueError):
        ddp.GradsDesc([4, 4], [[A]])
    with pytest.raises(ValueError):
        ddp.GradsDesc([4], [[A]], dtype=[0, 0])
    with pytest.raises(ValueError):
        ddp.GradsDesc([4], [[A]], out_ptrs=[[B], [B]])
    with pytest.raises(ValueError):
        ddp.GradsDesc([4], [[A]], out_ptrs=[[B]], out_dtype=[])


def test_list_calls_refuse_null_handles():
    L = ddp.lib()
    for rc in (L.ddp_grad_norm(None, ddp.DDP_NORM_L2, A, B, 1 << 20, None),
               L.ddp_clip_grad_norm(None, ddp.DDP_NORM_L2, 1.0, A, B, 1 << 20, None),
               L.ddp_clip_grads(None, 1.0, A, None), L.ddp_grads_scratch_bytes(None, None),
               L.ddp_grads_from_reducer(None, None, 0, None), L.ddp_grads_create(None, None)):
        assert rc == ddp.DDP_ERR_INVALID
    assert L.ddp_grads_destroy(None) == ddp.DDP_OK
    assert L.ddp_grads_workspace_bytes(None) == 0
    assert L.ddp_reducer_grads_workspace_bytes(None) == 0


def test_list_of_a_reducer_without_a_device_is_refused():
    desc = ddp.Desc(2, [16], [0], [0], 1)
    r = ddp.ddp_reducer_create(desc)
    _refused(lambda: ddp.ddp_reducer_grads_workspace_bytes(r), "no device")
    _refused(lambda: ddp.ddp_grads_from_reducer(r, WS, 1 << 20), "no device")
    ddp.ddp_reducer_destroy(r)


# ---------------------------------------------------------------- embedding
def _desc(**kw):
    return ddp.EmbeddingDesc(**{"n_rows": 100, "width": 64, **kw})


@pytest.mark.parametrize("kw,text", [
    ({"n_rows": -1}, "n_rows"), ({"n_rows": (1 << 31) - 1}, "n_rows"),
    ({"first_row": (1 << 63) - 100}, "first_row"), ({"first_row": (1 << 63) - 1}, "first_row"),
    ({"width": -1}, "width"), ({"width": 1 << 31}, "width"),
    ({"index_dtype": 2}, "index type"), ({"table_dtype": 3}, "element type"), ({"grad_dtype": -1}, "element type"),
    ({"act_dtype": 9}, "element type"), ({"table_stride": 63}, "table_stride"), ({"grad_stride": 63}, "grad_stride"),
    ({"table_stride": (1 << 31) + 1}, "table_stride"), ({"act_stride": -1}, "act_stride"),
    ({"act_stride": (1 << 31) + 1}, "act_stride"), ({"scale": math.nan}, "scale"),
])
def test_embedding_descs_are_checked(kw, text):
    d = _desc(**kw)
    _refused(lambda: ddp.ddp_embedding_lookup(d, A, B, 4, WS, 0), text)
    _refused(lambda: ddp.ddp_embedding_grad_workspace_bytes(d, 4), text)
    _refused(lambda: ddp.ddp_embedding_grad(d, A, B, 4, WS, True, WS, 1 << 30, 0), text)


@pytest.mark.parametrize("n", [-1, (1 << 30) + 1])
def test_embedding_token_counts_are_checked(n):
    d = _desc()
    _refused(lambda: ddp.ddp_embedding_lookup(d, A, B, n, WS, 0), "n_tokens")
    _refused(lambda: ddp.ddp_embedding_grad_workspace_bytes(d, n), "n_tokens")
    _refused(lambda: ddp.ddp_embedding_grad(d, A, B, n, WS, True, WS, 1 << 30, 0), "n_tokens")


def test_embedding_pointers_are_checked():
    d = _desc()
    for args, text in (((0, B, 4, WS), "table is NULL"), ((A, 0, 4, WS), "tokens is NULL"), ((A, B, 4, 0), "out is NULL"),
                       ((A + 2, B, 4, WS), "table is misaligned"), ((A, B + 4, 4, WS), "tokens is misaligned"),
                       ((A, B, 4, WS + 1), "out is misaligned")):
        _refused(lambda: ddp.ddp_embedding_lookup(d, *args, 0), text)
    big = 1 << 30
    for args, text in (((0, B, 4, A, True, WS, big), "dout is NULL"), ((A, 0, 4, A, True, WS, big), "tokens is NULL"),
                       ((A, B, 4, 0, True, WS, big), "grad is NULL"), ((A, B, 4, A + 2, True, WS, big), "grad is mis"),
                       ((A, B, 4, A, True, 0, big), "workspace missing"),
                       ((A, B, 4, A, True, WS + 16, big), "workspace missing"),
                       ((A, B, 4, A, True, WS, ddp.ddp_embedding_grad_workspace_bytes(d, 4) - 1), "workspace missing")):
        _refused(lambda: ddp.ddp_embedding_grad(d, *args, 0), text)
    _refused(lambda: ddp.ddp_embedding_lookup(_desc(act_stride=63), A, B, 2, WS, 0), "act_stride")
    L = ddp.lib()
    assert L.ddp_embedding_lookup(None, A, B, 1, WS, None) == ddp.DDP_ERR_INVALID
    assert L.ddp_embedding_grad(None, A, B, 1, A, 1, WS, 1 << 20, None) == ddp.DDP_ERR_INVALID
    assert L.ddp_embedding_grad_workspace_bytes(None, 1) == 0


def test_embedding_calls_too_large_for_a_launch_are_refused():
    wide = _desc(n_rows=10, width=(1 << 31) - 1)
    _refused(lambda: ddp.ddp_embedding_lookup(wide, A, B, 100, WS, 0), "too large")
    _refused(lambda: ddp.ddp_embedding_grad(wide, A, B, 1, A, True, WS, 1 << 62, 0), "too large")
    long = _desc(n_rows=10, width=1 << 20)
    _refused(lambda: ddp.ddp_embedding_grad(long, A, B, 1 << 30, A, True, WS, 1 << 62, 0), "too large")


def test_embedding_calls_with_nothing_to_do_touch_no_device():
    ddp.ddp_embedding_lookup(_desc(), 0, 0, 0, 0, 0)
    ddp.ddp_embedding_lookup(_desc(width=0), 0, 0, 5, 0, 0)
    ddp.ddp_embedding_grad(_desc(), 0, 0, 0, 0, True, 0, 0, 0)
    ddp.ddp_embedding_grad(_desc(width=0), 0, 0, 5, 0, False, 0, 0, 0)
    ddp.ddp_embedding_grad(_desc(n_rows=0), 0, 0, 5, 0, False, 0, 0, 0)


@pytest.mark.parametrize("width,act", [(1, 0), (64, 1), (512, 0), (2048, 1), (20000, 2)])
def test_embedding_workspace_serves_every_shorter_call(width, act):
    """The size for n positions is enough for any fewer: shorter calls are cut
    into shorter chunks, so their number does not simply fall."""
    d = _desc(width=width, act_dtype=act)
    last = 0
    for n in [0, 1, 7, 8, 9, 1000, 8191, 8192, 8193] + [1 << k for k in range(14, 21)]:
        size = ddp.ddp_embedding_grad_workspace_bytes(d, n)
        assert size >= last
        last = size
    # about a quarter of the positions' rows of fp32 at most
    n = 1 << 20
    assert ddp.ddp_embedding_grad_workspace_bytes(d, n) <= n // 4 * 4 * (width + 3) + 8 * n + 4 * 101 + 8 * 256


def test_the_header_is_c(tmp_path):
    """A C program that names every new type and entry point compiles."""
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    src = tmp_path / "use.c"
    src.write_text("""#include "ddp.h"
int use(void) {
    ddp_grads_desc g = {0}; ddp_embedding_desc e = {0}; ddp_grads *l = 0; size_t n = 0; float norm = 0;
    int rc = ddp_grads_create(&g, &l) + ddp_grads_from_reducer(0, 0, 0, &l) + ddp_grads_scratch_bytes(l, &n);
    n += ddp_grads_workspace_bytes(&g) + ddp_reducer_grads_workspace_bytes(0);
    rc += ddp_grad_norm(l, DDP_NORM_L2, &norm, 0, 0, 0) + ddp_clip_grad_norm(l, DDP_NORM_INF, 1.0f, &norm, 0, n, 0);
    rc += ddp_clip_grads(l, 1.0f, &norm, 0) + ddp_grads_destroy(l);
    n += ddp_embedding_grad_workspace_bytes(&e, 1);
    return rc + ddp_embedding_lookup(&e, 0, 0, 0, 0, 0) + ddp_embedding_grad(&e, 0, 0, 0, 0, DDP_BF16, 0, n, 0);
}
""")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), "-c", str(src),
                    "-o", str(tmp_path / "use.o")], check=True, timeout=120)


def test_host_sources_under_sanitizers(tmp_path):
    if shutil.which("g++") is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime_api.h"):
        pytest.skip("needs g++ and the ROCm headers")
    exe = tmp_path / "list_host_checks"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-static-libasan", "-static-libubsan", "-D__HIP_PLATFORM_AMD__",
           "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", NATIVE,
           os.path.join(CSRC, "reducer.cpp"), os.path.join(CSRC, "grad_list.cpp"), os.path.join(CSRC, "embedding.cpp"),
           os.path.join(NATIVE, "fake_hip.cpp"), os.path.join(NATIVE, "list_host_checks.cpp"),
           "-Wl,--wrap=_Znwm,--wrap=_Znam,--wrap=_ZnwmRKSt9nothrow_t,--wrap=_ZnamRKSt9nothrow_t", "-o", str(exe)]
    subprocess.run(cmd, check=True, timeout=600)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=600, env=env)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "list_host_checks ok" in r.stdout
