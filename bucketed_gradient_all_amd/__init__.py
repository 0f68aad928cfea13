"""Python binding of libddp.so (include/ddp.h): bucketed gradient reduction
for data-parallel training on MI355X (gfx950), the norm and clipping of the
gradients, the AdamW step, the embedding's lookup and gradient, and the layer
norm's two passes.

Argument marshalling only: every step of the path runs in the C++ host
library and its HIP kernels. The functions keep the C names; a negative
status raises DDPError carrying the code and the library's message. There is
no fallback: if libddp.so is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import subprocess
import threading
import weakref
from typing import Callable, List, NamedTuple, Optional, Sequence

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB_PATH = os.path.join(HERE, "libddp.so")
CSRC = os.path.join(HERE, "csrc")

DDP_OK = 0
DDP_ERR_INVALID = -1
DDP_ERR_ALREADY_READY = -2
DDP_ERR_UNFINISHED = -3
DDP_ERR_NOT_READY = -4
DDP_ERR_ORDER = -5
DDP_ERR_HIP = -6
DDP_ERR_HOOK = -7
DDP_ERR_NOMEM = -8

DDP_ORDER_REVERSE = 0
DDP_ORDER_GIVEN = 1
DDP_ORDER_FWD_THEN_REVERSE = 2

DDP_ALL_REDUCE = 0
DDP_REDUCE_SCATTER = 1

DDP_HOOK_ALLREDUCE = 0
DDP_HOOK_BF16_COMPRESS = 1
DDP_HOOK_FP16_COMPRESS = 2

DDP_IN_F32_COPY = 0
DDP_IN_F32_VIEW = 1
DDP_IN_BF16_ACCUM_F32 = 2

DDP_F32 = 0
DDP_BF16 = 1
DDP_F16 = 2

DDP_NORM_INF = 0
DDP_NORM_L1 = 1
DDP_NORM_L2 = 2

DDP_STATE_F32 = 0
DDP_STATE_8BIT = 1
DDP_STATE_BLOCK = 128

DDP_I32 = 0
DDP_I64 = 1

DDP_LAYER_NORM = 0
DDP_RMS_NORM = 1

HIPCC_FLAGS = ["--offload-arch=gfx950", "-O3", "-fPIC", "-std=c++17",
               "-ffp-contract=off", "-fno-fast-math",
               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]

# one object per source; the kernel families compile in parallel
SOURCES = ["reducer.cpp", "grad_list.cpp", "embedding.cpp", "adamw.cpp", "layernorm.cpp",
           "bucket_reduce.hip", "bucket_bf16_hook.hip", "bucket_fp16_hook.hip", "static_tables.hip", "grad_norm.hip",
           "embedding.hip", "embedding_small.hip", "adamw.hip", "layernorm.hip", "layernorm_grad.hip"]
HEADERS = ["host_common.h", "internal.h", "reduce_kernels.h", "static_area.h", "grad_list.h", "embedding.h",
           "embedding_kernels.h", "element.h", "spans.h", "adamw.h", "layernorm.h", "layernorm_kernels.h"]


BUILD_DIR = os.path.join(HERE, "_build")


def resource_report_path(src: str) -> str:
    """Where build() keeps the compiler's per-kernel resource report of a
    kernel source (registers, scratch, occupancy)."""
    return os.path.join(BUILD_DIR, src.replace(".", "_") + ".resources.txt")


def build(verbose: bool = False) -> None:
    """Compile libddp.so in place with hipcc for gfx950. For the kernel
    sources the compiler's resource report is kept beside the objects."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    procs, objs = [], []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".", "_") + ".o")
        cmd = ["/opt/rocm/bin/hipcc", *HIPCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-c", "-o", obj,
               os.path.join(CSRC, src)]
        report = None
        if src.endswith(".hip"):
            cmd.append("-Rpass-analysis=kernel-resource-usage")
            report = open(resource_report_path(src), "w")
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((cmd, subprocess.Popen(cmd, cwd=HERE, stderr=report), report))
        objs.append(obj)
    failed = []
    for cmd, p, report in procs:
        if p.wait() != 0:
            failed.append(cmd)
        if report is not None:
            report.close()
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    cmd = ["/opt/rocm/bin/hipcc", "--offload-arch=gfx950", "-shared", "-fPIC", "-o", LIB_PATH + ".tmp", *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True, cwd=HERE)
    os.replace(LIB_PATH + ".tmp", LIB_PATH)


class DDPError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[{code}] {msg}")
        self.code = code
        self.msg = msg


HOOK_FN = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_int32)


class ddp_reducer_desc(ctypes.Structure):
    _fields_ = [
        ("world", ctypes.c_int32),
        ("n_params", ctypes.c_int32),
        ("param_numel", ctypes.c_void_p),
        ("bucket_of", ctypes.c_void_p),
        ("offset_in_bucket", ctypes.c_void_p),
        ("n_buckets", ctypes.c_int32),
        ("input_mode", ctypes.c_int32),
        ("grads", ctypes.c_void_p),
        ("flat", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("compute_stream", ctypes.c_void_p),
        ("comm_stream", ctypes.c_void_p),
        ("collective", ctypes.c_int32),
        ("find_unused", ctypes.c_int32),
    ]


class ddp_grads_desc(ctypes.Structure):
    _fields_ = [
        ("n_tensors", ctypes.c_int32),
        ("n_copies", ctypes.c_int32),
        ("numel", ctypes.c_void_p),
        ("dtype", ctypes.c_void_p),
        ("grads", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("out_dtype", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
    ]


class ddp_adamw_desc(ctypes.Structure):
    _fields_ = [
        ("n_tensors", ctypes.c_int32),
        ("state", ctypes.c_int32),
        ("numel", ctypes.c_void_p),
        ("grad_dtype", ctypes.c_void_p),
        ("param_dtype", ctypes.c_void_p),
        ("grads", ctypes.c_void_p),
        ("params", ctypes.c_void_p),
        ("copies", ctypes.c_void_p),
        ("copy_dtype", ctypes.c_void_p),
        ("m", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("m_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
        ("weight_decay", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
    ]


class ddp_adamw_args(ctypes.Structure):
    _fields_ = [
        ("lr", ctypes.c_double),
        ("beta1", ctypes.c_double),
        ("beta2", ctypes.c_double),
        ("eps", ctypes.c_double),
        ("step", ctypes.c_int64),
        ("lr_ptr", ctypes.c_void_p),
        ("step_ptr", ctypes.c_void_p),
        ("norm", ctypes.c_void_p),
        ("max_norm", ctypes.c_float),
        ("skip_nonfinite", ctypes.c_int32),
    ]


class ddp_embedding_desc(ctypes.Structure):
    _fields_ = [
        ("n_rows", ctypes.c_int64),
        ("width", ctypes.c_int64),
        ("first_row", ctypes.c_int64),
        ("padding_idx", ctypes.c_int64),
        ("table_stride", ctypes.c_int64),
        ("grad_stride", ctypes.c_int64),
        ("act_stride", ctypes.c_int64),
        ("scale", ctypes.c_float),
        ("index_dtype", ctypes.c_int32),
        ("table_dtype", ctypes.c_int32),
        ("grad_dtype", ctypes.c_int32),
        ("act_dtype", ctypes.c_int32),
    ]


class ddp_layernorm_desc(ctypes.Structure):
    _fields_ = [
        ("width", ctypes.c_int64),
        ("x_stride", ctypes.c_int64),
        ("add_stride", ctypes.c_int64),
        ("z_stride", ctypes.c_int64),
        ("y_stride", ctypes.c_int64),
        ("eps", ctypes.c_float),
        ("kind", ctypes.c_int32),
        ("x_dtype", ctypes.c_int32),
        ("y_dtype", ctypes.c_int32),
        ("weight_dtype", ctypes.c_int32),
        ("grad_dtype", ctypes.c_int32),
    ]


_lib = None


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "(there is no fallback path)")
        L = ctypes.CDLL(LIB_PATH)
        P, I32, I64, F32, SIZE = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        sig = {
            "ddp_plan_buckets": [I32, P, P, I32, I64, I64, P, P, P, P, P, P],
            "ddp_reducer_create": [ctypes.POINTER(ddp_reducer_desc), ctypes.POINTER(ctypes.c_void_p)],
            "ddp_reducer_create_static": [ctypes.POINTER(ddp_reducer_desc), ctypes.POINTER(ctypes.c_void_p)],
            "ddp_reducer_destroy": [P],
            "ddp_prepare_for_backward": [P],
            "ddp_mark_ready": [P, I32],
            "ddp_mark_ready_many": [P, P, I32, P],
            "ddp_bucket_reduce": [P, I32, P],
            "ddp_finish": [P, I32],
            "ddp_register_comm_hook": [P, HOOK_FN, P],
            "ddp_get_bucket": [P, I32, P, P, P],
            "ddp_get_bucket_params": [P, I32, P],
            "ddp_get_ready_order": [P, P, P],
            "ddp_get_launched": [P, P],
            "ddp_set_timing": [P, I32],
            "ddp_get_timings": [P, P, P, P, I32, P],
            "ddp_set_require_sync": [P, I32],
            "ddp_set_local_used": [P, P],
            "ddp_register_builtin_hook": [P, I32],
            "ddp_set_bucket_groups": [P, P, I32],
            "ddp_set_workgroups_per_cu": [P, I32],
            "ddp_get_launch_lds": [P, P],
            "ddp_grads_create": [ctypes.POINTER(ddp_grads_desc), ctypes.POINTER(ctypes.c_void_p)],
            "ddp_grads_from_reducer": [P, P, SIZE, ctypes.POINTER(ctypes.c_void_p)],
            "ddp_grads_destroy": [P],
            "ddp_grads_scratch_bytes": [P, P],
            "ddp_grad_norm": [P, I32, P, P, SIZE, P],
            "ddp_clip_grad_norm": [P, I32, F32, P, P, SIZE, P],
            "ddp_clip_grads": [P, F32, P, P],
            "ddp_adamw_create": [ctypes.POINTER(ddp_adamw_desc), ctypes.POINTER(ctypes.c_void_p)],
            "ddp_adamw_destroy": [P],
            "ddp_adamw_step": [P, ctypes.POINTER(ddp_adamw_args), P],
            "ddp_embedding_lookup": [ctypes.POINTER(ddp_embedding_desc), P, P, I64, P, P],
            "ddp_embedding_grad": [ctypes.POINTER(ddp_embedding_desc), P, P, I64, P, I32, P, SIZE, P],
            "ddp_layernorm": [ctypes.POINTER(ddp_layernorm_desc), I64, P, P, P, P, P, P, P, P, P],
            "ddp_layernorm_grad": [ctypes.POINTER(ddp_layernorm_desc), I64, P, P, P, P, P, P, P, P, P, I32, P, SIZE, P],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        for name, args in {"ddp_workspace_bytes": [ctypes.POINTER(ddp_reducer_desc)],
                           "ddp_grads_workspace_bytes": [ctypes.POINTER(ddp_grads_desc)],
                           "ddp_reducer_grads_workspace_bytes": [P],
                           "ddp_adamw_workspace_bytes": [ctypes.POINTER(ddp_adamw_desc)],
                           "ddp_embedding_grad_workspace_bytes": [ctypes.POINTER(ddp_embedding_desc), I64],
                           "ddp_layernorm_grad_workspace_bytes": [ctypes.POINTER(ddp_layernorm_desc), I64]}.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_size_t
        L.ddp_last_error.argtypes = []
        L.ddp_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def ddp_last_error() -> str:
    return lib().ddp_last_error().decode()


def _check(rc: int, L=None) -> int:
    """Raises DDPError for a failed call; L: the library that made the call
    (its thread's last error text), the loaded one by default."""
    if rc < 0:
        raise DDPError(rc, (L or lib()).ddp_last_error().decode())
    return rc


class BucketPlan(NamedTuple):
    bucket_of: np.ndarray        # [P] int32
    offset_in_bucket: np.ndarray  # [P] int64 bytes
    bucket_params: np.ndarray    # [P] int32, bucket by bucket
    bucket_nparams: np.ndarray   # [B] int32
    bucket_bytes: np.ndarray     # [B] int64
    n_buckets: int

    def buckets(self) -> List[List[int]]:
        out, k = [], 0
        for c in self.bucket_nparams:
            out.append([int(p) for p in self.bucket_params[k:k + c]])
            k += c
        return out


def ddp_plan_buckets(param_bytes: Sequence[int], order_mode: int = DDP_ORDER_REVERSE,
                     cap_bytes: int = 25 << 20, first_cap_bytes: int = 1 << 20,
                     order: Optional[Sequence[int]] = None) -> BucketPlan:
    pb = np.ascontiguousarray(param_bytes, dtype=np.int64).reshape(-1)
    P = pb.size
    od = np.ascontiguousarray(order if order is not None else [], dtype=np.int32).reshape(-1)
    if order is not None and od.size != P:
        raise ValueError(f"order must list all {P} gradients, got {od.size}")
    bucket_of = np.empty(P, np.int32)
    offset = np.empty(P, np.int64)
    bparams = np.empty(P, np.int32)
    bn = np.empty(max(P, 1), np.int32)
    bb = np.empty(max(P, 1), np.int64)
    nb = ctypes.c_int32(0)
    _check(lib().ddp_plan_buckets(P, pb.ctypes.data, od.ctypes.data if order is not None else None, order_mode,
                                  cap_bytes, first_cap_bytes, bucket_of.ctypes.data, offset.ctypes.data,
                                  bparams.ctypes.data, bn.ctypes.data, bb.ctypes.data, ctypes.byref(nb)))
    B = nb.value
    return BucketPlan(bucket_of, offset, bparams, bn[:B].copy(), bb[:B].copy(), B)


class Desc:
    """Owns the host arrays a ddp_reducer_desc points to."""

    def __init__(self, world: int, param_numel: Sequence[int], bucket_of: Sequence[int],
                 offset_in_bucket: Sequence[int], n_buckets: int, input_mode: int = DDP_IN_F32_COPY,
                 grads: Optional[Sequence[Sequence[int]]] = None, flat: Optional[Sequence[int]] = None,
                 workspace: int = 0, workspace_bytes: int = 0, compute_stream: int = 0, comm_stream: int = 0,
                 collective: int = DDP_ALL_REDUCE, find_unused: bool = False):
        self.numel = np.ascontiguousarray(param_numel, dtype=np.int64).reshape(-1)
        self.bucket_of = np.ascontiguousarray(bucket_of, dtype=np.int32).reshape(-1)
        self.offset = np.ascontiguousarray(offset_in_bucket, dtype=np.int64).reshape(-1)
        P = self.numel.size
        if self.bucket_of.size != P or self.offset.size != P:
            raise ValueError(f"bucket_of and offset_in_bucket need {P} entries, got "
                             f"{self.bucket_of.size} and {self.offset.size}")
        self.grads = None
        if grads is not None:
            g = np.asarray(grads, dtype=np.uint64).reshape(-1)
            if g.size != world * P:
                raise ValueError(f"grads needs {world}*{P} pointers, got {g.size}")
            self.grads = np.ascontiguousarray(g if P else np.zeros(1, np.uint64))
        self.flat = None
        if flat is not None:
            self.flat = np.ascontiguousarray(flat, dtype=np.uint64).reshape(-1)
            if self.flat.size != world:
                raise ValueError(f"flat needs {world} pointers, got {self.flat.size}")
        d = ddp_reducer_desc()
        d.world = world
        d.n_params = P
        d.param_numel = self.numel.ctypes.data
        d.bucket_of = self.bucket_of.ctypes.data
        d.offset_in_bucket = self.offset.ctypes.data
        d.n_buckets = n_buckets
        d.input_mode = input_mode
        d.grads = self.grads.ctypes.data if self.grads is not None else None
        d.flat = self.flat.ctypes.data if self.flat is not None else None
        d.workspace = workspace or None
        d.workspace_bytes = workspace_bytes
        d.compute_stream = compute_stream or None
        d.comm_stream = comm_stream or None
        d.collective = collective
        d.find_unused = 1 if find_unused else 0
        self.c = d

    def set_workspace(self, ptr: int, nbytes: int) -> None:
        self.c.workspace = ptr or None
        self.c.workspace_bytes = nbytes


def ddp_workspace_bytes(desc: Desc) -> int:
    n = lib().ddp_workspace_bytes(ctypes.byref(desc.c))
    if n == 0:
        raise DDPError(DDP_ERR_INVALID, ddp_last_error())
    return int(n)


def _release(holder: list, keep, L) -> None:
    """Finalizer of a Reducer dropped without ddp_reducer_destroy: destroys
    the native reducer (which waits for its comm stream) while `keep` (the
    workspace and host tables it reads) is still referenced, so nothing the
    queued reductions use goes back to an allocator first. L is the library
    that created the reducer: only its destroy knows the reducer's layout."""
    h, holder[0] = holder[0], None
    if h:
        L.ddp_reducer_destroy(h)


class Reducer:
    """Handle of a ddp_reducer plus the objects it must keep alive."""

    def __init__(self, handle: int, desc: Desc):
        self._holder = [handle]
        self.desc = desc
        self._hook = None
        self._hook_error: Optional[BaseException] = None
        self.workspace = None
        self._lib = lib()   # the library that created the reducer serves every call on it
        self._finalizer = weakref.finalize(self, _release, self._holder, [desc], self._lib)

    @property
    def handle(self):
        return self._holder[0]

    def keep_alive(self, obj) -> None:
        """Keeps obj (e.g. the device workspace) referenced until the native
        reducer is destroyed, explicitly or by the finalizer."""
        self._finalizer.detach()
        self._finalizer = weakref.finalize(self, _release, self._holder, [self.desc, obj], self._lib)

    def check(self, rc: int) -> int:
        """_check for calls that may run the Python hook: an exception the
        hook raised becomes the cause of the DDPError."""
        err, self._hook_error = self._hook_error, None
        if rc < 0:
            raise DDPError(rc, self._lib.ddp_last_error().decode()) from err
        return rc


def ddp_reducer_create(desc: Desc) -> Reducer:
    h = ctypes.c_void_p()
    _check(lib().ddp_reducer_create(ctypes.byref(desc.c), ctypes.byref(h)))
    return Reducer(h.value, desc)


DDP_STATIC_TABLE_BYTES = 16 << 20


def ddp_reducer_create_static(desc: Desc) -> Reducer:
    """ddp_reducer_create with the device tables in the library's static
    table area (no workspace, no device allocation)."""
    h = ctypes.c_void_p()
    _check(lib().ddp_reducer_create_static(ctypes.byref(desc.c), ctypes.byref(h)))
    return Reducer(h.value, desc)


def ddp_reducer_destroy(r: Reducer) -> None:
    h = r.handle
    if h:
        r._holder[0] = None
        r._finalizer.detach()
        _check(r._lib.ddp_reducer_destroy(h), r._lib)


def ddp_prepare_for_backward(r: Reducer) -> None:
    _check(r._lib.ddp_prepare_for_backward(r.handle), r._lib)


def ddp_mark_ready(r: Reducer, param: int) -> None:
    r.check(r._lib.ddp_mark_ready(r.handle, param))


def ddp_mark_ready_many(r: Reducer, params) -> int:
    """Marks params in order; returns how many were marked (all, unless it raises)."""
    arr = np.ascontiguousarray(params, dtype=np.int32)
    done = ctypes.c_int32()
    rc = r._lib.ddp_mark_ready_many(r.handle, arr.ctypes.data, arr.size, ctypes.byref(done))
    try:
        r.check(rc)
    except DDPError as err:
        err.n_done = done.value
        raise
    return done.value


def ddp_set_require_sync(r: Reducer, sync: bool) -> None:
    _check(r._lib.ddp_set_require_sync(r.handle, 1 if sync else 0), r._lib)


def ddp_set_local_used(r: Reducer, used) -> None:
    """used: [W, P] (or flat W*P) array, nonzero = replica used the gradient."""
    arr = np.asarray(used)
    if arr.dtype != np.uint8:      # the library reads any nonzero byte as "used"
        arr = (arr != 0).astype(np.uint8)
    arr = np.ascontiguousarray(arr).reshape(-1)
    W, P = r.desc.c.world, r.desc.numel.size
    if arr.size != W * P:
        raise ValueError(f"used table must have {W}*{P} entries")
    _check(r._lib.ddp_set_local_used(r.handle, arr.ctypes.data), r._lib)


def ddp_bucket_reduce(r: Reducer, bucket: int, stream: int) -> None:
    _check(r._lib.ddp_bucket_reduce(r.handle, bucket, stream or None), r._lib)


def ddp_finish(r: Reducer, host_blocking: bool = False) -> None:
    r.check(r._lib.ddp_finish(r.handle, 1 if host_blocking else 0))


def ddp_register_comm_hook(r: Reducer, fn: Optional[Callable[[int], int]]) -> None:
    """fn(bucket) -> int (nonzero: failure); None restores the default
    reduction. An exception fn raises fails the call that launched the
    bucket, as a DDPError (DDP_ERR_HOOK) whose cause is that exception."""
    if fn is None:
        r._hook = None
        _check(r._lib.ddp_register_comm_hook(r.handle, HOOK_FN(), None), r._lib)
        return

    def call(ctx, b):
        try:
            return int(fn(b))
        except BaseException as e:   # ctypes would print it and return 0 (success)
            r._hook_error = e
            return -1

    r._hook = HOOK_FN(call)
    _check(r._lib.ddp_register_comm_hook(r.handle, r._hook, None), r._lib)


def ddp_set_bucket_groups(r: Reducer, first_buckets: Sequence[int]) -> None:
    """first_buckets: the first bucket of every group (empty: one group per bucket)."""
    arr = np.ascontiguousarray(np.asarray(list(first_buckets), dtype=np.int32))
    _check(r._lib.ddp_set_bucket_groups(r.handle, arr.ctypes.data if arr.size else None, int(arr.size)),
           r._lib)


def groups_by_bytes(bucket_bytes: Sequence[int], min_group_bytes: int) -> List[int]:
    """First buckets of consecutive groups of at least min_group_bytes each
    (the last group may be smaller)."""
    firsts, acc = [], min_group_bytes
    for b, nb in enumerate(bucket_bytes):
        if acc >= min_group_bytes:
            firsts.append(b)
            acc = 0
        acc += int(nb)
    return firsts


def ddp_set_workgroups_per_cu(r: Reducer, n: int) -> None:
    _check(r._lib.ddp_set_workgroups_per_cu(r.handle, int(n)), r._lib)


def ddp_get_launch_lds(r: Reducer) -> int:
    out = ctypes.c_int32()
    _check(r._lib.ddp_get_launch_lds(r.handle, ctypes.byref(out)), r._lib)
    return out.value


def ddp_register_builtin_hook(r: Reducer, hook: int) -> None:
    _check(r._lib.ddp_register_builtin_hook(r.handle, int(hook)), r._lib)


def ddp_get_bucket(r: Reducer, bucket: int):
    nbytes, off, n = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int32()
    _check(r._lib.ddp_get_bucket(r.handle, bucket, ctypes.byref(nbytes), ctypes.byref(off), ctypes.byref(n)),
           r._lib)
    return nbytes.value, off.value, n.value


def ddp_get_bucket_params(r: Reducer, bucket: int) -> List[int]:
    n = ddp_get_bucket(r, bucket)[2]
    out = np.empty(max(n, 1), np.int32)
    _check(r._lib.ddp_get_bucket_params(r.handle, bucket, out.ctypes.data), r._lib)
    return [int(x) for x in out[:n]]


def ddp_get_ready_order(r: Reducer) -> List[int]:
    out = np.empty(max(r.desc.numel.size, 1), np.int32)
    n = ctypes.c_int32()
    _check(r._lib.ddp_get_ready_order(r.handle, out.ctypes.data, ctypes.byref(n)), r._lib)
    return [int(x) for x in out[:n.value]]


def ddp_get_launched(r: Reducer) -> int:
    n = ctypes.c_int32()
    _check(r._lib.ddp_get_launched(r.handle, ctypes.byref(n)), r._lib)
    return n.value


def ddp_set_timing(r: Reducer, enable: bool) -> None:
    _check(r._lib.ddp_set_timing(r.handle, 1 if enable else 0), r._lib)


def ddp_get_timings(r: Reducer):
    """(first bucket, buckets covered, kernel ms) of every launch since timing
    was enabled, as three arrays."""
    n = ctypes.c_int32()
    _check(r._lib.ddp_get_timings(r.handle, None, None, None, 0, ctypes.byref(n)), r._lib)
    m = max(n.value, 1)
    b, c, ms = np.empty(m, np.int32), np.empty(m, np.int32), np.empty(m, np.float32)
    _check(r._lib.ddp_get_timings(r.handle, b.ctypes.data, c.ctypes.data, ms.ctypes.data, n.value,
                                  ctypes.byref(n)), r._lib)
    k = n.value
    return b[:k].copy(), c[:k].copy(), ms[:k].copy()


def make_reducer(world: int, param_numel: Sequence[int], plan: BucketPlan, input_mode: int,
                 grad_ptrs: Optional[Sequence[Sequence[int]]], flat_ptrs: Sequence[int],
                 compute_stream: int, comm_stream: int, collective: int = DDP_ALL_REDUCE,
                 find_unused: bool = False) -> Reducer:
    """Creates a device reducer; the workspace is a torch allocation kept
    alive by the returned handle."""
    import torch

    desc = Desc(world, param_numel, plan.bucket_of, plan.offset_in_bucket, plan.n_buckets, input_mode,
                grads=grad_ptrs, flat=flat_ptrs, compute_stream=compute_stream, comm_stream=comm_stream,
                collective=collective, find_unused=find_unused)
    nbytes = ddp_workspace_bytes(desc)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    desc.set_workspace(ws.data_ptr(), nbytes)
    r = ddp_reducer_create(desc)
    r.workspace = ws
    r.keep_alive(ws)   # released only after the native reducer, which waits for its reductions
    return r


class GradsDesc:
    """Owns the host arrays a ddp_grads_desc points to. grad_ptrs and out_ptrs:
    one list of device pointers per copy; dtype and out_dtype: DDP_F32 /
    DDP_BF16 / DDP_F16 per tensor (None: fp32, and as dtype)."""

    def __init__(self, numel: Sequence[int], grad_ptrs: Sequence[Sequence[int]],
                 dtype: Optional[Sequence[int]] = None, out_ptrs: Optional[Sequence[Sequence[int]]] = None,
                 out_dtype: Optional[Sequence[int]] = None, workspace: int = 0, workspace_bytes: int = 0):
        self.numel = np.ascontiguousarray(numel, dtype=np.int64).reshape(-1)
        N, R = self.numel.size, len(grad_ptrs)

        def pointers(what, v):
            a = np.asarray([list(c) for c in v], dtype=np.uint64).reshape(-1)
            if a.size != R * N or len(v) != R:
                raise ValueError(f"{what} needs {R} copies of {N} pointers")
            return np.ascontiguousarray(a)

        def types(what, v):
            a = np.ascontiguousarray(v, dtype=np.int32).reshape(-1)
            if a.size != N:
                raise ValueError(f"{what} needs {N} entries, got {a.size}")
            return a

        self.grads = pointers("grad_ptrs", grad_ptrs)
        self.out = pointers("out_ptrs", out_ptrs) if out_ptrs is not None else None
        self.dtype = types("dtype", dtype) if dtype is not None else None
        self.out_dtype = types("out_dtype", out_dtype) if out_dtype is not None else None
        d = ddp_grads_desc()
        d.n_tensors, d.n_copies = N, R
        d.numel = self.numel.ctypes.data
        d.grads = self.grads.ctypes.data
        d.dtype = self.dtype.ctypes.data if self.dtype is not None else None
        d.out = self.out.ctypes.data if self.out is not None else None
        d.out_dtype = self.out_dtype.ctypes.data if self.out_dtype is not None else None
        d.workspace, d.workspace_bytes = workspace or None, workspace_bytes
        self.c = d

    def set_workspace(self, ptr: int, nbytes: int) -> None:
        self.c.workspace = ptr or None
        self.c.workspace_bytes = nbytes


def ddp_grads_workspace_bytes(desc: GradsDesc) -> int:
    n = lib().ddp_grads_workspace_bytes(ctypes.byref(desc.c))
    if n == 0:
        raise DDPError(DDP_ERR_INVALID, ddp_last_error())
    return int(n)


class _ListMemory:
    """The torch allocations of one list, the stream they were allocated on,
    and whether calls were queued on any other."""
    __slots__ = ("tensors", "home", "elsewhere")

    def __init__(self):
        self.tensors, self.home, self.elsewhere = [], 0, False


# Memory of released lists that calls on other streams than its own may still
# read. It waits here for the next list, whose making drains the device. The
# streams themselves are not asked: they are the caller's, named by bare
# handles, and may have been destroyed by now. (An allocator that is told of a
# stream records an event on it when the memory is freed.)
_parked: list = []
_parked_lock = threading.Lock()


def _free_parked() -> None:
    import torch

    with _parked_lock:   # finalizers append meanwhile
        old = list(_parked)
        for device in {t.device for t in old}:
            torch.cuda.synchronize(device)
        del _parked[:len(old)]


def _release_list(holder: list, destroy, memory: _ListMemory) -> None:
    h, holder[0] = holder[0], None
    if h:
        destroy(h)
    if memory.elsewhere:
        _parked.extend(memory.tensors)
    memory.tensors = []


class _List:
    """Handle of a native list of tensors. It may be dropped with calls still
    queued, on any stream; their stream may be gone by then. A graph that
    recorded a call reads the handle's tables at every replay: keep the handle
    as long."""

    _destroy = ""   # name of the library's call that releases the handle

    def __init__(self, handle: int, L=None):
        self._holder = [handle]
        self._lib = L or lib()   # the library that created the list serves every call on it
        self._memory = _ListMemory()          # device allocations that live as long as the handle
        self._finalizer = weakref.finalize(self, _release_list, self._holder, getattr(self._lib, self._destroy),
                                           self._memory)
        self.workspace = None

    @property
    def handle(self):
        return self._holder[0]

    def own(self, *tensors) -> None:
        """Keeps the torch allocations that the list's calls use, the first of
        them its tables, made on the current stream."""
        import torch

        self.workspace = tensors[0]
        self._memory.tensors = list(tensors)
        self._memory.home = torch.cuda.current_stream(self.workspace.device).cuda_stream

    def used_on(self, stream: int) -> None:
        """Notes that a call goes to this stream. Memory used on its own
        stream alone may be freed at once: the allocator hands it out again in
        that stream's order. 1 names the null stream too."""
        if (0 if stream == 1 else stream or 0) != self._memory.home:
            self._memory.elsewhere = True

    def destroy(self) -> None:
        self._finalizer()


class Grads(_List):
    """Handle of a ddp_grads, and the scratch its calls use by default."""

    _destroy = "ddp_grads_destroy"

    def __init__(self, handle: int, L=None):
        super().__init__(handle, L)
        self.scratch = None
        self._scratch = (None, 0)

    def set_scratch(self, ptr: int, nbytes: int) -> None:
        """The scratch of calls that are given none."""
        self._scratch = (ptr or None, nbytes)

    def own(self, workspace, scratch) -> None:
        super().own(workspace, scratch)
        self.scratch = scratch
        self.set_scratch(scratch.data_ptr(), scratch.numel())


def ddp_grads_create(desc: GradsDesc) -> Grads:
    h = ctypes.c_void_p()
    _check(lib().ddp_grads_create(ctypes.byref(desc.c), ctypes.byref(h)))
    return Grads(h.value)


def ddp_reducer_grads_workspace_bytes(r: Reducer) -> int:
    n = r._lib.ddp_reducer_grads_workspace_bytes(r.handle)
    if n == 0:
        raise DDPError(DDP_ERR_INVALID, r._lib.ddp_last_error().decode())
    return int(n)


def ddp_grads_from_reducer(r: Reducer, workspace: int, workspace_bytes: int) -> Grads:
    h = ctypes.c_void_p()
    _check(r._lib.ddp_grads_from_reducer(r.handle, workspace or None, workspace_bytes, ctypes.byref(h)), r._lib)
    return Grads(h.value, r._lib)


def ddp_grads_destroy(g: Grads) -> None:
    g.destroy()


def ddp_grads_scratch_bytes(g: Grads) -> int:
    n = ctypes.c_size_t()
    _check(g._lib.ddp_grads_scratch_bytes(g.handle, ctypes.byref(n)), g._lib)
    return n.value


def ddp_grad_norm(g: Grads, norm_type: int, norm: int, stream: int, scratch: int = 0, scratch_bytes: int = 0) -> None:
    """norm: device pointer of one float. Without a scratch the handle's own
    is used: then no other call of the handle, nor a replay of one, may run at
    the same time."""
    p, n = (scratch, scratch_bytes) if scratch else g._scratch
    g.used_on(stream)
    _check(g._lib.ddp_grad_norm(g.handle, norm_type, norm or None, p, n, stream or None), g._lib)


def ddp_clip_grad_norm(g: Grads, norm_type: int, max_norm: float, norm: int, stream: int, scratch: int = 0,
                       scratch_bytes: int = 0) -> None:
    p, n = (scratch, scratch_bytes) if scratch else g._scratch
    g.used_on(stream)
    _check(g._lib.ddp_clip_grad_norm(g.handle, norm_type, max_norm, norm or None, p, n, stream or None), g._lib)


def ddp_clip_grads(g: Grads, max_norm: float, norm: int, stream: int) -> None:
    g.used_on(stream)
    _check(g._lib.ddp_clip_grads(g.handle, max_norm, norm or None, stream or None), g._lib)


def _idle_workspace(nbytes: int):
    """A torch allocation that no queued work touches any more: the tables are
    uploaded at once, and memory freed on the current stream may still be
    written by kernels queued there."""
    import torch

    _free_parked()
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda.current_stream().synchronize()
    return ws


def _with_scratch(g: Grads, ws) -> Grads:
    import torch
    g.own(ws, torch.empty(ddp_grads_scratch_bytes(g), dtype=torch.uint8, device=ws.device))
    return g


def make_grads(numel: Sequence[int], grad_ptrs: Sequence[Sequence[int]], dtype: Optional[Sequence[int]] = None,
               out_ptrs: Optional[Sequence[Sequence[int]]] = None,
               out_dtype: Optional[Sequence[int]] = None) -> Grads:
    """Creates a gradient list on the current device; its workspace and a
    scratch are torch allocations that the returned handle keeps alive."""
    desc = GradsDesc(numel, grad_ptrs, dtype, out_ptrs, out_dtype)
    nbytes = ddp_grads_workspace_bytes(desc)
    ws = _idle_workspace(nbytes)
    desc.set_workspace(ws.data_ptr(), nbytes)
    return _with_scratch(ddp_grads_create(desc), ws)


def make_reducer_grads(r: Reducer) -> Grads:
    """make_grads over a reducer's results (ddp_grads_from_reducer)."""
    nbytes = ddp_reducer_grads_workspace_bytes(r)
    ws = _idle_workspace(nbytes)
    return _with_scratch(ddp_grads_from_reducer(r, ws.data_ptr(), nbytes), ws)


class AdamWDesc:
    """Owns the host arrays a ddp_adamw_desc points to. Pointers, types and
    decays per tensor; weight_decay may be one number for all; copy_ptrs may
    hold 0 for tensors without a copy."""

    def __init__(self, numel: Sequence[int], grad_ptrs: Sequence[int], param_ptrs: Sequence[int],
                 m_ptrs: Sequence[int], v_ptrs: Sequence[int], grad_dtype: Optional[Sequence[int]] = None,
                 param_dtype: Optional[Sequence[int]] = None, copy_ptrs: Optional[Sequence[int]] = None,
                 copy_dtype: Optional[Sequence[int]] = None, state: int = DDP_STATE_F32,
                 m_scale_ptrs: Optional[Sequence[int]] = None, v_scale_ptrs: Optional[Sequence[int]] = None,
                 weight_decay=None, workspace: int = 0, workspace_bytes: int = 0):
        self.numel = np.ascontiguousarray(numel, dtype=np.int64).reshape(-1)
        N = self.numel.size
        self.arrays = []   # keeps what the desc points to

        def of(what, v, dtype):
            if v is None:
                return None
            a = np.ascontiguousarray(v, dtype=dtype).reshape(-1)
            if a.size != N:
                raise ValueError(f"{what} needs {N} entries, got {a.size}")
            self.arrays.append(a)
            return a.ctypes.data

        if weight_decay is not None and np.ndim(weight_decay) == 0:
            weight_decay = np.full(N, weight_decay, np.float64)
        d = ddp_adamw_desc()
        d.n_tensors, d.state = N, state
        d.numel = self.numel.ctypes.data
        d.grad_dtype = of("grad_dtype", grad_dtype, np.int32)
        d.param_dtype = of("param_dtype", param_dtype, np.int32)
        d.grads = of("grad_ptrs", grad_ptrs, np.uint64)
        d.params = of("param_ptrs", param_ptrs, np.uint64)
        d.copies = of("copy_ptrs", copy_ptrs, np.uint64)
        d.copy_dtype = of("copy_dtype", copy_dtype, np.int32)
        d.m = of("m_ptrs", m_ptrs, np.uint64)
        d.v = of("v_ptrs", v_ptrs, np.uint64)
        d.m_scale = of("m_scale_ptrs", m_scale_ptrs, np.uint64)
        d.v_scale = of("v_scale_ptrs", v_scale_ptrs, np.uint64)
        d.weight_decay = of("weight_decay", weight_decay, np.float64)
        d.workspace, d.workspace_bytes = workspace or None, workspace_bytes
        self.c = d

    def set_workspace(self, ptr: int, nbytes: int) -> None:
        self.c.workspace = ptr or None
        self.c.workspace_bytes = nbytes


class AdamW(_List):
    """Handle of a ddp_adamw."""

    _destroy = "ddp_adamw_destroy"


def ddp_adamw_workspace_bytes(desc: AdamWDesc) -> int:
    n = lib().ddp_adamw_workspace_bytes(ctypes.byref(desc.c))
    if n == 0:
        raise DDPError(DDP_ERR_INVALID, ddp_last_error())
    return int(n)


def ddp_adamw_create(desc: AdamWDesc) -> AdamW:
    h = ctypes.c_void_p()
    _check(lib().ddp_adamw_create(ctypes.byref(desc.c), ctypes.byref(h)))
    return AdamW(h.value)


def ddp_adamw_destroy(o: AdamW) -> None:
    o.destroy()


def ddp_adamw_step(o: AdamW, lr: float, step: int, stream: int, beta1: float = 0.9, beta2: float = 0.999,
                   eps: float = 1e-8, max_norm: float = math.inf, norm: int = 0, skip_nonfinite: bool = False,
                   lr_ptr: int = 0, step_ptr: int = 0) -> None:
    """norm, lr_ptr and step_ptr: device pointers (float, float, int64); with
    the last two lr and step are not read. Without max_norm a norm does not clip."""
    a = ddp_adamw_args(lr, beta1, beta2, eps, step, lr_ptr or None, step_ptr or None, norm or None, max_norm,
                       1 if skip_nonfinite else 0)
    o.used_on(stream)
    _check(o._lib.ddp_adamw_step(o.handle, ctypes.byref(a), stream or None), o._lib)


def make_adamw(numel: Sequence[int], grad_ptrs: Sequence[int], param_ptrs: Sequence[int], m_ptrs: Sequence[int],
               v_ptrs: Sequence[int], **kw) -> AdamW:
    """Creates an AdamW list on the current device from AdamWDesc's arguments;
    its workspace is a torch allocation that the returned handle keeps alive."""
    desc = AdamWDesc(numel, grad_ptrs, param_ptrs, m_ptrs, v_ptrs, **kw)
    nbytes = ddp_adamw_workspace_bytes(desc)
    ws = _idle_workspace(nbytes)
    desc.set_workspace(ws.data_ptr(), nbytes)
    o = ddp_adamw_create(desc)
    o.own(ws)
    return o


class EmbeddingDesc:
    """A ddp_embedding_desc; strides default to the width."""

    def __init__(self, n_rows: int, width: int, table_dtype: int = DDP_F32, grad_dtype: int = DDP_F32,
                 act_dtype: int = DDP_F32, index_dtype: int = DDP_I64, scale: float = 1.0, first_row: int = 0,
                 padding_idx: int = -1, table_stride: Optional[int] = None, grad_stride: Optional[int] = None,
                 act_stride: Optional[int] = None):
        d = ddp_embedding_desc()
        d.n_rows, d.width, d.first_row, d.padding_idx = n_rows, width, first_row, padding_idx
        d.table_stride = width if table_stride is None else table_stride
        d.grad_stride = width if grad_stride is None else grad_stride
        d.act_stride = width if act_stride is None else act_stride
        d.scale = scale
        d.index_dtype, d.table_dtype, d.grad_dtype, d.act_dtype = index_dtype, table_dtype, grad_dtype, act_dtype
        self.c = d


def ddp_embedding_lookup(desc: EmbeddingDesc, table: int, tokens: int, n_tokens: int, out: int, stream: int) -> None:
    _check(lib().ddp_embedding_lookup(ctypes.byref(desc.c), table or None, tokens or None, n_tokens, out or None,
                                      stream or None))


def ddp_embedding_grad_workspace_bytes(desc: EmbeddingDesc, n_tokens: int) -> int:
    n = lib().ddp_embedding_grad_workspace_bytes(ctypes.byref(desc.c), n_tokens)
    if n == 0:
        raise DDPError(DDP_ERR_INVALID, ddp_last_error())
    return int(n)


def ddp_embedding_grad(desc: EmbeddingDesc, dout: int, tokens: int, n_tokens: int, grad: int, accumulate: bool,
                       workspace: int, workspace_bytes: int, stream: int) -> None:
    _check(lib().ddp_embedding_grad(ctypes.byref(desc.c), dout or None, tokens or None, n_tokens, grad or None,
                                    1 if accumulate else 0, workspace or None, workspace_bytes, stream or None))


class LayerNormDesc:
    """A ddp_layernorm_desc; strides default to the width."""

    def __init__(self, width: int, kind: int = DDP_LAYER_NORM, x_dtype: int = DDP_F32, y_dtype: Optional[int] = None,
                 weight_dtype: int = DDP_F32, grad_dtype: int = DDP_F32, eps: float = 1e-5,
                 x_stride: Optional[int] = None, add_stride: Optional[int] = None, z_stride: Optional[int] = None,
                 y_stride: Optional[int] = None):
        d = ddp_layernorm_desc()
        d.width, d.eps, d.kind = width, eps, kind
        d.x_stride = width if x_stride is None else x_stride
        d.add_stride = width if add_stride is None else add_stride
        d.z_stride = width if z_stride is None else z_stride
        d.y_stride = width if y_stride is None else y_stride
        d.x_dtype, d.y_dtype = x_dtype, x_dtype if y_dtype is None else y_dtype
        d.weight_dtype, d.grad_dtype = weight_dtype, grad_dtype
        self.c = d


def ddp_layernorm(desc: LayerNormDesc, n_rows: int, x: int, weight: int, bias: int, y: int, stream: int, add: int = 0,
                  z: int = 0, mean: int = 0, rstd: int = 0) -> None:
    _check(lib().ddp_layernorm(ctypes.byref(desc.c), n_rows, x or None, add or None, weight or None, bias or None,
                               z or None, y or None, mean or None, rstd or None, stream or None))


def ddp_layernorm_grad_workspace_bytes(desc: LayerNormDesc, n_rows: int) -> int:
    n = lib().ddp_layernorm_grad_workspace_bytes(ctypes.byref(desc.c), n_rows)
    if n == 0:
        raise DDPError(DDP_ERR_INVALID, ddp_last_error())
    return int(n)


def ddp_layernorm_grad(desc: LayerNormDesc, n_rows: int, dy: int, z: int, weight: int, mean: int, rstd: int, dx: int,
                       dweight: int, dbias: int, accumulate: bool, workspace: int, workspace_bytes: int, stream: int,
                       dz: int = 0) -> None:
    _check(lib().ddp_layernorm_grad(ctypes.byref(desc.c), n_rows, dy or None, z or None, dz or None, weight or None,
                                    mean or None, rstd or None, dx or None, dweight or None, dbias or None,
                                    1 if accumulate else 0, workspace or None, workspace_bytes, stream or None))
