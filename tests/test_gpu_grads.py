"""GPU: the norm of a gradient list and its clipping against the formulas in 64
bits, over tensor sizes around the tiles, odd addresses, mixed types, copies,
second buffers, infinities and NaN; a reducer's list after both collectives;
graphs and streams; refusals.

Tolerances, set before the first run. u = eps / 2 of a type is its largest
relative rounding.
  norm   sums run in 64 bits, so only the final rounding to fp32 counts: u32,
         and the same again for what 64-bit sums of up to 2^24 terms lose
         (2^24 * 2^-53 < u32).
  clip   f = max_norm / (norm + 1e-6): the norm (2 u32 by the line above), the
         bound given as fp32 (u32), the sum and the quotient (u32 each), then
         the product g * f (u32): 6 u32. A narrower output adds its own
         rounding u. Below the smallest normal value a rounding is absolute:
         half the smallest subnormal.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


def _torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def _lib():
    import bucketed_gradient_all_amd as ddp
    return ddp


def _types(torch):
    ddp = _lib()
    return {ddp.DDP_F32: torch.float32, ddp.DDP_BF16: torch.bfloat16, ddp.DDP_F16: torch.float16}


HALF_SUBNORMAL = {"torch.float32": 2.0 ** -150, "torch.bfloat16": 2.0 ** -134, "torch.float16": 2.0 ** -25}


def say(*a):
    print(*a, flush=True)


class Case:
    """Tensors at odd places of one buffer a copy, guarded on both sides."""

    def __init__(self, numel, dtype=None, copies=1, out=None, seed=0, sigma=1.0, gap=3):
        torch, ddp = _torch(), _lib()
        types = _types(torch)
        self.numel = list(numel)
        self.dtype = list(dtype) if dtype is not None else [ddp.DDP_F32] * len(self.numel)
        self.out_dtype = list(out) if out is not None else None
        g = torch.Generator().manual_seed(seed)
        self.values = [(torch.randn(n, generator=g, dtype=torch.float64) * sigma).to(types[t])
                       for n, t in zip(self.numel, self.dtype)]
        self.copies = copies
        self.bufs, self.views = self._place(self.values, self.dtype, gap)
        self.out_views = None
        if out is not None:
            blank = [torch.full((n,), 7.0, dtype=types[t]) for n, t in zip(self.numel, out)]
            self.out_bufs, self.out_views = self._place(blank, out, gap + 2)

    def _place(self, values, dtype, gap):
        torch = _torch()
        bufs, views = [], []
        for _ in range(self.copies):
            mine_b, mine_v = [], []
            for i, v in enumerate(values):
                b = torch.full((v.numel() + 2 * gap + i,), 9.0, dtype=v.dtype)
                b[gap + i:gap + i + v.numel()] = v
                b = b.cuda()
                mine_b.append(b)
                mine_v.append(b[gap + i:gap + i + v.numel()])
            bufs.append(mine_b)
            views.append(mine_v)
        return bufs, views

    def make(self):
        ddp = _lib()
        ptrs = [[v.data_ptr() for v in vs] for vs in self.views]
        out = [[v.data_ptr() for v in vs] for vs in self.out_views] if self.out_views else None
        return ddp.make_grads(self.numel, ptrs, self.dtype, out, self.out_dtype)

    def guards_hold(self):
        """Every element of the buffers outside the tensors still holds its filler."""
        for bufs, views, filler in ((self.bufs, self.views, 9.0),) + (
                ((self.out_bufs, self.out_views, 9.0),) if self.out_views else ()):
            for bs, vs in zip(bufs, views):
                for b, v in zip(bs, vs):
                    at = v.storage_offset()
                    assert bool((b[:at] == filler).all()) and bool((b[at + v.numel():] == filler).all())

    def flat64(self):
        torch = _torch()
        return torch.cat([v.double() for v in self.values]) if self.values else torch.zeros(0, dtype=torch.float64)


def ref_norm(x, kind):
    ddp = _lib()
    if x.numel() == 0:
        return 0.0
    if kind == ddp.DDP_NORM_INF:
        return float(x.abs().max()) if not bool(x.isnan().any()) else math.nan
    return float(x.abs().sum()) if kind == ddp.DDP_NORM_L1 else float(x.square().sum().sqrt())


def new_norm():
    return _torch().full((), -5.0, dtype=_torch().float32, device="cuda")


def check_norm(got, want):
    if math.isnan(want):
        assert math.isnan(got)
    elif math.isinf(want) or want > 3.4028235677973366e38:
        assert got == math.inf
    else:
        assert abs(got - want) <= 2 * U32 * want + 2.0 ** -150, (got, want)


def check_clip(case, norm64, max_norm):
    torch = _torch()
    f = min(1.0, max_norm / (norm64 + 1e-6))
    for views in (case.out_views or case.views):
        for v, x in zip(views, case.values):
            want = x.double() * f
            got = v.cpu().double()
            u = torch.finfo(v.dtype).eps / 2 if v.dtype != torch.float32 else 0.0
            tol = want.abs() * (6 * U32 + u) * (1 + 1e-3) + HALF_SUBNORMAL[str(v.dtype)] + 2.0 ** -149
            bad = (got - want).abs() > tol
            assert not bool(bad.any()), (v.dtype, got[bad][:4], want[bad][:4])


LISTS = {
    "empty": [],
    "nothing": [0, 0],
    "one": [1],
    "few": [1, 0, 2, 3, 5],
    "tile_edges": [8191, 8192, 8193, 127, 128, 129],
    "small_edge": [3 * 8192 - 200],
    "past_small": [7 * 8192, 17],
    "norm_edge": [11 * 8192 - 200, 5],
    "mixed_sizes": [100003, 64, 1, 0, 30000, 8192 * 9 + 5],
    "many": [(i * 37) % 1100 for i in range(700)],
}


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("name", sorted(LISTS))
def test_norm_of_fp32_lists(name, kind):
    torch, ddp = _torch(), _lib()
    say("case norm", name, kind)
    c = Case(LISTS[name], seed=len(name) + kind, sigma=0.1)
    norm = new_norm()
    ddp.ddp_grad_norm(c.make(), kind, norm.data_ptr(), torch.cuda.current_stream().cuda_stream)
    check_norm(float(norm), ref_norm(c.flat64(), kind))
    c.guards_hold()


@pytest.mark.parametrize("name", sorted(LISTS))
@pytest.mark.parametrize("types", ["f32", "bf16", "f16", "mixed"])
@pytest.mark.parametrize("apart", [False, True])
def test_clip_over_types(name, types, apart):
    torch, ddp = _torch(), _lib()
    say("case clip", name, types, apart)
    n = LISTS[name]
    dtype = [{"f32": 0, "bf16": 1, "f16": 2}.get(types, i % 3) for i in range(len(n))]
    out = [(i + 1) % 3 for i in range(len(n))] if apart else None
    c = Case(n, dtype, copies=2, out=out, seed=3, sigma=0.3)
    norm = new_norm()
    ddp.ddp_clip_grad_norm(c.make(), ddp.DDP_NORM_L2, 0.25, norm.data_ptr(), torch.cuda.current_stream().cuda_stream)
    want = ref_norm(c.flat64(), ddp.DDP_NORM_L2)
    check_norm(float(norm), want)
    check_clip(c, want, 0.25)
    c.guards_hold()
    if apart:   # the sources stay as they were
        for vs in c.views:
            for v, x in zip(vs, c.values):
                assert torch.equal(v.cpu(), x)


@pytest.mark.parametrize("name,dtype,out", [("tensors", 0, 0), ("tensors", 1, 0), ("tensors", 1, 2), ("odd", 2, 1)])
def test_clip_of_many_tiles_into_other_buffers(name, dtype, out):
    """Past the size from which the clipping is a workgroup a part of a tile."""
    torch, ddp = _torch(), _lib()
    say("case many", name, dtype, out)
    n = [(40 << 20) + 17, 1, 12345, 8192] if name == "tensors" else [9999 + i for i in range(2600)]
    c = Case(n, [dtype] * len(n), out=[out] * len(n), seed=21, sigma=0.01)
    norm = new_norm()
    g = c.make()
    s = torch.cuda.current_stream().cuda_stream
    ddp.ddp_clip_grad_norm(g, 2, 0.5, norm.data_ptr(), s)
    want = ref_norm(c.flat64(), 2)
    check_norm(float(norm), want)
    check_clip(c, want, 0.5)
    c.guards_hold()
    first = [v.clone() for v in c.out_views[0]]
    ddp.ddp_clip_grads(g, 0.5, norm.data_ptr(), s)
    assert all(torch.equal(a, b) for a, b in zip(first, c.out_views[0]))


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("size", [5, 70000])
def test_clip_by_each_norm(kind, size):
    torch, ddp = _torch(), _lib()
    say("case clip by", kind, size)
    c = Case([size, 1000], seed=9, sigma=0.2)
    norm = new_norm()
    ddp.ddp_clip_grad_norm(c.make(), kind, 0.05, norm.data_ptr(), torch.cuda.current_stream().cuda_stream)
    want = ref_norm(c.flat64(), kind)
    check_norm(float(norm), want)
    check_clip(c, want, 0.05)


@pytest.mark.parametrize("size", [40, 200000])
def test_a_norm_below_the_bound_leaves_the_list_untouched(size):
    torch, ddp = _torch(), _lib()
    say("case below", size)
    c = Case([size], seed=1, sigma=1e-4)
    c.views[0][0][3] = -0.0
    before = c.bufs[0][0].clone()
    norm = new_norm()
    ddp.ddp_clip_grad_norm(c.make(), 2, 100.0, norm.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert torch.equal(c.bufs[0][0].view(torch.int32), before.view(torch.int32))
    # into another buffer it is a copy
    d = Case([size], out=[0], seed=1, sigma=1e-4)
    ddp.ddp_clip_grad_norm(d.make(), 2, 100.0, norm.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert torch.equal(d.out_views[0][0].cpu(), d.values[0])


@pytest.mark.parametrize("size,copies", [(500, 8), (30000, 8), (100000, 5)])
def test_many_copies_of_a_small_list(size, copies):
    torch, ddp = _torch(), _lib()
    say("case copies", size, copies)
    c = Case([size, 7], [0, 1], copies=copies, seed=copies)
    norm = new_norm()
    ddp.ddp_clip_grad_norm(c.make(), 2, 0.3, norm.data_ptr(), torch.cuda.current_stream().cuda_stream)
    want = ref_norm(c.flat64(), 2)
    check_norm(float(norm), want)
    check_clip(c, want, 0.3)
    c.guards_hold()


def test_tensors_of_no_elements_may_have_no_address():
    torch, ddp = _torch(), _lib()
    x = torch.full((10,), 2.0, device="cuda")
    g = ddp.make_grads([0, 10, 0], [[0, x.data_ptr(), 3]])
    norm = new_norm()
    ddp.ddp_grad_norm(g, 2, norm.data_ptr(), torch.cuda.current_stream().cuda_stream)
    check_norm(float(norm), 40.0 ** 0.5)


def test_a_bound_of_zero_gives_zeros():
    torch, ddp = _torch(), _lib()
    c = Case([100, 90000], seed=2)
    norm = new_norm()
    ddp.ddp_clip_grad_norm(c.make(), 2, 0.0, norm.data_ptr(), torch.cuda.current_stream().cuda_stream)
    check_norm(float(norm), ref_norm(c.flat64(), 2))
    assert all(not bool(v.any()) for v in c.views[0])


@pytest.mark.parametrize("size", [50, 100000])
@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("bad", ["inf", "-inf", "nan", "both"])
def test_infinities_and_nan(size, kind, bad):
    torch, ddp = _torch(), _lib()
    say("case special", size, kind, bad)
    c = Case([size], seed=4)
    if bad != "nan":
        c.values[0][size // 2] = -math.inf if bad == "-inf" else math.inf
    if bad in ("nan", "both"):
        c.values[0][size - 1] = math.nan
    c.views[0][0].copy_(c.values[0])
    norm = new_norm()
    ddp.ddp_clip_grad_norm(c.make(), kind, 1.0, norm.data_ptr(), torch.cuda.current_stream().cuda_stream)
    got = c.views[0][0].cpu()
    if bad in ("nan", "both"):
        assert math.isnan(float(norm)) and bool(got.isnan().all())
    else:
        assert float(norm) == math.inf
        inf = c.values[0].isinf()
        assert bool(got[inf].isnan().all()) and not bool(got[~inf].any())


@pytest.mark.parametrize("value,count", [(1e30, 1000), (1e-30, 1000), (3e38, 9), (1e-44, 5000), (65504.0, 70000)])
def test_extreme_values_neither_overflow_nor_vanish(value, count):
    torch, ddp = _torch(), _lib()
    say("case extreme", value, count)
    c = Case([count], seed=5)
    c.values[0].fill_(value)
    c.views[0][0].copy_(c.values[0])
    for kind in (0, 1, 2):
        norm = new_norm()
        ddp.ddp_grad_norm(c.make(), kind, norm.data_ptr(), torch.cuda.current_stream().cuda_stream)
        check_norm(float(norm), ref_norm(c.flat64(), kind))


@pytest.mark.parametrize("size", [100, 300000])
def test_a_given_norm(size):
    torch, ddp = _torch(), _lib()
    c = Case([size], copies=2, seed=6)
    norm = torch.full((), 50.0, dtype=torch.float32, device="cuda")
    ddp.ddp_clip_grads(c.make(), 2.0, norm.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert float(norm) == 50.0
    check_clip(c, 50.0, 2.0)
    c.guards_hold()


def test_the_same_bits_every_time():
    torch, ddp = _torch(), _lib()
    c = Case([3000001, 77], seed=8)
    g = c.make()
    got = set()
    for _ in range(5):
        norm = new_norm()
        ddp.ddp_grad_norm(g, 2, norm.data_ptr(), torch.cuda.current_stream().cuda_stream)
        got.add(int(norm.view(torch.int32)))
    assert len(got) == 1


def test_a_large_list():
    """More tiles than workgroups, and element offsets past 2^31 in one tensor."""
    torch, ddp = _torch(), _lib()
    n = (1 << 31) + 12345
    say("case large", n)
    x = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    x[0], x[n - 1], x[n // 2] = 3.0, 4.0, 12.0
    g = ddp.make_grads([n], [[x.data_ptr()]], [ddp.DDP_BF16])
    norm = new_norm()
    s = torch.cuda.current_stream().cuda_stream
    ddp.ddp_clip_grad_norm(g, 2, 1.3, norm.data_ptr(), s)
    assert float(norm) == 13.0
    got = [float(x[i]) for i in (0, n // 2, n - 1)]
    assert all(abs(a - b) <= b * 2.0 ** -7 for a, b in zip(got, (0.3, 1.2, 0.4))), got
    assert int(x.count_nonzero()) == 3


# ---------------------------------------------------------------- reducers
@pytest.mark.parametrize("collective", [0, 1])
@pytest.mark.parametrize("W", [1, 3, 8])
def test_the_list_of_a_reducer(W, collective):
    """The norm is the mean gradient's, and what clipping leaves is the reduced
    result times one factor: everywhere after an all-reduce, in the owners'
    chunks after a reduce-scatter, whose other parts stay as they were."""
    torch, ddp = _torch(), _lib()
    say("case reducer", W, collective)
    numel = [4099, 64, 20000, 1, 8192]
    plan = ddp.ddp_plan_buckets([4 * n for n in numel], ddp.DDP_ORDER_REVERSE, 50000, 50000)
    total = sum(numel)
    gen = torch.Generator().manual_seed(W)
    grads = [[torch.randn(n, generator=gen).cuda() for n in numel] for _ in range(W)]
    flat = [torch.full((total,), 0.5, device="cuda") for _ in range(W)]
    compute, comm = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    r = ddp.make_reducer(W, numel, plan, ddp.DDP_IN_F32_COPY, [[t.data_ptr() for t in g] for g in grads],
                         [f.data_ptr() for f in flat], compute.cuda_stream, comm.cuda_stream, collective=collective)
    g = ddp.make_reducer_grads(r)
    ddp.ddp_prepare_for_backward(r)
    ddp.ddp_mark_ready_many(r, list(range(len(numel)))[::-1])
    ddp.ddp_finish(r, host_blocking=True)
    reduced = [f.clone() for f in flat]
    torch.cuda.synchronize()
    norm = new_norm()
    torch.cuda.synchronize()
    ddp.ddp_clip_grad_norm(g, 2, 0.5, norm.data_ptr(), compute.cuda_stream)
    torch.cuda.synchronize()
    mean = sum(torch.cat([t.cpu().double() for t in gr]) for gr in grads) / W
    # fp32 fold of W terms: W roundings a term at most, so its norm is as near
    want = float(mean.norm())
    assert abs(float(norm) - want) <= 4 * W * U32 * sum(float(torch.cat([t.cpu().double() for t in gr]).norm())
                                                         for gr in grads) / W
    owned = [torch.zeros(total, dtype=torch.bool) for _ in range(W)]
    start = 0
    for b in range(plan.n_buckets):
        n = int(plan.bucket_bytes[b]) // 4
        q = -(-n // W)
        for w in range(W):
            lo, hi = (min(n, w * q), min(n, (w + 1) * q)) if collective else (0, n)
            owned[w][start + lo:start + hi] = True
        start += n
    f = 0.5 / (float(norm) + 1e-6)
    for w in range(W):
        got, was = flat[w].cpu(), reduced[w].cpu()
        assert torch.equal(got[~owned[w]], was[~owned[w]])
        want_w = was.double()[owned[w]] * min(1.0, f)
        assert bool(((got.double()[owned[w]] - want_w).abs() <= want_w.abs() * 6 * U32).all())
    ddp.ddp_grads_destroy(g)
    ddp.ddp_reducer_destroy(r)


def test_the_list_of_a_static_reducer():
    """Its tables lie in the library's own area; the list's are its own."""
    torch, ddp = _torch(), _lib()
    numel, W = [5000, 3], 3
    plan = ddp.ddp_plan_buckets([4 * n for n in numel], ddp.DDP_ORDER_REVERSE, 1 << 30, 1 << 30)
    flat = [torch.full((5003,), float(w + 1), device="cuda") for w in range(W)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    desc = ddp.Desc(W, numel, plan.bucket_of, plan.offset_in_bucket, plan.n_buckets, ddp.DDP_IN_F32_VIEW,
                    flat=[f.data_ptr() for f in flat], compute_stream=s.cuda_stream, comm_stream=s.cuda_stream)
    r = ddp.ddp_reducer_create_static(desc)
    g = ddp.make_reducer_grads(r)
    ddp.ddp_prepare_for_backward(r)
    ddp.ddp_mark_ready_many(r, [1, 0])
    ddp.ddp_finish(r)
    norm = new_norm()
    torch.cuda.synchronize()
    ddp.ddp_clip_grad_norm(g, ddp.DDP_NORM_INF, 1.0, norm.data_ptr(), s.cuda_stream)
    torch.cuda.synchronize()
    # 2 three times over thirds: each term one rounding, two additions
    assert abs(float(norm) - 2.0) <= 2.0 * 5 * U32
    # 2 * (1 / (2 + 1e-6)) is 5e-7 below 1, and 10 roundings
    assert all(bool(((f - 1.0).abs() <= 5e-7 + 10 * U32).all()) for f in flat)
    ddp.ddp_grads_destroy(g)
    ddp.ddp_reducer_destroy(r)


# ---------------------------------------------------------------- streams and graphs
@pytest.mark.parametrize("size", [300, 500000])
def test_replays_of_a_captured_clip(size):
    """Every replay is compared with the eager result on the same gradients,
    with eager work and synchronizations between the replays."""
    torch, ddp = _torch(), _lib()
    say("case graph", size)
    c = Case([size, 33], out=[0, 1], seed=12)
    g = c.make()
    norm = new_norm()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ddp.ddp_clip_grad_norm(g, 2, 0.75, norm.data_ptr(), s.cuda_stream)
    for k in range(4):
        new = torch.randn(size, generator=torch.Generator().manual_seed(k)).cuda() * (k + 1)
        c.views[0][0].copy_(new)
        c.values[0] = new.cpu()
        norm.fill_(-1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        replayed = [float(norm)] + [v.clone() for v in c.out_views[0]]
        eager = new_norm()
        ddp.ddp_clip_grad_norm(g, 2, 0.75, eager.data_ptr(), torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert replayed[0] == float(eager)
        assert all(torch.equal(a, b) for a, b in zip(replayed[1:], c.out_views[0]))
        check_norm(replayed[0], ref_norm(c.flat64(), 2))


def test_calls_of_one_list_at_once_on_two_streams():
    torch, ddp = _torch(), _lib()
    c = Case([2000003], seed=13)
    g = c.make()
    n = ddp.ddp_grads_scratch_bytes(g)
    scratch = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    norms = [[torch.zeros((), device="cuda") for _ in range(10)] for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for k in range(10):
        for i in range(2):
            ddp.ddp_grad_norm(g, 2 - i, norms[i][k].data_ptr(), streams[i].cuda_stream, scratch[i].data_ptr(), n)
    torch.cuda.synchronize()
    for i in range(2):
        want = ref_norm(c.flat64(), 2 - i)
        for x in norms[i]:
            check_norm(float(x), want)


def test_list_refusals_on_the_device():
    torch, ddp = _torch(), _lib()
    c = Case([100000], seed=14)
    g = c.make()
    norm = new_norm()
    s = torch.cuda.current_stream().cuda_stream
    need = ddp.ddp_grads_scratch_bytes(g)
    assert need >= 8
    before = c.bufs[0][0].clone()
    for call in (lambda: ddp.ddp_grad_norm(g, 3, norm.data_ptr(), s),
                 lambda: ddp.ddp_grad_norm(g, 2, 0, s),
                 lambda: ddp.ddp_grad_norm(g, 2, norm.data_ptr() + 1, s),
                 lambda: ddp.ddp_grad_norm(g, 2, norm.data_ptr(), s, g.scratch.data_ptr(), need - 8),
                 lambda: ddp.ddp_grad_norm(g, 2, norm.data_ptr(), s, g.scratch.data_ptr() + 4, need),
                 lambda: ddp.ddp_clip_grad_norm(g, 2, -1.0, norm.data_ptr(), s),
                 lambda: ddp.ddp_clip_grad_norm(g, 2, math.inf, norm.data_ptr(), s),
                 lambda: ddp.ddp_clip_grad_norm(g, 2, math.nan, norm.data_ptr(), s),
                 lambda: ddp.ddp_clip_grads(g, 1.0, 0, s)):
        with pytest.raises(ddp.DDPError) as e:
            call()
        assert e.value.code == ddp.DDP_ERR_INVALID
    torch.cuda.synchronize()
    assert float(norm) == -5.0 and torch.equal(c.bufs[0][0], before)
    ddp.ddp_grads_destroy(g)
    with pytest.raises(ddp.DDPError):
        ddp.ddp_grad_norm(g, 2, norm.data_ptr(), s)


def test_a_norm_in_the_scratch_and_a_workspace_in_a_tensor_are_refused():
    torch, ddp = _torch(), _lib()
    c = Case([100000], seed=16)
    g = c.make()
    s = torch.cuda.current_stream().cuda_stream
    need = ddp.ddp_grads_scratch_bytes(g)
    scratch = torch.zeros(need + 8, dtype=torch.uint8, device="cuda")
    p = scratch.data_ptr()
    for inside in (p, p + need - 4):
        for call in (lambda: ddp.ddp_grad_norm(g, 2, inside, s, p, need),
                     lambda: ddp.ddp_clip_grad_norm(g, 2, 0.5, inside, s, p, need)):
            with pytest.raises(ddp.DDPError) as e:
                call()
            assert e.value.code == ddp.DDP_ERR_INVALID and "inside the scratch" in e.value.msg
    ddp.ddp_grad_norm(g, 2, p + need, s, p, need)   # right behind it
    check_norm(float(scratch[need:need + 4].view(torch.float32)), ref_norm(c.flat64(), 2))
    x = torch.full((1 << 16,), 3.0, device="cuda")
    with pytest.raises(ddp.DDPError) as e:
        ddp.ddp_grads_create(ddp.GradsDesc([1 << 16], [[x.data_ptr()]], workspace=x.data_ptr() + 1024,
                                           workspace_bytes=4096))
    assert e.value.code == ddp.DDP_ERR_INVALID and "the workspace and gradient 0 overlap" in e.value.msg
    assert bool((x == 3.0).all())


def test_a_handle_dropped_with_its_calls_queued_on_another_stream():
    """The memory of its tables is not handed out before they have run."""
    torch, ddp = _torch(), _lib()
    c = Case([20000003], copies=2, out=[1], seed=15)
    side = torch.cuda.Stream()
    norms = [new_norm() for _ in range(8)]
    torch.cuda.synchronize()
    for x in norms:
        ddp.ddp_clip_grad_norm(c.make(), 2, 0.5, x.data_ptr(), side.cuda_stream)
        for _ in range(4):   # takes what the allocator thinks free, on the stream it was allocated on
            torch.full((400000,), 255, dtype=torch.uint8, device="cuda")
            torch.full((30000,), 255, dtype=torch.uint8, device="cuda")
            torch.full((8192,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    want = ref_norm(c.flat64(), 2)
    for x in norms:
        check_norm(float(x), want)
    check_clip(c, want, 0.5)
