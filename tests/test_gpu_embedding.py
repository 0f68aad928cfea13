"""GPU: the embedding lookup and the table's gradient against the formulas in
64 bits: token counts and row counts around the chunks and the sorting
workgroups' ranges, frequent tokens, indices outside the table, padding, odd
widths, strides and addresses, every type, graphs and streams; the gradient
against differences of the lookup; refusals are in the CPU tests.

Tolerances, set before the first run (u = eps / 2 of a type):
  lookup    scale * x in fp32 (u32), then one rounding to the output's type.
  gradient  the sum of n terms in fp32 in any order is off by at most
            (n - 1) u32 / (1 - n u32) times the sum of their magnitudes; the
            scale comes with one rounding (its product fused with the addition,
            or alone), then one rounding to the gradient's type.
Below the smallest normal value a rounding is absolute: half the smallest
subnormal.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
HALF_SUBNORMAL = {"torch.float32": 2.0 ** -150, "torch.bfloat16": 2.0 ** -134, "torch.float16": 2.0 ** -25}


def _torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def _lib():
    import bucketed_gradient_all_amd as ddp
    return ddp


def _type(k):
    torch = _torch()
    return {0: torch.float32, 1: torch.bfloat16, 2: torch.float16}[k]


def say(*a):
    print(*a, flush=True)


def strided(rows, width, stride, dtype, seed, shift=0, sigma=1.0, filler=9.0):
    """A [rows, width] view with the given row stride, `shift` elements into
    its buffer, of random values; everything else of the buffer is filler."""
    torch = _torch()
    n = shift + (rows - 1) * stride + width + 5 if rows else shift + 5
    buf = torch.full((max(n, 1),), filler, dtype=dtype, device="cuda")
    v = torch.as_strided(buf, (rows, width), (stride, 1), shift)
    if rows and width:
        g = torch.Generator().manual_seed(seed)
        v.copy_((torch.randn(rows, width, generator=g) * sigma).to(dtype))
    return buf, v


def outside(buf, view):
    """The buffer's elements that are not the view's."""
    torch = _torch()
    mask = torch.ones(buf.numel(), dtype=torch.bool, device="cuda")
    torch.as_strided(mask, view.shape, view.stride(), view.storage_offset()).fill_(False)
    return buf[mask]


def tokens_of(kind, T, V, first, seed):
    torch = _torch()
    g = torch.Generator().manual_seed(seed)
    if kind == "uniform":
        t = torch.randint(0, V, (T,), generator=g) + first
    elif kind == "same":
        t = torch.full((T,), V // 2) + first
    elif kind == "two":
        t = torch.randint(0, 2, (T,), generator=g) * (V - 1) + first
    elif kind == "falling":   # frequent and rare tokens: rank as 1/u
        t = (1.0 / (torch.rand(T, generator=g, dtype=torch.float64) + 1.0 / V)).long().clamp(max=V) - 1 + first
    elif kind == "sorted":
        t = torch.arange(T) * V // max(T, 1) + first
    elif kind == "outside":
        t = torch.randint(0, V, (T,), generator=g) + first + V
    elif kind == "wild":      # inside, outside on both sides, extreme
        t = torch.randint(-V, 2 * V, (T,), generator=g) + first
        t[::5] = -1
        t[1::7] = 2 ** 31 - 1
        t[2::11] = -2 ** 31
    else:
        raise KeyError(kind)
    return t.long()


class Case:
    def __init__(self, T, V, H, kind="uniform", act=0, row=0, index64=True, scale=1.0, first=0, padding=-1,
                 stride_extra=0, shift=0, seed=0):
        torch, ddp = _torch(), _lib()
        self.T, self.V, self.H, self.scale, self.first, self.padding = T, V, H, scale, first, padding
        stride = H + stride_extra
        self.host_tokens = tokens_of(kind, T, V, first, seed)
        # one element into its buffer, so that tokens start at an odd address
        buf = torch.zeros(T + 1, dtype=torch.int64 if index64 else torch.int32)
        buf[1:] = self.host_tokens.to(buf.dtype)
        self.token_buf = buf.cuda()
        self.tokens = self.token_buf[1:]
        self.act_buf, self.act = strided(T, H, stride, _type(act), seed + 1, shift)
        self.row_buf, self.row = strided(V, H, stride, _type(row), seed + 2, shift)
        self.desc = ddp.EmbeddingDesc(V, H, table_dtype=row, grad_dtype=row, act_dtype=act,
                                      index_dtype=ddp.DDP_I64 if index64 else ddp.DDP_I32, scale=scale,
                                      first_row=first, padding_idx=padding, table_stride=stride, grad_stride=stride,
                                      act_stride=stride)
        self.scale32 = float(torch.tensor(scale, dtype=torch.float32))

    def stream(self):
        return _torch().cuda.current_stream().cuda_stream

    # ---- lookup
    def lookup(self):
        _lib().ddp_embedding_lookup(self.desc, self.row.data_ptr(), self.tokens.data_ptr(), self.T,
                                    self.act.data_ptr(), self.stream())

    def check_lookup(self):
        torch = _torch()
        rest = outside(self.act_buf, self.act)
        assert bool((rest == 9.0).all())
        r = self.host_tokens - self.first
        held = (r >= 0) & (r < self.V)
        want = torch.zeros(self.T, self.H, dtype=torch.float64)
        want[held] = self.row.cpu().double()[r[held]] * self.scale32
        got = self.act.cpu()
        assert not bool(got[~held].any())
        u = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0
        tol = want.abs() * (U32 + u) * (1 + 1e-3) + HALF_SUBNORMAL[str(got.dtype)] + 2.0 ** -150
        assert bool(((got.double() - want).abs() <= tol).all())

    # ---- gradient
    def grad(self, accumulate, workspace=None):
        torch, ddp = _torch(), _lib()
        n = ddp.ddp_embedding_grad_workspace_bytes(self.desc, self.T)
        if workspace is None:   # garbage: nothing of it may matter
            workspace = torch.full((n,), 0xAB, dtype=torch.uint8, device="cuda")
        ddp.ddp_embedding_grad(self.desc, self.act.data_ptr(), self.tokens.data_ptr(), self.T, self.row.data_ptr(),
                               accumulate, workspace.data_ptr(), n, self.stream())
        return workspace

    def check_grad(self, before, accumulate):
        """before: the gradient as it was (a CPU tensor)."""
        torch = _torch()
        assert bool((outside(self.row_buf, self.row) == 9.0).all())
        r = self.host_tokens - self.first
        held = (r >= 0) & (r < self.V)
        if self.padding >= 0:
            held &= self.host_tokens != self.padding
        x = self.act.cpu().double()[held] if self.T else torch.zeros(0, self.H, dtype=torch.float64)
        r = r[held]
        total = torch.zeros(self.V, self.H, dtype=torch.float64).index_add_(0, r, x)
        size = torch.zeros(self.V, self.H, dtype=torch.float64).index_add_(0, r, x.abs())
        n = torch.bincount(r, minlength=self.V).double()[:, None]
        got = self.row.cpu()
        untouched = (n == 0)[:, 0]
        if accumulate:
            assert torch.equal(got[untouched], before[untouched])
        else:
            assert not bool(got[untouched].any())
        want = total * self.scale32 + (before.double() if accumulate else 0.0)
        u = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0
        gamma = n * U32 / (1 - n * U32)
        off = abs(self.scale32) * gamma * size
        tol = off + (want.abs() + off) * (U32 + u) * (1 + 1e-3) + HALF_SUBNORMAL[str(got.dtype)] + 2.0 ** -150
        bad = ((got.double() - want).abs() > tol) & (n > 0)
        assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:5], got[bad][:5], want[bad][:5])

    def run_grad(self, accumulate):
        before = self.row.cpu().clone()
        self.grad(accumulate)
        self.check_grad(before, accumulate)


# ---------------------------------------------------------------- lookup
@pytest.mark.parametrize("T", [0, 1, 2, 5, 300, 20001])
@pytest.mark.parametrize("H", [1, 3, 4, 7, 8, 9, 256, 513])
def test_lookup_sizes(T, H):
    say("case lookup", T, H)
    c = Case(T, 97, H, kind="wild", scale=1.7, seed=T + H)
    c.lookup()
    c.check_lookup()


@pytest.mark.parametrize("row", [0, 1, 2])
@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("index64", [False, True])
@pytest.mark.parametrize("shift,extra", [(0, 0), (1, 3)])
def test_lookup_types_and_addresses(row, act, index64, shift, extra):
    say("case lookup types", row, act, index64, shift, extra)
    c = Case(130, 61, 75, kind="wild", act=act, row=row, index64=index64, scale=0.37, first=40, shift=shift,
             stride_extra=extra, seed=row * 3 + act)
    c.lookup()
    c.check_lookup()


@pytest.mark.parametrize("T,H,row,act", [(9000, 2048, 1, 1), (70000, 64, 0, 1), (33, 5000, 0, 0)])
def test_lookup_large(T, H, row, act):
    say("case lookup large", T, H)
    c = Case(T, 300, H, kind="falling", act=act, row=row, scale=math.sqrt(H), seed=2)
    c.lookup()
    c.check_lookup()


def test_lookup_and_gradient_past_32_bits():
    """Row offsets past 2^32 bytes and 2^31 elements in the table, the
    positions' rows and the gradient."""
    torch, ddp = _torch(), _lib()
    V, H = 1100000, 2048   # 2.25e9 elements
    say("case far", V, H)
    table = torch.zeros(V, H, dtype=torch.bfloat16, device="cuda")
    rows = [0, V // 2, V - 1, 1048577]
    for k, r in enumerate(rows):
        table[r] = float(k + 1)
    tok = torch.tensor(rows + [V], device="cuda")
    stride = 1 << 29
    out = torch.zeros(4 * stride + H, dtype=torch.bfloat16, device="cuda")   # the last row begins at 2^31
    d = ddp.EmbeddingDesc(V, H, table_dtype=1, grad_dtype=1, act_dtype=1, act_stride=stride)
    s = torch.cuda.current_stream().cuda_stream
    ddp.ddp_embedding_lookup(d, table.data_ptr(), tok.data_ptr(), 5, out.data_ptr(), s)
    for k in range(5):
        assert bool((out[k * stride:k * stride + H] == (float(k + 1) if k < 4 else 0.0)).all())
    out[4 * stride:] = 64.0
    tok = torch.tensor(rows + [V - 1], device="cuda")
    n = ddp.ddp_embedding_grad_workspace_bytes(d, 5)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    ddp.ddp_embedding_grad(d, out.data_ptr(), tok.data_ptr(), 5, table.data_ptr(), True, ws.data_ptr(), n, s)
    for k, r in enumerate(rows):
        assert bool((table[r] == 2.0 * (k + 1) + (64.0 if r == V - 1 else 0.0)).all()), r
    assert int(table.count_nonzero()) == 4 * H


# ---------------------------------------------------------------- gradient
@pytest.mark.parametrize("T", [0, 1, 2, 7, 8, 9, 63, 64, 65, 1000, 4097])
@pytest.mark.parametrize("kind", ["uniform", "same", "falling", "wild", "outside", "sorted"])
@pytest.mark.parametrize("accumulate", [True, False])
def test_gradient_token_counts(T, kind, accumulate):
    say("case grad", T, kind, accumulate)
    Case(T, 50, 68, kind=kind, scale=1.3, seed=T).run_grad(accumulate)


@pytest.mark.parametrize("V", [1, 2, 15, 16, 17, 255, 4096, 4097, 20000, 70001, 530001])
@pytest.mark.parametrize("kind", ["uniform", "two", "falling"])
def test_gradient_row_counts(V, kind):
    say("case grad rows", V, kind)
    Case(3001, V, 12, kind=kind, seed=V).run_grad(V % 2 == 0)


@pytest.mark.parametrize("H", [1, 2, 3, 4, 5, 7, 8, 9, 255, 256, 257, 511, 512, 513, 1030, 2047])
@pytest.mark.parametrize("act", [0, 1])
def test_gradient_widths(H, act):
    say("case grad width", H, act)
    Case(515, 40, H, kind="falling", act=act, seed=H).run_grad(True)
    Case(515, 40, H, kind="falling", act=act, row=act, seed=H).run_grad(False)


@pytest.mark.parametrize("row", [0, 1, 2])
@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("index64", [False, True])
@pytest.mark.parametrize("shift,extra", [(0, 0), (1, 3)])
@pytest.mark.parametrize("accumulate", [True, False])
def test_gradient_types_and_addresses(row, act, index64, shift, extra, accumulate):
    say("case grad types", row, act, index64, shift, extra, accumulate)
    Case(700, 90, 77, kind="wild", act=act, row=row, index64=index64, scale=0.6, first=33, shift=shift,
         stride_extra=extra, seed=row * 3 + act).run_grad(accumulate)


@pytest.mark.parametrize("T,V,H,kind", [(40000, 300, 64, "falling"), (40000, 32000, 513, "falling"),
                                        (70000, 7, 20, "uniform"), (33000, 1000, 2048, "same"),
                                        (200000, 50000, 8, "two"), (20000, 2, 3, "uniform"),
                                        (600000, 300, 4, "falling"), (530000, 3000, 5, "uniform"),
                                        (140000, 400000, 4, "falling"), (70001, 1, 33, "same")])
@pytest.mark.parametrize("accumulate", [True, False])
def test_gradient_long_runs(T, V, H, kind, accumulate):
    say("case grad long", T, V, H, kind, accumulate)
    Case(T, V, H, kind=kind, act=1, scale=2.0, seed=5).run_grad(accumulate)


@pytest.mark.parametrize("accumulate", [True, False])
def test_padding_contributes_nothing(accumulate):
    c = Case(2000, 30, 40, kind="falling", padding=0, seed=3)
    assert int((c.host_tokens == 0).sum()) > 300
    c.run_grad(accumulate)
    # every position is padding
    c = Case(2000, 30, 40, kind="same", padding=15, seed=3)
    c.run_grad(accumulate)
    # a padding index of another shard concerns no row of this one
    c = Case(500, 30, 40, kind="uniform", first=100, padding=3, seed=4)
    c.run_grad(accumulate)


# Tables of so many rows take the path of several launches whatever the number
# of positions; small ones the one of a single launch for few positions.
FEW, MANY = 64, 600000


@pytest.mark.parametrize("V", [FEW, MANY])
@pytest.mark.parametrize("lead", range(9))
def test_runs_at_every_place_of_a_chunk(V, lead):
    """Runs of every length up to past two chunks, one after the other, so that
    they begin and end everywhere in the chunks, and in the waves' parts."""
    torch = _torch()
    lengths = [n for n in range(1, 21)] + [17, 16, 15, 9, 8, 7, 1, 1, 33, 8, 24, 16, 8, 70, 64, 65, 130]
    t = torch.cat([torch.full((n,), i) for i, n in enumerate(lengths)])
    tok = torch.cat([torch.zeros(lead, dtype=torch.long), t + 1]) * (V // 64)
    tok = tok[torch.randperm(tok.numel(), generator=torch.Generator().manual_seed(lead))]
    for accumulate in (True, False):
        c = Case(tok.numel(), V, 16, seed=lead)
        c.host_tokens = tok
        c.tokens.copy_(tok)
        c.run_grad(accumulate)


@pytest.mark.parametrize("T", [1, 2, 9, 63, 65, 1000, 3000])
@pytest.mark.parametrize("kind", ["uniform", "same", "falling", "wild", "two"])
def test_gradient_of_few_tokens_in_a_large_table(T, kind):
    say("case grad large table", T, kind)
    Case(T, MANY, 20, kind=kind, scale=1.3, first=7, padding=9, seed=T).run_grad(True)


@pytest.mark.parametrize("V,H,act,row", [(32000, 2048, 1, 0), (32000, 2048, 1, 1), (30522, 1024, 0, 0), (200, 4099, 2, 2),
                                         (130000, 300, 1, 0), (5, 130, 0, 1)])
@pytest.mark.parametrize("T", [1, 500, 2047, 4096, 4097])
@pytest.mark.parametrize("kind", ["falling", "same"])
def test_gradient_of_few_tokens(V, H, act, row, T, kind):
    say("case grad few", V, H, act, row, T, kind)
    Case(T, V, H, kind=kind, act=act, row=row, scale=0.7, padding=1, seed=T + V).run_grad(True)


def test_one_row_for_every_position():
    """act_stride 0: the positions share one row of dout."""
    torch, ddp = _torch(), _lib()
    c = Case(999, 20, 50, kind="falling", seed=6)
    one = c.act[:1].clone()
    c.act.copy_(one.expand(999, 50))
    before = c.row.cpu().clone()
    d = ddp.EmbeddingDesc(20, 50, act_stride=0)
    n = ddp.ddp_embedding_grad_workspace_bytes(d, 999)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    ddp.ddp_embedding_grad(d, one.data_ptr(), c.tokens.data_ptr(), 999, c.row.data_ptr(), True, ws.data_ptr(), n,
                           c.stream())
    c.check_grad(before, True)


@pytest.mark.parametrize("kind", ["falling", "same"])
def test_gradient_gives_the_same_bits(kind):
    torch = _torch()
    c = Case(30000, 400, 129, kind=kind, seed=7)
    start = c.row.clone()
    seen = None
    for _ in range(4):
        c.row.copy_(start)
        c.grad(True)
        if seen is None:
            seen = c.row.clone()
        assert torch.equal(seen.view(torch.int32), c.row.view(torch.int32))


def test_old_contents_do_not_matter_when_the_whole_gradient_is_written():
    c = Case(300, 64, 33, kind="uniform", seed=8)
    c.row.fill_(math.nan)
    c.grad(False)
    c.check_grad(c.row.cpu() * 0, False)


def test_infinities_stay_in_their_rows():
    torch = _torch()
    c = Case(400, 20, 24, kind="uniform", seed=9)
    where = int((c.host_tokens == 3).nonzero()[0])
    c.act[where] = math.inf
    c.act[int((c.host_tokens == 5).nonzero()[0])] = math.nan
    c.grad(True)
    got = c.row.cpu()
    assert bool((got[3] == math.inf).all()) and bool(got[5].isnan().all())
    rest = [r for r in range(20) if r not in (3, 5)]
    assert bool(torch.isfinite(got[rest]).all())


def test_gradient_against_differences():
    """d/dtable of <dout, lookup(table)>: the lookup is linear in the table, so
    a difference over a step of any size is exact but for the roundings of its
    two fp32 evaluations of the outputs."""
    torch = _torch()
    c = Case(60, 9, 5, kind="uniform", scale=0.5, first=2, seed=10)
    dout = c.act.clone()
    table = c.row.clone()
    c.row.zero_()
    c.act.copy_(dout)
    c.grad(True)
    grad = c.row.cpu().double()
    step = 1.0

    def value(t):
        c.row.copy_(t)
        c.lookup()
        return float((c.act.cpu().double() * dout.cpu().double()).sum())

    for r, h in ((0, 0), (4, 2), (8, 4)):
        up, down = table.clone(), table.clone()
        up[r, h] += step
        down[r, h] -= step
        width = float(up.cpu().double()[r, h] - down.cpu().double()[r, h])
        diff = (value(up) - value(down)) / width
        n = int((c.host_tokens - 2 == r).sum())
        col = dout.cpu().double()[c.host_tokens - 2 == r, h].abs().sum()
        # outputs of up to 3: half a step of 2^-22 each, twice; the gradient's own bound
        tol = float(col) * (2 * 2.0 ** -23 / width + (n + 1) * U32)
        assert abs(diff - float(grad[r, h])) <= tol, (r, h, diff, float(grad[r, h]))


@pytest.mark.parametrize("kind", ["falling", "same"])
def test_replays_of_captured_calls(kind):
    torch, ddp = _torch(), _lib()
    c = Case(5000, 200, 65, kind=kind, seed=11)
    table = c.row.clone()
    out = torch.zeros(5000, 65, device="cuda")
    n = ddp.ddp_embedding_grad_workspace_bytes(c.desc, c.T)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ddp.ddp_embedding_lookup(c.desc, table.data_ptr(), c.tokens.data_ptr(), c.T, out.data_ptr(), s.cuda_stream)
        ddp.ddp_embedding_grad(c.desc, c.act.data_ptr(), c.tokens.data_ptr(), c.T, c.row.data_ptr(), True,
                               ws.data_ptr(), n, s.cuda_stream)
    for k in range(4):
        c.host_tokens = tokens_of("falling" if k % 2 else kind, c.T, c.V, 0, 100 + k)
        c.tokens.copy_(c.host_tokens)
        c.act.normal_()
        before = c.row.cpu().clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        c.check_grad(before, True)
        tok = c.host_tokens.cuda()
        held = ((tok >= 0) & (tok < c.V))[:, None]   # an index below the table gives zeros
        assert torch.equal(out, torch.where(held, table[tok.clamp(0, c.V - 1)], torch.zeros_like(out)))
        c.grad(True)              # eager work between the replays, with a workspace of its own
        torch.cuda.synchronize()


def test_two_gradients_at_once_on_two_streams():
    torch = _torch()
    cases = [Case(6000, 100, 128, kind="falling", seed=20 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    before = [c.row.cpu().clone() for c in cases]
    ddp = _lib()
    n = ddp.ddp_embedding_grad_workspace_bytes(cases[0].desc, 6000)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for c, s, w in zip(cases, streams, ws):
        with torch.cuda.stream(s):
            c.grad(True, w)
    torch.cuda.synchronize()
    for c, b in zip(cases, before):
        c.check_grad(b, True)


@pytest.mark.parametrize("V", [FEW, MANY])
@pytest.mark.parametrize("lead", range(20))
def test_padding_between_other_rows_of_a_chunk(V, lead):
    """The padding row's positions lie between other rows' in the sorted order,
    at every offset from the chunks' borders."""
    torch = _torch()
    tok = torch.cat([torch.arange(lead), torch.full((5 + lead,), 30), torch.arange(31, 60), torch.full((40,), 61)])
    tok = tok[torch.randperm(tok.numel(), generator=torch.Generator().manual_seed(lead))] * (V // 64)
    for accumulate in (True, False):
        c = Case(tok.numel(), V, 24, padding=30 * (V // 64), seed=lead)
        c.host_tokens = tok
        c.tokens.copy_(tok)
        c.run_grad(accumulate)


def test_more_rows_than_a_launch_has_waves():
    """The lookup and the filled rows take further launches."""
    torch, ddp = _torch(), _lib()
    V, H, T = 1300003, 300, 4500001   # narrow rows: one wave a row, four rows a lookup's wave
    say("case waves", V, H, T)
    table = torch.arange(V, device="cuda", dtype=torch.float32)[:, None].expand(V, H).to(torch.bfloat16).contiguous()
    tok = torch.randint(0, V, (T,), device="cuda")
    out = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    d = ddp.EmbeddingDesc(V, H, table_dtype=1, grad_dtype=1, act_dtype=1)
    s = torch.cuda.current_stream().cuda_stream
    ddp.ddp_embedding_lookup(d, table.data_ptr(), tok.data_ptr(), T, out.data_ptr(), s)
    for k in range(0, T, 500000):
        assert torch.equal(out[k:k + 500000], table[tok[k:k + 500000]])
    del table
    few = 1000
    dout = torch.ones(few, H, dtype=torch.bfloat16, device="cuda")
    grad = torch.full((V, H), 3.0, dtype=torch.bfloat16, device="cuda")
    n = ddp.ddp_embedding_grad_workspace_bytes(d, few)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    ddp.ddp_embedding_grad(d, dout.data_ptr(), tok.data_ptr(), few, grad.data_ptr(), False, ws.data_ptr(), n, s)
    count = torch.bincount(tok[:few], minlength=V)
    assert torch.equal(grad[:, 0].float(), count.float()) and torch.equal(grad[:, H - 1], grad[:, 0])
    assert int(grad.count_nonzero()) == int(count.count_nonzero()) * H


@pytest.mark.parametrize("stream", [0, 1, 2])
def test_the_null_the_legacy_and_the_per_thread_stream(stream):
    """Streams with names of their own: hipStreamLegacy is 1, hipStreamPerThread 2."""
    torch, ddp = _torch(), _lib()
    c = Case(3000, 40, 30, kind="falling", seed=31)
    before = c.row.cpu().clone()
    n = ddp.ddp_embedding_grad_workspace_bytes(c.desc, c.T)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    ddp.ddp_embedding_grad(c.desc, c.act.data_ptr(), c.tokens.data_ptr(), c.T, c.row.data_ptr(), True, ws.data_ptr(), n,
                           stream)
    torch.cuda.synchronize()
    c.check_grad(before, True)


@pytest.mark.parametrize("T,V", [(900, 50), (20000, 50), (900, 600000)])
@pytest.mark.parametrize("act", [0, 1])
def test_nan_in_places_that_do_not_count(T, V, act):
    """Rows of dout at padding positions and at indices outside the table are
    NaN or infinite, and so are rows of the table that no token names."""
    torch = _torch()
    for accumulate in (True, False):
        c = Case(T, V, 24, kind="wild", act=act, padding=V // 2, first=0, seed=T + V)
        r = c.host_tokens
        c.host_tokens = torch.where(torch.arange(T) % 3 == 0, torch.full_like(r, V // 2), r)
        c.tokens.copy_(c.host_tokens)
        out = (c.host_tokens < 0) | (c.host_tokens >= V) | (c.host_tokens == V // 2)
        c.act[out.cuda()] = math.nan
        c.act[(out & (torch.arange(T) % 2 == 0)).cuda()] = math.inf
        before = c.row.cpu().clone()
        c.grad(accumulate)
        assert bool(torch.isfinite(c.row).all())
        clean = c.act.clone()
        c.act[out.cuda()] = 0.0   # for the reference, which leaves them out by the mask
        c.check_grad(before, accumulate)
        del clean
    c = Case(T, V, 24, kind="wild", act=act, seed=1)
    named = torch.zeros(V, dtype=torch.bool)
    held = (c.host_tokens >= 0) & (c.host_tokens < V)
    named[c.host_tokens[held]] = True
    c.row[(~named).cuda()] = math.nan
    c.lookup()
    c.check_lookup()


def test_lookup_in_an_empty_table():
    torch, ddp = _torch(), _lib()
    out = torch.full((7, 33), 5.0, device="cuda")
    tok = torch.arange(7, device="cuda")
    d = ddp.EmbeddingDesc(0, 33)
    ddp.ddp_embedding_lookup(d, 0, tok.data_ptr(), 7, out.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert not bool(out.any())


@pytest.mark.parametrize("first", [-20, -(1 << 40), 1 << 40, (1 << 63) - 41])
@pytest.mark.parametrize("T", [300, 9000])
def test_shards_anywhere_in_64_bits(first, T):
    """Tables whose rows stand for negative indices, or for the largest."""
    say("case first", first, T)
    torch = _torch()
    g = torch.Generator().manual_seed(T)
    c = Case(T, 40, 17, seed=T)
    rows = torch.randint(-40, 80, (T,), generator=g).clamp(max=39 if first > 1 << 62 else 80)
    c.host_tokens = rows + first
    c.tokens.copy_(c.host_tokens)
    c.first = c.desc.c.first_row = first
    c.run_grad(True)
    c.run_grad(False)
    c.lookup()
    c.check_lookup()


@pytest.mark.parametrize("scale", [0.0, -1.5, 1e20])
@pytest.mark.parametrize("T", [300, 9000])
def test_scales(scale, T):
    """The gradient leaves the table's rows scaled once, and the lookup scales them again: with the largest scale
    that is 1e20 * 1e20 = 1e40, past 2^128 - 2^103 = 3.4e38, from where on float32 rounds to infinity. A product of two float32 has 48 bits and is exact in 64; rounded once it is the one right answer, so the
    lookup is compared with it bit for bit instead of within a tolerance."""
    torch = _torch()
    say("case scales", scale, T)
    c = Case(T, 40, 17, kind="falling", scale=scale, seed=T)
    c.run_grad(True)
    c.run_grad(False)
    c.lookup()
    assert bool((outside(c.act_buf, c.act) == 9.0).all())
    held = (c.host_tokens >= 0) & (c.host_tokens < c.V)
    want = torch.zeros(T, c.H, dtype=torch.float32)
    want[held] = (c.row.cpu().double()[c.host_tokens[held]] * c.scale32).float()
    assert torch.equal(c.act.cpu(), want)


@pytest.mark.parametrize("T", [500, 9000])
def test_strides_of_their_own(T):
    """The table, the gradient and the positions' rows with three strides."""
    torch, ddp = _torch(), _lib()
    V, H = 60, 45
    c = Case(T, V, H, kind="wild", seed=T)
    c.act_buf, c.act = strided(T, H, 47, torch.float32, 1)
    c.row_buf, c.row = strided(V, H, 64, torch.float32, 2)
    c.desc = ddp.EmbeddingDesc(V, H, table_stride=64, grad_stride=64, act_stride=47)
    c.run_grad(True)
    c.run_grad(False)
    c.lookup()
    c.check_lookup()
    grad_buf, grad = strided(V, H, 51, torch.bfloat16, 3)
    d = ddp.EmbeddingDesc(V, H, table_dtype=0, grad_dtype=1, table_stride=64, grad_stride=51, act_stride=47)
    n = ddp.ddp_embedding_grad_workspace_bytes(d, T)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    before = grad.cpu().clone()
    ddp.ddp_embedding_grad(d, c.act.data_ptr(), c.tokens.data_ptr(), T, grad.data_ptr(), True, ws.data_ptr(), n, c.stream())
    c.row_buf, c.row = grad_buf, grad
    c.check_grad(before, True)


def test_one_row_for_many_positions():
    """act_stride 0 past the size of the single launch."""
    torch, ddp = _torch(), _lib()
    c = Case(9000, 20, 50, kind="falling", seed=6)
    one = c.act[:1].clone()
    c.act.copy_(one.expand(9000, 50))
    before = c.row.cpu().clone()
    d = ddp.EmbeddingDesc(20, 50, act_stride=0)
    n = ddp.ddp_embedding_grad_workspace_bytes(d, 9000)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    ddp.ddp_embedding_grad(d, one.data_ptr(), c.tokens.data_ptr(), 9000, c.row.data_ptr(), True, ws.data_ptr(), n,
                           c.stream())
    c.check_grad(before, True)
