"""GPU: clipping of lists of more than 4096 tiles into other buffers, which is
a workgroup a part of a tile behind a launch that finishes the norm: several
copies, odd sizes, each norm, bounds on both sides of the norm, infinities and
NaN, a given norm, replays. The bounds are those of test_gpu_grads.py."""
import math

import pytest

from test_gpu_grads import Case, _lib, _torch, check_clip, check_norm, new_norm, ref_norm, say

pytestmark = pytest.mark.gpu

# copies * elements > 4096 * 8192; a tensor that ends inside a tile and some
# shorter than one, at odd addresses
SIZES = {2: [16777217, 1, 0, 12345, 8191], 4: [8400001, 129, 20000], 5: [9999 + i for i in range(700)]}


def call(c, kind, bound, norm):
    torch, ddp = _torch(), _lib()
    ddp.ddp_clip_grad_norm(c.make(), kind, bound, norm.data_ptr(), torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("copies", sorted(SIZES))
@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("dtype,out", [(0, 0), (1, 0), (2, 1)])
def test_copies_and_norms(copies, kind, dtype, out):
    torch = _torch()
    say("case parts", copies, kind, dtype, out)
    n = SIZES[copies]
    assert sum(n) * copies > 4096 * 8192
    c = Case(n, [dtype] * len(n), copies=copies, out=[out] * len(n), seed=copies + kind, sigma=0.05)
    want = ref_norm(c.flat64(), kind)
    norm = new_norm()
    for bound in (want / 3, want * 3, 0.0):
        for v in (v for vs in c.out_views for v in vs):
            v.fill_(7.0)
        call(c, kind, bound, norm)
        check_norm(float(norm), want)
        if bound > want:   # a copy, each value rounded once
            for vs in c.out_views:
                assert all(torch.equal(v.cpu(), x.to(v.dtype)) for v, x in zip(vs, c.values))
        elif bound == 0.0:
            assert not any(bool(v.any()) for vs in c.out_views for v in vs)
        else:
            # check_clip takes the bound as fp32 rounds it: one of its six roundings
            check_clip(c, want, bound)
    c.guards_hold()
    for vs in c.views:   # the sources stay as they were
        assert all(torch.equal(v.cpu(), x) for v, x in zip(vs, c.values))


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("bad", ["inf", "nan", "both"])
def test_infinities_and_nan(kind, bad):
    """In the first copy, whose norm it is; the factor reaches every copy."""
    torch = _torch()
    say("case parts special", kind, bad)
    c = Case(SIZES[4], copies=4, out=[0] * len(SIZES[4]), seed=4)
    if bad != "nan":
        c.values[0][8192] = -math.inf
    if bad != "inf":
        c.values[2][19999] = math.nan
    for v, x in zip(c.views[0], c.values):
        v.copy_(x)
    norm = new_norm()
    call(c, kind, 1.0, norm)
    if bad == "inf":
        assert float(norm) == math.inf
        assert bool(c.out_views[0][0][8192].isnan())
        for k, vs in enumerate(c.out_views):
            assert sum(int(v.isnan().sum()) for v in vs) == (k == 0)
            assert sum(int(v.count_nonzero()) for v in vs) == (k == 0)   # everything else is 0
    else:
        assert math.isnan(float(norm))
        assert all(bool(v.isnan().all()) for vs in c.out_views for v in vs)
    c.guards_hold()


def test_a_given_norm_and_the_same_bits():
    torch, ddp = _torch(), _lib()
    c = Case(SIZES[4], copies=4, out=[1] * len(SIZES[4]), seed=6)
    g = c.make()
    norm = new_norm()
    s = torch.cuda.current_stream().cuda_stream
    ddp.ddp_clip_grad_norm(g, 2, 0.5, norm.data_ptr(), s)
    first = [[v.clone() for v in vs] for vs in c.out_views]
    for v in (v for vs in c.out_views for v in vs):
        v.zero_()
    ddp.ddp_clip_grads(g, 0.5, norm.data_ptr(), s)
    for a, b in zip(first, c.out_views):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    check_clip(c, ref_norm(c.flat64(), 2), 0.5)


def test_replays():
    torch, ddp = _torch(), _lib()
    c = Case(SIZES[2], copies=2, out=[0] * len(SIZES[2]), seed=12)
    g = c.make()
    norm = new_norm()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ddp.ddp_clip_grad_norm(g, 2, 0.75, norm.data_ptr(), s.cuda_stream)
    for k in range(4):
        new = torch.randn(c.numel[0], generator=torch.Generator().manual_seed(k)) * (k + 1)
        c.values[0] = new
        for vs in c.views:
            vs[0].copy_(new)
        norm.fill_(-1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        replayed = [[v.clone() for v in vs] for vs in c.out_views]
        at = float(norm)
        eager = new_norm()
        ddp.ddp_clip_grad_norm(g, 2, 0.75, eager.data_ptr(), torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert at == float(eager)
        for a, b in zip(replayed, c.out_views):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
        check_norm(at, ref_norm(c.flat64(), 2))
