"""GPU: the embedding table's gradient of whole numbers, bit for bit.

The rows of dout are whole numbers of -3..3, the old gradient's of -100..100,
the scale a power of two between 1/2 and 2. Any partial sum of up to 800,000
positions is a multiple of 1/2 below 3 * 800000 * 2 + 100 < 2^23, which float32
holds exactly (24 bits: multiples of 1/2 up to 2^23), so the sum is the same
number in whatever order it is taken and the one rounding to a 16-bit gradient
has one right result. A piece of a frequent token's run that is lost, doubled
or put elsewhere shows, however many positions the token has: rounding bounds
grow with them, whole numbers do not.
"""
import pytest

from test_gpu_embedding import Case, _torch, outside, say

pytestmark = pytest.mark.gpu

FEW, MANY = 64, 600000   # rows for the single launch, and for several whatever the number of positions


def whole(shape, most, seed, dtype):
    torch = _torch()
    return torch.randint(-most, most + 1, shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def check(c, accumulate, seed):
    torch = _torch()
    dout = whole((c.T, c.H), 3, seed + 1, torch.float64)
    old = whole((c.V, c.H), 100, seed + 2, torch.float64)
    c.act.copy_(dout.to(c.act.dtype))
    c.row.copy_(old.to(c.row.dtype))
    r = c.host_tokens - c.first
    held = (r >= 0) & (r < c.V)
    if c.padding >= 0:
        held &= c.host_tokens != c.padding
    want = torch.zeros(c.V, c.H, dtype=torch.float64).index_add_(0, r[held], dout[held]) * c.scale
    assert float(want.abs().max()) < 2 ** 23
    if accumulate:
        want += old
    c.grad(accumulate)
    got = c.row.cpu()
    want = want.float().to(got.dtype)
    assert bool((outside(c.row_buf, c.row) == 9.0).all())
    bad = got != want
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:5], got[bad][:5], want[bad][:5])


@pytest.mark.parametrize("T,V,H,kind,act,row", [
    (40000, 300, 64, "falling", 1, 0), (40000, 32000, 513, "falling", 1, 0), (70000, 7, 20, "uniform", 1, 1),
    (33000, 1000, 2048, "same", 1, 0), (33000, 1000, 2048, "two", 1, 1), (200000, 50000, 8, "two", 1, 0),
    (200000, 50000, 8, "same", 0, 0), (20000, 2, 3, "uniform", 2, 0), (600000, 300, 4, "falling", 1, 0),
    (600000, 3, 5, "falling", 0, 2), (530000, 3000, 5, "uniform", 1, 0), (140000, 400000, 4, "falling", 1, 0),
    (70001, 1, 33, "same", 1, 0), (800000, 40, 1, "two", 2, 0)])
@pytest.mark.parametrize("accumulate", [True, False])
def test_long_runs(T, V, H, kind, act, row, accumulate):
    say("case exact long", T, V, H, kind, act, row, accumulate)
    check(Case(T, V, H, kind=kind, act=act, row=row, scale=2.0, seed=5), accumulate, T)


@pytest.mark.parametrize("T", [1, 9, 64, 65, 1000, 2047, 2048, 4096, 4097, 9000])
@pytest.mark.parametrize("kind", ["same", "two", "falling", "wild"])
@pytest.mark.parametrize("V,H", [(FEW, 68), (MANY, 20), (30522, 256)])
def test_few_and_some_tokens(T, kind, V, H):
    say("case exact few", T, kind, V, H)
    check(Case(T, V, H, kind=kind, scale=0.5, first=7, padding=9, seed=T), T % 2 == 0, T)


# Positions of a chunk grow with the positions of a call (rows of four columns):
# 8 up to 65536, 16 up to 131072, then 32. Up to 4096 positions of a small table
# go the way of the single launch.
@pytest.mark.parametrize("chunk,T,V", [(8, 0, FEW), (8, 0, MANY), (8, 20000, 4000), (16, 80000, 4000), (32, 150000, 4000)])
@pytest.mark.parametrize("pieces", [2, 3, 15, 16, 17, 18, 33, 64, 300])
def test_a_run_of_so_many_pieces(chunk, T, V, pieces):
    """One token of chunk * pieces positions and a few, behind a few others, at
    three places relative to the chunks' borders."""
    torch = _torch()
    say("case exact pieces", chunk, T, V, pieces)
    step = V // 64
    for before, more in ((0, 0), (3, 1), (chunk - 1, chunk - 1)):
        tok = torch.cat([torch.arange(before) % 3, torch.full((chunk * pieces + more,), 10),
                         torch.arange(11, 20), torch.full((2 * chunk + 1,), 40)]) * step
        g = torch.Generator().manual_seed(pieces)
        tok = torch.cat([tok, torch.randint(41 * step, V, (max(0, T - tok.numel()),), generator=g)])
        tok = tok[torch.randperm(tok.numel(), generator=g)]
        c = Case(tok.numel(), V, 4, act=1, seed=pieces)
        c.host_tokens = tok
        c.tokens.copy_(tok)
        check(c, pieces % 2 == 0, pieces)


@pytest.mark.parametrize("accumulate", [True, False])
@pytest.mark.parametrize("T,V,H", [(30000, 50, 129), (30000, 3000, 16), (200000, 20, 7)])
@pytest.mark.parametrize("frequent", [0, 1, 9])
def test_frequent_padding_among_frequent_tokens(T, V, H, accumulate, frequent):
    """A third of the positions are padding, a third one other token."""
    torch = _torch()
    c = Case(T, V, H, kind="falling", act=1, padding=frequent, scale=2.0, seed=8)
    turn = torch.arange(T) % 3
    c.host_tokens = torch.where(turn == 0, torch.full((T,), frequent),
                                torch.where(turn == 1, torch.full((T,), 10), c.host_tokens))
    c.tokens.copy_(c.host_tokens)
    check(c, accumulate, T)
