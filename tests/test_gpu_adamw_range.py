"""GPU: the AdamW step over the whole range of fp32, in both kinds of states, bit
for bit against the definition's operations in fp32, each rounded by itself:
gradients whose squares are subnormal, quotients that overflow, divisors near the
ends of the range. The definition is computed with numpy, whose elementwise sums,
products, quotients and roots are IEEE operations, subnormals included.

With 8-bit states the quotient d of a first moment m may be off: by a unit in its
last place, rarely, and by two where |m| is below 2^-100, at most 2^-22 of it or
2^-148. The product with the step's size and the difference then round each side
once: u = 2^-24 of each value for each side.
"""
import math

import numpy as np
import pytest

from test_gpu_adamw import Case, dequantise, quantise

pytestmark = pytest.mark.gpu

B1, B2, LR = 0.9, 0.999, 1e-3
SIZES = [5000, 1023, 1024, 1025, 129]
f32 = np.float32


def _torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def definition(g, p, m, v, decay, step, eps, b1=B1, b2=B2, lr=LR):
    """p, m, v, the root of v and the quotient of a step."""
    with np.errstate(all="ignore"):
        m = m * f32(b1) + g * f32(1.0 - b1)
        v = v * f32(b2) + (g * g) * f32(1.0 - b2)
        r = np.sqrt(v)
        d = m / (r * f32(1.0 / math.sqrt(1.0 - b2 ** step)) + f32(eps))
        p = p * f32(1.0 - lr * decay) - d * f32(lr / (1.0 - b1 ** step))
    assert all(x.dtype == f32 for x in (p, m, v, r, d))
    return p, m, v, r, d


def same(got, want, what):
    got, want = got.cpu().numpy(), np.asarray(want)
    bad = ~((got == want) | (np.isnan(got) & np.isnan(want))) if got.dtype == f32 else got != want
    assert not bad.any(), (what, int(bad.sum()), [(got[i], want[i]) for i in np.flatnonzero(bad)[:3]])


def near(got, want, d, size, m, what):
    """A parameter stepped by a quotient of the 8-bit step."""
    got, want, d, m = (np.asarray(x, np.float64) for x in (got.cpu().numpy(), want, d, m))
    with np.errstate(all="ignore"):
        err = size * (2.0 ** -22 * np.abs(d) + 2.0 ** -148) * 1.01
        err += 2 * 2.0 ** -24 * 1.01 * (size * np.abs(d) + np.abs(want)) + 2.0 ** -148
        equal = (got == want) | (np.isnan(got) & np.isnan(want))
        end = np.abs(d) >= float(np.finfo(f32).max) * (1 - 2.0 ** -22)   # one side may be beyond the range
        ok = equal | (np.abs(got - want) <= err) | (end & (np.isinf(got) | np.isinf(want)))
    assert ok.all(), (what, int((~ok).sum()), [(got[i], want[i], d[i], m[i]) for i in np.flatnonzero(~ok)[:3]])
    usual = (m == 0) | (np.abs(m) >= 2.0 ** -100)
    assert (~equal & usual).sum() <= 1e-3 * got.size, what


def step_and_compare(c, step, eps, **kw):
    """One step of the case, and everything it leaves against the definition."""
    torch = _torch()
    c.remember()
    c.step(LR, step, eps=eps, **{"beta1": kw.get("b1", B1), "beta2": kw.get("b2", B2)})
    torch.cuda.synchronize()
    for i in range(len(c.sizes)):
        g, p, m, v, ms, vs = (None if t[i] is None else t[i].cpu() for t in c.old)
        if c.bits == 8:
            r = dequantise(v, vs).numpy()
            m = dequantise(m, ms)
            with np.errstate(under="ignore"):
                v = torch.from_numpy(r * r)
        p, m, v, r, d = definition(g.numpy(), p.numpy(), m.numpy(), v.numpy(), c.decay[i], step, eps, **kw)
        if c.bits == 32:
            same(c.p[i], p, (i, "p"))
            same(c.m[i], m, (i, "m"))
            same(c.v[i], v, (i, "v"))
        else:
            near(c.p[i], p, d, LR / (1.0 - kw.get("b1", B1) ** step), m, (i, "p"))
            for x, positive, code, scale, what in ((m, False, c.m[i], c.ms[i], "m"), (r, True, c.v[i], c.vs[i], "v")):
                codes, scales = quantise(torch.from_numpy(x), positive)
                same(scale, scales.numpy(), (i, what, "scale"))
                same(code, codes.numpy(), (i, what, "codes"))


def powers(n, lo, hi, gen):
    """Random values of both signs, their logarithms spread over [lo, hi)."""
    torch = _torch()
    x = torch.exp2(torch.rand(n, generator=gen, dtype=torch.float64) * (hi - lo) + lo)
    return torch.where(torch.rand(n, generator=gen) < 0.5, -x, x).float()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [0.0, 1e-20, 1e-8])
def test_gradients_whose_squares_are_subnormal(bits, eps):
    """|g| from 1e-22 to 1e-13: (1 - beta2) g^2 from 0 over the subnormal
    numbers to 2^-96 and above. From the first step's states on."""
    torch = _torch()
    c = Case(SIZES, bits=bits, first=True)
    gen = torch.Generator().manual_seed(4)
    for step in (1, 2, 3):
        for i, n in enumerate(SIZES):
            c.g[i].copy_(powers(n, math.log2(1e-22), math.log2(1e-13), gen))
        step_and_compare(c, step, eps)


@pytest.mark.parametrize("size", [1e-19, 1e-18, 1e-17, 1e-15])
def test_the_first_step_is_the_rate_however_small_the_gradient(size):
    """With eps = 0 the first step is lr, up to the roundings: v = (1 - beta2) g^2
    is at least 2^-137 here, so a subnormal number's half step, 2^-150, is 2^-13 of
    it at most and half of that in its root; a dozen others are 2^-24 each."""
    torch = _torch()
    for bits in (32, 8):
        c = Case([1000], bits=bits, first=True, decay=0.0)
        c.g[0].fill_(size)
        c.p[0].zero_()
        c.step(LR, 1, eps=0.0)
        torch.cuda.synchronize()
        assert ((c.p[0].double() / -LR - 1.0).abs() <= 2.0 ** -14 + 12 * 2.0 ** -24).all()
        if bits == 8:   # no root is held as zero beside a first moment that is not
            assert (c.vs[0] > 0).all() and (c.v[0] > 0).all() and (c.ms[0] > 0).all()


@pytest.mark.parametrize("eps", [0.0, 2e-38, 1e-8, 1.0, 3e38])
@pytest.mark.parametrize("b2", [0.0, B2])
def test_every_magnitude_of_32_bit_states(eps, b2):
    torch = _torch()
    c = Case([200003], bits=32)
    gen = torch.Generator().manual_seed(5)
    n = 200003
    c.m[0].copy_(powers(n, -149, 128, gen))
    v = powers(n, -149, 128, gen).abs()
    v[::17] = 0.0
    c.v[0].copy_(v)
    g = powers(n, -149, 128, gen)
    g[::3] = 0.0
    c.g[0].copy_(g)
    c.p[0][::5] = 0.0
    step_and_compare(c, 2, eps, b2=b2)


@pytest.mark.parametrize("eps", [0.0, 2e-38, 1e-8, 1.0, 2.0 ** 125])
@pytest.mark.parametrize("b1,b2", [(B1, B2), (0.0, 0.0)])
def test_every_magnitude_of_8_bit_states(eps, b1, b2):
    """Blocks of 128 at magnitudes of their own; squares that stay finite, so
    that all states do."""
    torch = _torch()
    blocks = 1500
    n = blocks * 128 - 5
    c = Case([n], bits=8)
    gen = torch.Generator().manual_seed(6)

    def of(lo, hi):
        size = powers(blocks, lo, hi - 1, gen).abs().repeat_interleave(128)[:n]
        return powers(n, -14, 0, gen) * size

    for x, positive, code, scale in ((of(-100, 127), False, c.m[0], c.ms[0]), (of(-74, 62).abs(), True, c.v[0], c.vs[0])):
        new = quantise(x, positive)
        code.copy_(new[0])
        scale.copy_(new[1])
    g = of(-130, 62)
    g[::3] = 0.0
    c.g[0].copy_(g)
    step_and_compare(c, 2, eps, b1=b1, b2=b2)
