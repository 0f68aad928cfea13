"""GPU: the AdamW step against its formula in 64 bits: sizes around the tiles
and the states' blocks, every type, addresses, clipping, schedules read on the
device, graphs and streams; 8-bit states within half a step of the 64-bit
moments and bit for bit against the fp32 steps of the definition. Refusals are
in the CPU tests.

Tolerances, set before the first run, with u = 2^-24 and every operation of the
definition rounded once (products and sums of fp32, IEEE division and root):
  g = grad * f      f is a sum, a reciprocal and a product, and the product with
                    the gradient a fourth rounding: 4u relative, none without a
                    norm.
  m                 beta1 * m: the factor and the product, 2u of |beta1 m|;
                    (1 - beta1) g: 2u + 4u of |(1 - beta1) g|; the sum u of both.
                    dm = u (3 |beta1 m| + 7 |(1 - beta1) g|)
  v                 both terms are positive: 2u + u, and 2 * 4u + 3u + u, so
                    12u relative.
  denominator       positive terms: sqrt(v) 6u + u, the factor and the product
                    2u, the sum u: 10u relative.
  update            size * m / denominator: dm carries through; 10u and the
                    quotient, size and the product 3u: 13u of it.
  p                 p * keep 2u of it, the difference u of both terms.
Second orders are covered by a factor of 1.01. 16-bit parameters are rounded
once more: eps / 2 of the type, at least half the smallest subnormal.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_SUBNORMAL = {0: 2.0 ** -150, 1: 2.0 ** -134, 2: 2.0 ** -25}
BLOCK = 128
CODE = 2.0 ** -4          # half a step of an e4m3 code, relative
SMALLEST = 2.0 ** -9      # the smallest positive code; half of it is a step's half near zero


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


class Buffer:
    """Tensors of given sizes in one allocation, `gap` elements of filler
    before each and after the last."""

    def __init__(self, sizes, dtype, gap, fill):
        torch = _torch()
        n = sum(sizes) + gap * (len(sizes) + 1)
        self.flat = torch.full((max(n, 1),), fill, dtype=dtype, device="cuda")
        self.fill, self.views, at = fill, [], gap
        for s in sizes:
            self.views.append(self.flat[at:at + s])
            at += s + gap
        self.mask = torch.ones(self.flat.numel(), dtype=torch.bool, device="cuda")
        at = gap
        for s in sizes:
            self.mask[at:at + s] = False
            at += s + gap

    def ptrs(self):
        return [v.data_ptr() for v in self.views]

    def gaps_untouched(self):
        left = self.flat[self.mask]
        return bool((left == self.fill).all()) if left.numel() else True


def blocks(n):
    return -(-n // BLOCK)


def quantise(x, positive):
    """fp32 on any device: codes (uint8) and scales as the definition rounds them."""
    torch = _torch()
    n = x.numel()
    b = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)
    top = b.abs().amax(1)
    none = top < 2.0 ** -100
    scale = torch.where(none, torch.zeros_like(top), top * (1.0 / 448.0))
    up = torch.where(none, torch.zeros_like(top), top.reciprocal() * 448.0)
    code = (b * up[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    if positive:
        code = torch.where((b > 0) & (code == 0), torch.ones_like(code), code)
    return code.view(-1)[:n], scale


def dequantise(code, scale):
    torch = _torch()
    n = code.numel()
    c = torch.nn.functional.pad(code, (0, -n % BLOCK)).view(-1, BLOCK).view(torch.float8_e4m3fn).float()
    return (c * scale[:, None]).view(-1)[:n]


class Case:
    """A list of tensors with random contents, the library's list over it, and
    copies of everything from before the step."""

    def __init__(self, sizes, grad=0, param=0, copy=None, bits=32, gap=0, seed=0, sigma=1e-2, first=False, decay=0.1):
        torch, ddp = _torch(), _lib()
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed + 1)
        grads = grad if isinstance(grad, list) else [grad] * len(sizes)
        params = param if isinstance(param, list) else [param] * len(sizes)
        copies = copy if isinstance(copy, list) else [copy] * len(sizes)
        self.sizes, self.bits, self.params, self.copies = sizes, bits, params, copies
        # one buffer per tensor where the types differ
        def make(types, fill):
            if len(set(types)) <= 1:
                return [Buffer(sizes, _type(types[0]) if types else torch.float32, gap, fill)]
            return [Buffer([n], _type(t), gap, fill) for n, t in zip(sizes, types)]

        def views(bufs):
            return [v for b in bufs for v in b.views]

        self.gb, self.pb = make(grads, 7.0), make(params, 5.0)
        self.g, self.p = views(self.gb), views(self.pb)
        self.cb = [None if c is None else Buffer([n], _type(c), gap, 3.0) for n, c in zip(sizes, copies)]
        self.mb = [Buffer(sizes, torch.float32 if bits == 32 else torch.uint8, gap, 11)]
        self.vb = [Buffer(sizes, torch.float32 if bits == 32 else torch.uint8, gap, 13)]
        self.m, self.v = views(self.mb), views(self.vb)
        self.sb = [Buffer([blocks(n) for n in sizes], torch.float32, 1, f) for f in (17.0, 19.0)] if bits == 8 else []
        self.ms, self.vs = ([b.views for b in self.sb] if bits == 8 else ([None] * len(sizes),) * 2)
        for i, n in enumerate(sizes):
            # gradients over six orders of magnitude within a tensor
            spread = torch.exp(torch.randn(n, device="cuda", generator=gen) * 2.0)
            self.g[i].copy_(torch.randn(n, device="cuda", generator=gen) * spread * sigma)
            self.p[i].copy_(torch.randn(n, device="cuda", generator=gen) * 0.05)
            m = torch.randn(n, device="cuda", generator=gen) * spread * sigma * (0.0 if first else 0.3)
            r = torch.rand(n, device="cuda", generator=gen).add_(0.2) * spread * sigma * (0.0 if first else 1.0)
            if bits == 32:
                self.m[i].copy_(m)
                self.v[i].copy_(r * r)
            else:
                for x, pos, c, s in ((m, False, self.m[i], self.ms[i]), (r, True, self.v[i], self.vs[i])):
                    code, scale = quantise(x, pos)
                    c.copy_(code)
                    s.copy_(scale)
        self.decay = [decay if i % 2 == 0 else 0.0 for i in range(len(sizes))]
        self.remember()
        self.opt = ddp.make_adamw(
            sizes, [t.data_ptr() for t in self.g], [t.data_ptr() for t in self.p],
            [t.data_ptr() for t in self.m], [t.data_ptr() for t in self.v], grad_dtype=grads, param_dtype=params,
            copy_ptrs=[0 if b is None else b.views[0].data_ptr() for b in self.cb] if any(copies) else None,
            copy_dtype=[c or 1 for c in copies] if any(copies) else None,
            state=ddp.DDP_STATE_F32 if bits == 32 else ddp.DDP_STATE_8BIT,
            m_scale_ptrs=[t.data_ptr() for t in self.ms] if bits == 8 else None,
            v_scale_ptrs=[t.data_ptr() for t in self.vs] if bits == 8 else None, weight_decay=self.decay)

    def buffers(self):
        return self.gb + self.pb + [b for b in self.cb if b is not None] + self.mb + self.vb + self.sb

    def remember(self):
        self.before = [b.flat.clone() for b in self.buffers()]
        self.old = [[None if t is None else t.clone() for t in ts] for ts in
                    (self.g, self.p, self.m, self.v, self.ms, self.vs)]

    def restore(self):
        for b, o in zip(self.buffers(), self.before):
            b.flat.copy_(o)

    def contents(self):
        return [b.flat.clone() for b in self.buffers()]

    def step(self, lr=1e-3, step=10, stream=None, **kw):
        torch, ddp = _torch(), _lib()
        s = torch.cuda.current_stream().cuda_stream if stream is None else stream
        ddp.ddp_adamw_step(self.opt, lr, step, s, **kw)

    def check(self, lr, step, beta1=0.9, beta2=0.999, eps=1e-8, factor=1.0, clipped=False):
        """Everything the step left against the formula in 64 bits."""
        torch = _torch()
        torch.cuda.synchronize()
        for b in self.buffers():
            assert b.gaps_untouched()
        cg = 4 if clipped else 0
        for i, n in enumerate(self.sizes):
            if n == 0:
                continue
            g, p, m, v, ms, vs = (None if t[i] is None else t[i] for t in self.old)
            assert torch.equal(g, self.g[i]) or bool(torch.isnan(g).any())
            if self.bits == 8:
                r = dequantise(v, vs).double()
                m, v = dequantise(m, ms).double(), r * r
                # the root's square is rounded to fp32 once more
                dv0 = U
            else:
                m, v, dv0 = m.double(), v.double(), 0.0
            g = g.double() * factor
            m1, ga = beta1 * m, (1.0 - beta1) * g
            new_m = m1 + ga
            new_v = beta2 * v + (1.0 - beta2) * g * g
            dm = U * (3 * m1.abs() + (3 + cg) * ga.abs()) * 1.01 + 2.0 ** -148
            rel_v = ((4 + 2 * cg) * U + dv0) * 1.01
            den = new_v.sqrt() / math.sqrt(1.0 - beta2 ** step) + eps
            size = lr / (1.0 - beta1 ** step)
            up = size * new_m / den
            keep = p.double() * (1.0 - lr * self.decay[i])
            new_p = keep - up
            rel_den = rel_v / 2 + U * 4
            dp = (size * dm / den + (rel_den + 3 * U) * up.abs() + 3 * U * keep.abs() + U * up.abs()) * 1.01 + 2.0 ** -148
            out = self.p[i].double()
            t = self.params[i]
            if t:
                dp = dp + (torch.finfo(_type(t)).eps / 2) * (new_p.abs() + dp) + HALF_SUBNORMAL[t]
            worst = ((out - new_p).abs() / dp).max()
            assert worst <= 1, (i, n, "p", float(worst))
            if self.cb[i] is not None:   # the copy is the stepped parameter, rounded once
                assert torch.equal(self.cb[i].views[0], self.p[i].to(_type(self.copies[i])))
            if self.bits == 32:
                assert ((self.m[i].double() - new_m).abs() <= dm).all(), (i, "m")
                assert ((self.v[i].double() - new_v).abs() <= rel_v * new_v + 2.0 ** -148).all(), (i, "v")
            else:
                self.check_codes(i, new_m, dm, self.m[i], self.ms[i], False)
                new_r = new_v.sqrt()
                self.check_codes(i, new_r, (rel_v / 2 + U) * new_r, self.v[i], self.vs[i], True)

    def check_codes(self, i, x, dx, code, scale, positive):
        """Within half a step of the exact value: 2^-4 of it, or half the
        smallest code near zero; a positive root may be held as the smallest
        code instead. The scale is a product with 1 / 448, itself rounded; its
        inverse a reciprocal times 448, both rounded; the products u each."""
        torch = _torch()
        n = x.numel()
        top = torch.nn.functional.pad(x.abs(), (0, -n % BLOCK)).view(-1, BLOCK).amax(1)
        dtop = torch.nn.functional.pad(dx, (0, -n % BLOCK)).view(-1, BLOCK).amax(1)
        assert ((scale.double() - top / 448.0).abs() <= (2 * U * top + dtop) / 448.0 * 1.01 + 2.0 ** -149).all(), (i, "scale")
        per = scale.double().repeat_interleave(BLOCK)[:n]
        got = dequantise(code, scale).double()
        near = (CODE * x.abs()).maximum(SMALLEST / 2 * per)
        if positive:
            near = torch.where(x < SMALLEST * per, (SMALLEST * per - x).maximum(near), near)
            assert ((code > 0) | (x <= 2.0 ** -74)).all()
        slack = dx * 1.2 + 8 * U * x.abs() + 2.0 ** -148
        assert ((got - x).abs() <= near + slack).all(), (i, "codes", float(((got - x).abs() - near - slack).max()))


SIZES = [1, 2, 3, 4, 5, 127, 128, 129, 255, 256, 257, 1023, 2047, 2048, 2049, 4096, 6145, 0, 70001]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gap", [0, 1, 3, 64])
def test_sizes_and_addresses(bits, gap):
    say("sizes", bits, gap)
    c = Case(SIZES, bits=bits, gap=gap, seed=gap)
    c.step(1e-3, 10)
    c.check(1e-3, 10)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", [0, 1, 2])
@pytest.mark.parametrize("param,copy", [(0, None), (0, 1), (0, 2), (1, None), (2, None)])
def test_types(bits, grad, param, copy):
    say("types", bits, grad, param, copy)
    c = Case([5, 2048, 130, 9001], grad=grad, param=param, copy=copy, bits=bits, gap=1, seed=3)
    c.step(1e-3, 100)
    c.check(1e-3, 100)


@pytest.mark.parametrize("bits", [32, 8])
def test_types_mixed_in_one_list(bits):
    grads, params, copies = [], [], []
    for g in (0, 1, 2):
        for p, k in ((0, None), (0, 1), (0, 2), (1, None), (2, None)):
            grads.append(g), params.append(p), copies.append(k)
    c = Case([2048 + 37 * i for i in range(15)], grad=grads, param=params, copy=copies, bits=bits, gap=2, seed=5)
    c.step(1e-3, 3)
    c.check(1e-3, 3)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("step", [1, 2, 1000, 10 ** 6, 2 ** 40])
def test_steps_and_first_states(bits, step):
    c = Case([300, 5000], bits=bits, seed=7, first=step == 1)
    c.step(3e-4, step, beta1=0.8, beta2=0.95, eps=1e-6)
    c.check(3e-4, step, beta1=0.8, beta2=0.95, eps=1e-6)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("ratio", [0.0, 0.25, 0.999, 1.0, 4.0, math.inf])
def test_clipping_by_a_norm(bits, ratio):
    torch = _torch()
    c = Case([300, 5000], bits=bits, seed=8, grad=1)
    norm = torch.tensor([3.7], device="cuda")
    c.step(1e-3, 10, norm=norm.data_ptr(), max_norm=3.7 * ratio)
    f = 1.0 if ratio == math.inf else min(1.0, float(torch.tensor(3.7 * ratio)) / (float(norm) + 1e-6))
    c.check(1e-3, 10, factor=f, clipped=True)


@pytest.mark.parametrize("bits", [32, 8])
def test_zeros_stay_zeros(bits):
    """No gradient, no moments, eps > 0: only the decay moves a parameter."""
    torch = _torch()
    c = Case([1000], bits=bits, first=True)
    c.g[0].zero_()
    c.remember()
    c.step(0.5, 1)
    torch.cuda.synchronize()
    assert (c.m[0] == 0).all() and (c.v[0] == 0).all()
    keep = 1.0 - 0.5 * 0.1
    assert torch.equal(c.p[0], c.old[1][0] * torch.tensor(keep, dtype=torch.float32, device="cuda"))
    if bits == 8:
        assert (c.ms[0] == 0).all() and (c.vs[0] == 0).all()


@pytest.mark.parametrize("gap", [0, 3])
@pytest.mark.parametrize("copy", [None, 1])
def test_8_bit_steps_bit_for_bit(gap, copy):
    """Three steps against the definition's fp32 operations on the CPU."""
    torch = _torch()
    c = Case(SIZES, bits=8, gap=gap, copy=copy, grad=0, seed=11)
    norm = torch.tensor([2.0], device="cuda")
    lr, b1, b2, eps = 1e-3, 0.9, 0.999, 1e-8
    state = [[t[i].cpu() for t in (c.p, c.m, c.v, c.ms, c.vs, c.g)] for i in range(len(SIZES))]
    f = (torch.tensor(2.0) + torch.tensor(1e-6)).reciprocal() * 1.0
    for step in (4, 5, 6):
        c.step(lr, step, norm=norm.data_ptr(), max_norm=1.0)
        root, size = 1.0 / math.sqrt(1.0 - b2 ** step), lr / (1.0 - b1 ** step)
        for i, s in enumerate(state):
            p, m, v, ms, vs, g = s
            g = g * f
            m = dequantise(m, ms) * b1 + g * (1.0 - b1)
            r = dequantise(v, vs)
            # torch's root on the CPU is not always the nearest fp32 value; that of the 64-bit root is
            r = ((r * r) * b2 + (g * g) * (1.0 - b2)).double().sqrt().float()
            p = p * (1.0 - lr * c.decay[i]) - (m / (r * root + eps)) * size
            (code_m, scale_m), (code_v, scale_v) = quantise(m, False), quantise(r, True)
            s[:5] = p, code_m, code_v, scale_m, scale_v
    torch.cuda.synchronize()
    for i, (p, m, v, ms, vs, g) in enumerate(state):
        for name, want, got in (("p", p, c.p[i]), ("m", m, c.m[i]), ("v", v, c.v[i]), ("ms", ms, c.ms[i]),
                                ("vs", vs, c.vs[i])):
            assert torch.equal(want, got.cpu()), (i, SIZES[i], name)


def test_a_positive_root_keeps_a_positive_code():
    """One large gradient in a block of tiny ones: their roots are far below
    the smallest code, and are held as that."""
    torch = _torch()
    c = Case([256], bits=8, first=True)
    c.g[0].fill_(1e-7)
    c.g[0][5] = 100.0
    c.g[0][200] = 0.0
    c.remember()
    c.step(1e-3, 1)
    c.check(1e-3, 1)
    assert c.v[0][:128].tolist().count(1) == 127 and c.v[0][5] == 0x7e
    assert c.v[0][200] == 0 and (c.v[0][128:200] == 0x7e).all()
    c.g[0].zero_()   # nothing new: the step stays of the old step's size
    before = c.p[0].clone()
    c.step(1e-3, 2)
    torch.cuda.synchronize()
    assert (c.p[0] - before).abs().max() < 5e-3


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_gradients_that_are_not_finite_without_a_norm(bad):
    torch = _torch()
    c = Case([1000], bits=32, seed=2)
    c.g[0][700] = bad
    c.step(1e-3, 10)
    d = Case([1000], bits=8, seed=2)
    d.g[0][700] = bad
    d.step(1e-3, 10)
    torch.cuda.synchronize()
    for x in (c.p[0], d.p[0]):
        assert torch.isnan(x).nonzero().tolist() == [[700]]
    assert torch.isfinite(c.m[0]).logical_not().nonzero().tolist() == [[700]]
    m, r = dequantise(d.m[0], d.ms[0]), dequantise(d.v[0], d.vs[0])
    hit = torch.zeros(1000, dtype=torch.bool, device="cuda")
    hit[640:768] = True   # its block: codes times a scale that is not finite; positive codes times inf are inf
    assert torch.equal(torch.isnan(m), hit) and torch.equal(torch.isfinite(r), ~hit)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_norms_that_are_not_finite(bits, bad):
    torch = _torch()
    c = Case([1000, 3000], bits=bits, copy=1)
    norm = torch.tensor([bad], device="cuda")
    c.step(1e-3, 10, norm=norm.data_ptr(), max_norm=1.0, skip_nonfinite=True)
    c.step(1e-3, 10, norm=norm.data_ptr(), max_norm=math.inf, skip_nonfinite=True)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(c.before, c.contents()))
    c.step(1e-3, 10, norm=norm.data_ptr(), max_norm=1.0)
    if math.isnan(bad):
        torch.cuda.synchronize()
        assert torch.isnan(c.p[0]).all()
    else:   # finite gradients times 0
        c.check(1e-3, 10, factor=0.0, clipped=True)
    # a finite norm is not skipped
    c.restore()
    norm.fill_(2.0)
    c.step(1e-3, 10, norm=norm.data_ptr(), max_norm=1.0, skip_nonfinite=True)
    c.check(1e-3, 10, factor=1.0 / (2.0 + 1e-6), clipped=True)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("step", [1, 7, 12345, 2 ** 33])
def test_schedules_read_on_the_device_give_the_same_bits(bits, step):
    torch = _torch()
    c = Case([1000, 3000], bits=bits, copy=2)
    lr = torch.tensor([3e-4], device="cuda")
    t = torch.tensor([step], device="cuda")
    c.step(float(lr), step)
    want = c.contents()
    for kw in ({"step_ptr": t.data_ptr()}, {"lr_ptr": lr.data_ptr()},
               {"step_ptr": t.data_ptr(), "lr_ptr": lr.data_ptr()}):
        c.restore()
        c.step(math.nan if "lr_ptr" in kw else float(lr), 0 if "step_ptr" in kw else step, **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, c.contents())), kw
    t.fill_(-5)   # counts as 1
    c.restore()
    c.step(float(lr), 0, step_ptr=t.data_ptr())
    got = c.contents()
    c.restore()
    c.step(float(lr), 1)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, c.contents()))


@pytest.mark.parametrize("bits", [32, 8])
def test_recorded_steps_follow_the_schedule(bits):
    """Replays advance the step and the rate on the device; every replay
    equals the eager step, with eager work between."""
    torch = _torch()
    c, e = (Case([1000, 70000, 5], bits=bits, copy=1, grad=1, seed=21) for _ in range(2))
    lr, t = torch.tensor([1e-3], device="cuda"), torch.tensor([0], device="cuda")
    norm = torch.tensor([2.0], device="cuda")
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        t.add_(1)
        c.step(0.0, 0, lr_ptr=lr.data_ptr(), step_ptr=t.data_ptr(), norm=norm.data_ptr(), max_norm=1.0)
        lr.mul_(0.5)
    rate = torch.tensor([1e-3], device="cuda")
    for k in range(1, 5):
        graph.replay()
        e.step(float(rate), k, norm=norm.data_ptr(), max_norm=1.0)
        rate.mul_(0.5)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(c.contents(), e.contents())), k
        c.g[0].mul_(1.5)
        e.g[0].mul_(1.5)


def test_lists_step_on_streams_of_their_own():
    torch = _torch()
    cases = [Case([200000, 33], bits=b, seed=s) for b, s in ((32, 1), (8, 2), (32, 3), (8, 4))]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for k in (1, 2, 3):
        for c, s in zip(cases, streams):
            c.step(1e-3, k, stream=s.cuda_stream)
    torch.cuda.synchronize()
    got = [c.contents() for c in cases]
    for c in cases:
        c.restore()
        for k in (1, 2, 3):
            c.step(1e-3, k)
    torch.cuda.synchronize()
    for c, g in zip(cases, got):
        assert all(torch.equal(a, b) for a, b in zip(c.contents(), g))


@pytest.mark.parametrize("bits", [32, 8])
def test_two_tensors_with_one_gradient(bits):
    """Replicas' parameters that step from one reduced gradient."""
    torch, ddp = _torch(), _lib()
    c, d = (Case([5000], bits=bits, seed=3) for _ in range(2))
    o = ddp.make_adamw(
        [5000, 5000], [c.g[0].data_ptr()] * 2, [x.p[0].data_ptr() for x in (c, d)], [x.m[0].data_ptr() for x in (c, d)],
        [x.v[0].data_ptr() for x in (c, d)], state=ddp.DDP_STATE_F32 if bits == 32 else ddp.DDP_STATE_8BIT,
        m_scale_ptrs=[x.ms[0].data_ptr() for x in (c, d)] if bits == 8 else None,
        v_scale_ptrs=[x.vs[0].data_ptr() for x in (c, d)] if bits == 8 else None, weight_decay=0.1)
    ddp.ddp_adamw_step(o, 1e-3, 10, torch.cuda.current_stream().cuda_stream)
    c.check(1e-3, 10)
    assert all(torch.equal(a, b) for a, b in zip(c.contents(), d.contents()))


def test_special_streams_and_an_empty_list():
    torch, ddp = _torch(), _lib()
    c = Case([4000], bits=32)
    c.step(1e-3, 1)
    want = c.contents()
    for stream in (0, 1, 2):   # null, legacy, per-thread
        c.restore()
        torch.cuda.synchronize()
        c.step(1e-3, 1, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, c.contents()))
    for sizes in ([], [0], [0, 0]):
        none = [0] * len(sizes)
        o = ddp.make_adamw(sizes, none, none, none, none)
        ddp.ddp_adamw_step(o, 1e-3, 1, 0)
        ddp.ddp_adamw_destroy(o)


def test_a_dropped_list_keeps_its_tables_for_queued_steps():
    torch = _torch()
    c, e = (Case([3_000_000], bits=8, seed=4) for _ in range(2))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for k in range(1, 20):
        c.step(1e-3, k, stream=s.cuda_stream)
    c.opt = None
    trash = [torch.full((1 << 16,), 0x7f, dtype=torch.uint8, device="cuda") for _ in range(64)]
    for k in range(1, 20):
        e.step(1e-3, k)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(c.contents(), e.contents()))
    del trash


@pytest.mark.parametrize("bits", [32, 8])
def test_a_flat_buffer_of_odd_views_equals_separate_tensors(bits):
    """The same tensors at other addresses give the same bits."""
    torch = _torch()
    c = Case(SIZES, bits=bits, gap=0, seed=9)
    d = Case(SIZES, bits=bits, gap=128, seed=9)
    for x in (c, d):
        x.step(1e-3, 5)
    torch.cuda.synchronize()
    for a, b in zip(c.p + c.m + c.v, d.p + d.m + d.v):
        assert torch.equal(a, b)


def test_more_elements_than_a_launch_holds():
    """2^33 elements and some, in 16 bits with 8-bit states: the last ones step
    as in a list of their own."""
    torch, ddp = _torch(), _lib()
    n, tail = (1 << 33) + 5000, 9000
    c = Case([tail], grad=1, param=1, bits=8, seed=6, decay=0.1)
    big = {k: torch.zeros(n, dtype=t, device="cuda") for k, t in
           (("g", torch.bfloat16), ("p", torch.bfloat16), ("m", torch.uint8), ("v", torch.uint8))}
    scales = [torch.zeros(blocks(n), device="cuda") for _ in range(2)]
    lead = (n - tail) // BLOCK * BLOCK   # a block's border
    k = tail // BLOCK * BLOCK
    for name, t in (("g", c.g[0]), ("p", c.p[0]), ("m", c.m[0]), ("v", c.v[0])):
        big[name][lead:lead + k] = t[:k]
    for s, t in zip(scales, (c.ms[0], c.vs[0])):
        s[lead // BLOCK:lead // BLOCK + k // BLOCK] = t[:k // BLOCK]
    opt = ddp.make_adamw([n], [big["g"].data_ptr()], [big["p"].data_ptr()], [big["m"].data_ptr()], [big["v"].data_ptr()],
                         grad_dtype=[1], param_dtype=[1], state=ddp.DDP_STATE_8BIT, m_scale_ptrs=[scales[0].data_ptr()],
                         v_scale_ptrs=[scales[1].data_ptr()], weight_decay=0.1)
    ddp.ddp_adamw_step(opt, 1e-3, 10, torch.cuda.current_stream().cuda_stream)
    c.step(1e-3, 10)
    torch.cuda.synchronize()
    for name, t in (("p", c.p[0]), ("m", c.m[0]), ("v", c.v[0])):
        assert torch.equal(big[name][lead:lead + k], t[:k]), name
    assert not big["p"][:1 << 20].any() and not big["m"][lead - (1 << 20):lead].any()
