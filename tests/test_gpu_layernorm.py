"""GPU: the layer norm's two passes against their formulas in 64 bits: widths
around the vectors and the kernels' limits, odd ones, every type, strides and
addresses, rows far off centre and constant ones, in place, infinities and NaN,
graphs and streams; the gradient against the formula's and against differences.
Refusals are in the CPU tests.

Tolerances, set before the first run, with u = 2^-24. A sum over a row goes
through at most P = 100 additions: 16 to 64 in a thread, 6 over a wave, up to 16
waves, and the few of one vector.
  z      one rounding of an fp32 sum: compared bit for bit.
  mean   the rounded mean m, plus the mean of z - m: u |mean| and P + 3 times u
         of the mean deviation A = mean |z - m|, where |z - m| is at most
         |z - mean| + P u mean |z|.
  rstd   squares P + 4, twice the deviations' rounding, quotient, eps: P + 8 of
         the variance, half of it for the root, root and quotient 2u:
         D = P / 2 + 6.
  y      deviation: u |z - m| twice and (P + 3) u A, all times rstd * weight; D
         and two products; the sum with the bias u. Then eps / 2 of y's type.
  dx     hat 2u, d = dy * weight u; the sums (P + 4) u of the mean of |d| and of
         |d * hat|, with quotient; then 4 operations each rounded once, with dz
         another; eps / 2 of x's type.
  dweight, dbias   a sum over the rows in S additions: (S + 4) u of the sum of
         magnitudes; eps / 2 of the type.
Second orders are covered by a factor of 1.01; below the smallest normal value a
rounding is absolute: half the smallest subnormal.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
P = 100
D = P / 2 + 6
HALF_SUBNORMAL = {0: 2.0 ** -150, 1: 2.0 ** -134, 2: 2.0 ** -25}
PAIRS = [(0, 0), (0, 1), (0, 2), (1, 1), (2, 2)]   # x, y
WIDTHS = [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 63, 64, 65, 100, 127, 128, 255, 256, 257, 380, 500, 511, 512, 513, 640,
          768, 769, 1000, 1023, 1024, 1025, 1281, 1530, 1537, 2047, 2048, 2049, 2559, 2561, 4095, 4096, 4097, 5000,
          5119, 5121, 6143, 6145, 8191, 8192, 8193, 10239, 10241, 12287, 12289, 16383, 16384, 16385, 32767, 32768,
          32769, 40001]


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


def ptr(t):
    return t.data_ptr() if t is not None and t.numel() else 0


def strided(rows, width, stride, dtype, seed, shift=0, sigma=1.0, off=0.0, filler=9.0):
    """A [rows, width] view with the given row stride, `shift` elements into
    its buffer, of random values; everything else of the buffer is filler."""
    torch = _torch()
    n = shift + (rows - 1) * stride + width + 5 if rows else shift + 5
    buf = torch.full((max(n, 1),), filler, dtype=dtype, device="cuda")
    v = torch.as_strided(buf, (rows, width), (stride, 1), shift)
    if rows and width:
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 1)
        # a stride of 0 repeats one row
        r = torch.randn(1 if stride == 0 else rows, width, device="cuda", generator=g) * sigma + off
        v[:1 if stride == 0 else rows].copy_(r.to(dtype))
    return buf, v


def outside(buf, view):
    torch = _torch()
    mask = torch.ones(buf.numel(), dtype=torch.bool, device="cuda")
    torch.as_strided(mask, view.shape, view.stride(), view.storage_offset()).fill_(False)
    return buf[mask]


def rounded(err, x, t):
    """err of an fp32 value, and its rounding to type t."""
    torch = _torch()
    return err if t == 0 else err + (torch.finfo(_type(t)).eps / 2) * (x.abs() + err) + HALF_SUBNORMAL[t]


def close(got, want, err, what):
    bad = (got.double() - want).abs() - err
    assert got.shape == want.shape and not bad.isnan().any() and (bad <= 0).all(), (
        what, float(bad.max()), int(bad.argmax()), float(((got.double() - want).abs() / err).max()))


class Forward:
    def __init__(self, rows, width, kind=0, x=0, y=0, weight=0, affine=3, add=None, z=True, stats=True, eps=1e-5,
                 strides=(0, 0, 0, 0), shift=0, sigma=1.0, off=0.0, seed=0):
        """affine: 1 weight, 2 bias. add: None, "rows" or "row". strides: what
        each is more than the width."""
        torch, ddp = _torch(), _lib()
        sx, sa, sz, sy = (width + s for s in strides)
        self.rows, self.width, self.kind, self.x_type, self.y_type, self.eps = rows, width, kind, x, y, eps
        self.xb, self.x = strided(rows, width, sx, _type(x), seed, shift, sigma, off)
        self.add = None
        if add:
            self.ab, self.add = strided(rows, width, 0 if add == "row" else sa, _type(x), seed + 50, shift, sigma * 0.5)
        self.zb, self.z = strided(rows, width, sz, _type(x), seed, shift, 0.0, 4.0) if add and z else (None, None)
        self.yb, self.y = strided(rows, width, sy, _type(y), seed, shift, 0.0, 5.0)
        w = strided(1, width, width, _type(weight), seed + 60, shift, 0.5, 1.0)[1][0]
        b = strided(1, width, width, _type(weight), seed + 70, shift, 0.5)[1][0]
        self.weight, self.bias = w if affine & 1 else None, b if affine & 2 else None
        self.mean, self.rstd = (torch.full((rows + 1,), 6.0, device="cuda") if stats else None for _ in range(2))
        self.desc = ddp.LayerNormDesc(width, kind=kind, x_dtype=x, y_dtype=y, weight_dtype=weight, eps=eps, x_stride=sx,
                                      add_stride=0 if add == "row" else sa, z_stride=sz, y_stride=sy)
        self.x0 = self.x.clone()

    def run(self, stream=None):
        torch, ddp = _torch(), _lib()
        s = torch.cuda.current_stream().cuda_stream if stream is None else stream
        ddp.ddp_layernorm(self.desc, self.rows, ptr(self.x), ptr(self.weight), ptr(self.bias), ptr(self.y), s,
                          add=ptr(self.add), z=ptr(self.z), mean=ptr(self.mean), rstd=ptr(self.rstd))

    def expected(self):
        z = self.x0
        if self.add is not None:
            z = (z.float() + self.add.float()).to(z.dtype)
        z64 = z.double()
        mean = z64.mean(1, keepdim=True) if self.kind == 0 else z64[:, :1] * 0
        dev = z64 - mean
        rstd = (dev.square().mean(1, keepdim=True) + self.eps).rsqrt()
        return z, mean, dev, rstd

    def check(self, untouched=True):
        torch = _torch()
        torch.cuda.synchronize()
        if untouched:
            assert (outside(self.yb, self.y) == 9.0).all() and (outside(self.xb, self.x) == 9.0).all()
            assert torch.equal(self.x, self.x0)
        z, mean, dev, rstd = self.expected()
        if self.z is not None:
            assert torch.equal(self.z, z)
            if untouched:
                assert (outside(self.zb, self.z) == 9.0).all()
        spread = dev.abs() + P * U * z.double().abs().mean(1, keepdim=True) * (self.kind == 0)
        A = spread.mean(1, keepdim=True) * (self.kind == 0)
        # eps keeps the variance's relative error small where a row is nearly constant
        shift = P * U * z.double().abs().mean(1, keepdim=True) * (self.kind == 0)
        drel = (D * U + (2 * (P + 4) * U * shift * (A + shift)) * rstd.square()) * 1.01
        if self.mean is not None:
            if self.kind == 0:
                close(self.mean[:self.rows], mean[:, 0], (U * mean.abs() + (P + 3) * U * A)[:, 0] * 1.01 + 2.0 ** -148, "mean")
            else:
                assert (self.mean[:self.rows] == 0).all()
            assert self.mean[self.rows] == 6.0 and self.rstd[self.rows] == 6.0
            close(self.rstd[:self.rows], rstd[:, 0], (drel * rstd)[:, 0], "rstd")
        w = self.weight.double() if self.weight is not None else torch.ones_like(dev[0])
        b = self.bias.double() if self.bias is not None else torch.zeros_like(dev[0])
        y = dev * rstd * w + b
        err = ((3 * U * spread + (P + 3) * U * A) * rstd * w.abs() + (drel + 3 * U) * (dev * rstd * w).abs()
               + U * y.abs()) * 1.01 + 2.0 ** -148
        close(self.y, y, rounded(err, y, self.y_type), "y")


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("x,y", PAIRS)
def test_forward_widths(kind, x, y):
    for width in WIDTHS:
        say("width", width)
        f = Forward(5, width, kind, x, y, weight=x, add="rows" if width % 2 else None, strides=(1, 2, 3, 4), shift=width % 3,
                    seed=width)
        f.run()
        f.check()


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 63, 257, 4099])
@pytest.mark.parametrize("width", [6, 40, 100, 200, 768, 1024, 2050])
def test_forward_rows(rows, width):
    for kind, (x, y) in ((0, (1, 1)), (1, (0, 2))):
        f = Forward(rows, width, kind, x, y, weight=0, add="rows", seed=rows)
        f.run()
        f.check()


@pytest.mark.parametrize("affine", [0, 1, 2, 3])
@pytest.mark.parametrize("weight", [0, 1, 2])
@pytest.mark.parametrize("add,z", [(None, False), ("rows", True), ("rows", False), ("row", True)])
def test_forward_arguments(affine, weight, add, z):
    for width in (5, 520, 3001, 20003):
        say(width)
        f = Forward(3, width, affine % 2, 0, 1, weight, affine, add, z, stats=affine != 1, strides=(7, 0, 1, 2), seed=3)
        f.run()
        f.check()


@pytest.mark.parametrize("width", [64, 1000, 4096, 16390, 33000])
@pytest.mark.parametrize("off", [0.0, 30.0, 1e4])
def test_rows_far_off_centre(width, off):
    for rows_equal in (False, True):
        f = Forward(4, width, 0, 0, 0, off=off, sigma=0.0 if rows_equal else 1.0)
        f.run()
        f.check()


def test_constant_and_zero_rows():
    torch = _torch()
    for kind in (0, 1):
        f = Forward(3, 700, kind, sigma=0.0, off=0.0, eps=1e-5)
        f.run()
        f.check()
        assert torch.equal(f.y, f.bias.expand(3, -1))
        g = Forward(2, 700, kind, sigma=0.0, off=0.0, eps=0.0)   # 0 * inf
        g.run()
        torch.cuda.synchronize()
        assert torch.isnan(g.y).all() and torch.isinf(g.rstd[:2]).all()


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("width", [9, 1001, 20001, 33001])
def test_values_that_are_not_finite_stay_in_their_row(bad, width):
    """Also in the columns that the last, overlapping vector loads twice."""
    torch = _torch()
    for col in (0, width // 2, width - 1, width - 2):
        f, clean = (Forward(5, width, 0, 0, 1, seed=4) for _ in range(2))
        f.x[2, col] = bad
        f.run()
        clean.run()
        torch.cuda.synchronize()
        assert torch.isnan(f.y[2]).all() and torch.isnan(f.rstd[2])
        others = [0, 1, 3, 4]
        assert torch.equal(f.y[others], clean.y[others]) and torch.equal(f.mean[others], clean.mean[others])


@pytest.mark.parametrize("width", [5, 100, 2047, 4100, 16391, 33001])
@pytest.mark.parametrize("where", ["y is x", "z is x", "z is add", "z is x and y is add"])
def test_forward_in_place(width, where):
    torch = _torch()
    for kind in (0, 1):
        f = Forward(7, width, kind, 0, 0, add="rows", z="z" in where, seed=6)
        g = Forward(7, width, kind, 0, 0, add="rows", z="z" in where, seed=6)
        f.run()
        if "z is x" in where:
            g.z = g.x
        if "z is add" in where:
            g.z = g.add
        if "y is x" in where:
            g.y = g.x
        if "y is add" in where:
            g.y = g.add
        g.run()
        torch.cuda.synchronize()
        assert torch.equal(f.y, g.y) and (f.z is None or torch.equal(f.z, g.z))


def test_interleaved_rows():
    """x and y as the halves of one buffer's rows."""
    torch, ddp = _torch(), _lib()
    buf = torch.randn(9, 2 * 300, device="cuda")
    x, y = buf[:, :300], buf[:, 300:]
    f = Forward(9, 300, 0, affine=0, stats=False)
    f.x.copy_(x)
    f.run()
    d = ddp.LayerNormDesc(300, x_stride=600, y_stride=600)
    ddp.ddp_layernorm(d, 9, x.data_ptr(), 0, 0, y.data_ptr(), 0)
    torch.cuda.synchronize()
    assert torch.equal(f.y, y) and torch.equal(f.x, x)


class Backward:
    def __init__(self, rows, width, kind=0, x=0, y=0, weight=0, grad=0, affine=True, dz=True, dx=True, sums=3,
                 accumulate=True, strides=(0, 0, 0), shift=0, seed=0, dy_row=False, off=0.0):
        torch, ddp = _torch(), _lib()
        sx, sz, sy = (width + s for s in strides)
        self.rows, self.width, self.kind, self.x_type, self.y_type = rows, width, kind, x, y
        self.grad_type, self.accumulate = grad, accumulate
        self.z = strided(rows, width, sz, _type(x), seed, shift, 1.0, off)[1]
        self.dyb, self.dy = strided(rows, width, 0 if dy_row else sy, _type(y), seed + 40, shift, 1e-2)
        self.dz = strided(rows, width, sz, _type(x), seed + 50, shift, 1e-2)[1] if dz else None
        self.dxb, self.dx = strided(rows, width, sx, _type(x), seed, shift, 0.0) if dx else (None, None)
        self.weight = strided(1, width, width, _type(weight), seed + 60, shift, 0.5, 1.0)[1][0] if affine else None
        self.dw, self.db = (strided(1, width, width, _type(grad), seed + k, shift, 1e-2)[1][0] if sums & m else None
                            for k, m in ((80, 1), (90, 2)))
        z = self.z.double()
        m = z.mean(1, keepdim=True) if kind == 0 else z[:, :1] * 0
        self.mean = m[:, 0].float() if kind == 0 else None
        self.rstd = ((z - m).square().mean(1) + 1e-5).rsqrt().float()
        self.desc = ddp.LayerNormDesc(width, kind=kind, x_dtype=x, y_dtype=y, weight_dtype=weight, grad_dtype=grad,
                                      x_stride=sx, z_stride=sz, y_stride=0 if dy_row else sy)
        self.bytes = ddp.ddp_layernorm_grad_workspace_bytes(self.desc, rows)
        self.work = torch.full((self.bytes + 256,), 0xff, dtype=torch.uint8, device="cuda")   # NaN, to be written first
        self.old = [t.clone() if t is not None else None for t in (self.dw, self.db, self.dy, self.dz)]

    def run(self, stream=None, work=None):
        torch, ddp = _torch(), _lib()
        s = torch.cuda.current_stream().cuda_stream if stream is None else stream
        work = self.work if work is None else work
        ddp.ddp_layernorm_grad(self.desc, self.rows, ptr(self.dy), ptr(self.z), ptr(self.weight), ptr(self.mean),
                               ptr(self.rstd), ptr(self.dx), ptr(self.dw), ptr(self.db), self.accumulate, ptr(work),
                               self.bytes, s, dz=ptr(self.dz))

    def terms(self):
        torch = _torch()
        z, dy = self.z.double(), self.old[2].double()
        mean = self.mean.double()[:, None] if self.kind == 0 else 0.0
        rstd = self.rstd.double()[:, None]
        w = self.weight.double() if self.weight is not None else torch.ones(self.width, dtype=torch.float64, device="cuda")
        return dy, (z - mean) * rstd, dy * w, rstd

    def formula(self):
        dy, hat, d, rstd = self.terms()
        dx = rstd * (d - (d.mean(1, keepdim=True) if self.kind == 0 else 0.0) - hat * (d * hat).mean(1, keepdim=True))
        return dx + (self.old[3].double() if self.dz is not None else 0.0), (dy * hat).sum(0), dy.sum(0)

    def dx_error(self):
        dy, hat, d, rstd = self.terms()
        want = self.formula()[0]
        along = (d * hat).abs().mean(1, keepdim=True)
        inner = (d.abs() + (d.abs().mean(1, keepdim=True) if self.kind == 0 else 0.0) + hat.abs() * along)
        err = U * rstd * ((P + 4) * (d.abs().mean(1, keepdim=True) * (self.kind == 0) + hat.abs() * along) + 8 * inner)
        return rounded((err + U * want.abs()) * 1.01 + 2.0 ** -148, want, self.x_type)

    def check(self):
        torch = _torch()
        torch.cuda.synchronize()
        assert (self.work[self.bytes:] == 0xff).all()
        dx, dw, db = self.formula()
        dy, hat, d, rstd = self.terms()
        if self.dx is not None:
            close(self.dx, dx, self.dx_error(), "dx")
            if self.dxb is not None:
                assert (outside(self.dxb, self.dx) == 9.0).all()
        parts = max(1, (self.bytes - 256) // (8 * self.width)) if self.width else 1
        S = math.ceil(self.rows / parts) + 16 + math.ceil(parts / 32) + 32
        for got, old, sum_, mag, what in ((self.dw, self.old[0], dw, (dy * hat).abs().sum(0), "dweight"),
                                          (self.db, self.old[1], db, dy.abs().sum(0), "dbias")):
            if got is None:
                continue
            want = sum_ + (old.double() if self.accumulate else 0.0)
            err = ((S + 4) * U * mag + U * want.abs()) * 1.01 + 2.0 ** -148
            close(got, want, rounded(err, want, self.grad_type), what)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("x,y", PAIRS)
def test_backward_widths(kind, x, y):
    for width in WIDTHS:
        say("width", width)
        b = Backward(13, width, kind, x, y, weight=x, grad=0 if width % 2 else x, dz=width % 3 == 0,
                     accumulate=width % 2 == 1, strides=(1, 2, 3), shift=width % 3, seed=width, sums=1 if kind else 3)
        b.run()
        b.check()


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 63, 511, 512, 513, 2049, 9001])
@pytest.mark.parametrize("width", [6, 40, 100, 200, 768, 1024, 2050])
def test_backward_rows(rows, width):
    for kind, (x, y) in ((0, (1, 1)), (1, (0, 2))):
        b = Backward(rows, width, kind, x, y, seed=rows)
        b.run()
        b.check()


@pytest.mark.parametrize("sums", [1, 2, 3])
@pytest.mark.parametrize("dx", [False, True])
def test_backward_on_both_sides_of_the_one_launch_path(sums, dx):
    for rows, width, x, y in ((1, 33, 1, 1), (127, 64, 0, 0), (128, 65, 0, 1), (129, 2000, 2, 2), (513, 300, 1, 1),
                              (1024, 1024, 0, 0), (1025, 1024, 0, 0), (1024, 2047, 1, 1), (2048, 512, 1, 1),
                              (2048, 513, 1, 1), (2049, 40, 0, 2), (300, 5000, 1, 1), (60, 16384, 2, 2), (2048, 1, 1, 1)):
        for acc in (False, True):
            b = Backward(rows, width, sums % 2, x, y, 0, x if acc else 0, dz=dx, dx=dx, sums=sums, accumulate=acc,
                         strides=(1, 4, 2), seed=rows)
            b.run()
            b.check()


def test_backward_of_wide_rows_and_many():
    for rows, width in ((300, 40001), (2000, 16400)):
        b = Backward(rows, width, 0, 0, 0, seed=rows)
        b.run()
        b.check()


@pytest.mark.parametrize("sums", [0, 1, 2, 3])
@pytest.mark.parametrize("dx", [False, True])
@pytest.mark.parametrize("accumulate", [False, True])
def test_backward_outputs_that_are_not_wanted(sums, dx, accumulate):
    for width in (5, 520, 3001, 20003):
        for grad in (0, 1, 2):
            b = Backward(9, width, sums % 2, 0, 1, 1, grad, affine=sums != 1, dz=dx, dx=dx, sums=sums,
                         accumulate=accumulate, strides=(3, 2, 1))
            b.run()
            b.check()


@pytest.mark.parametrize("width", [5, 100, 751, 1500, 2047, 4100, 10003, 16391, 33001])
@pytest.mark.parametrize("where", ["dy", "dz"])
def test_backward_in_place(width, where):
    for kind in (0, 1):
        b = Backward(21, width, kind, 0, 0, seed=7)
        b.dx, b.dxb = getattr(b, where), None
        b.run()
        b.check()


def test_one_row_of_dy_for_all():
    for width in (33, 1024, 20001):
        b = Backward(50, width, 0, 0, 0, dy_row=True)
        b.run()
        b.check()


def test_no_rows():
    torch = _torch()
    for acc in (True, False):
        b = Backward(0, 100, accumulate=acc)
        old = b.dw.clone()
        b.run()
        torch.cuda.synchronize()
        assert torch.equal(b.dw, old) if acc else (b.dw == 0).all() and (b.db == 0).all()
    f = Forward(0, 100)
    f.run()
    Forward(3, 0).run()


@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("width", [9, 1001, 20001, 33001])
def test_gradients_that_are_not_finite_stay_in_row_and_column(bad, width):
    torch = _torch()
    for col in (0, width - 1, width - 2):
        b, clean = (Backward(9, width, 0, 0, 0, seed=4) for _ in range(2))
        b.dy[5, col] = bad
        b.run()
        clean.run()
        torch.cuda.synchronize()
        others = [r for r in range(9) if r != 5]
        assert not torch.isfinite(b.dx[5, col]) and torch.equal(b.dx[others], clean.dx[others])
        hit = torch.zeros(width, dtype=torch.bool, device="cuda")
        hit[col] = True
        for got, want in ((b.dw, clean.dw), (b.db, clean.db)):
            assert torch.equal(~torch.isfinite(got), hit) and torch.equal(got[~hit], want[~hit])


@pytest.mark.parametrize("kind", [0, 1])
def test_the_gradient_against_differences(kind):
    """In 64 bits the formula's gradient equals a difference of the formula
    with a small step; the library's forward pass has the differences that the
    formula has with a large one; and dx is the formula's (above), so it is the
    gradient of the library's own forward pass."""
    torch = _torch()
    rows, width = 4, 200
    b = Backward(rows, width, kind, dz=False, seed=12)
    b.run()
    b.check()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    way = torch.randn(rows, width, device="cuda", generator=gen).double()
    w = b.weight.double()

    def loss64(z):
        m = z.mean(1, keepdim=True) if kind == 0 else 0.0
        return (b.old[2].double() * (z - m) * ((z - m).square().mean(1, keepdim=True) + 1e-5).rsqrt() * w).sum()

    z, h = b.z.double(), 2.0 ** -17
    slope = (loss64(z + h * way) - loss64(z - h * way)) / (2 * h)
    got = (b.dx.double() * way).sum()
    # the truncation is of the order of h^2 = 6e-11 of terms of the size of the loss's magnitude
    size = (b.dx.double().abs() * way.abs()).sum()
    assert (got - slope).abs() <= (b.dx_error() * way.abs()).sum() + 1e-7 * size

    h = 2.0 ** -6
    losses, rounding = [], 0.0
    for sign in (1, -1):
        f = Forward(rows, width, kind, seed=12)
        f.x.copy_(b.z + sign * h * way.float())
        f.x0 = f.x.clone()
        f.weight, f.bias = b.weight, None
        f.run()
        f.check()
        losses.append((b.old[2].double() * f.y.double()).sum())
        # y's error by the forward pass's bound: at most 3 (P + 3) u and 3 D u of rows of unit size
        rounding += float((b.old[2].double().abs() * w.abs() * 8.0 * (P + 3) * U).sum())
        z64 = f.x0.double()
        losses[-1] = (losses[-1], loss64(z64))
    (up, up64), (down, down64) = losses
    assert ((up - down) - (up64 - down64)).abs() <= rounding


def test_replays_with_eager_calls_between():
    torch = _torch()
    for width in (100, 2048, 20001):
        f, b = Forward(40, width, add="rows", seed=2), Backward(700, width, 0, 0, 0, accumulate=True, seed=3)
        ref = Backward(700, width, 0, 0, 0, accumulate=True, seed=3)
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            f.run()
            b.run()
        for k in range(4):
            graph.replay()
            ref.run()
            torch.cuda.synchronize()
            f.check()
            for p, q in ((b.dx, ref.dx), (b.dw, ref.dw), (b.db, ref.db)):
                assert torch.equal(p, q), (width, k)
            f.y.zero_()
            for t in (b, ref):
                t.dy.mul_(1.25)


def test_calls_at_once_with_workspaces_of_their_own():
    torch = _torch()
    cases = [Backward(3000, w, 0, 1, 1, seed=w) for w in (64, 1024, 2047, 16400)]
    refs = [Backward(3000, w, 0, 1, 1, seed=w) for w in (64, 1024, 2047, 16400)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, s in zip(cases, streams):
            c.run(stream=s.cuda_stream)
    torch.cuda.synchronize()
    for r in refs:
        for _ in range(3):
            r.run()
    torch.cuda.synchronize()
    for c, r in zip(cases, refs):
        assert torch.equal(c.dx, r.dx) and torch.equal(c.dw, r.dw) and torch.equal(c.db, r.db)


def test_special_streams():
    torch = _torch()
    f = Forward(9, 333)
    b = Backward(9, 333, accumulate=False)
    for stream in (0, 1, 2):   # null, legacy, per-thread
        f.y.zero_()
        b.dx.zero_()
        torch.cuda.synchronize()
        f.run(stream=stream)
        b.run(stream=stream)
        f.check()
        b.check()


@pytest.mark.parametrize("rows,width,x,y", [(600001, 60, 1, 1), (140001, 250, 0, 0), (70001, 500, 1, 1), (33001, 1001, 0, 2),
                                            (17001, 2047, 0, 1), (4201, 8100, 2, 2), (70001, 765, 1, 1), (50001, 380, 0, 2),
                                            (25001, 1501, 2, 2), (30001, 750, 0, 0), (4001, 10003, 1, 1), (18001, 2501, 1, 1), (16001, 1150, 0, 0)])
def test_large_inputs(rows, width, x, y):
    """Rows that are read past the caches."""
    for kind in (0, 1):
        f = Forward(rows, width, kind, x, y, weight=x, add="rows", seed=1)
        f.run()
        f.check()
        del f
        b = Backward(rows, width, kind, x, y, weight=x, seed=2)
        b.run()
        b.check()
        del b


def test_more_rows_than_a_launch_holds():
    torch, ddp = _torch(), _lib()
    rows, width = (1 << 26) + 77, 8
    x = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros_like(x)
    f = Forward(500, width, 0, 1, 1, seed=8)
    x[:250] = f.x[:250]
    x[-250:] = f.x[250:]
    f.run()
    ddp.ddp_layernorm(ddp.LayerNormDesc(width, x_dtype=1), rows, x.data_ptr(), ptr(f.weight), ptr(f.bias), y.data_ptr(), 0)
    torch.cuda.synchronize()
    assert torch.equal(y[:250], f.y[:250]) and torch.equal(y[-250:], f.y[250:])
    assert (y[1000000:1000100] == f.bias.bfloat16()).all() and (y[-1000:-900] == f.bias.bfloat16()).all()


def test_one_row_of_z_for_all():
    b = Backward(40, 300, 0, 0, 0, dz=False)
    b.z = b.z[:1].expand(40, -1)
    b.desc.c.z_stride = 0
    b.mean, b.rstd = b.mean[:1].expand(40).contiguous(), b.rstd[:1].expand(40).contiguous()
    b.run()
    b.check()


def test_offsets_past_32_bits():
    """Rows more than 2^32 bytes apart from the first."""
    torch, ddp = _torch(), _lib()
    rows, width, stride = 3, 1000, (1 << 31) - 8
    x = torch.zeros(2 * stride + width, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(2 * stride + width, dtype=torch.bfloat16, device="cuda")
    f = Forward(rows, width, 0, 1, 1, seed=8)
    xv, yv = (torch.as_strided(t, (rows, width), (stride, 1)) for t in (x, y))
    xv.copy_(f.x)
    f.run()
    d = ddp.LayerNormDesc(width, x_dtype=1, x_stride=stride, y_stride=stride, z_stride=stride)
    ddp.ddp_layernorm(d, rows, x.data_ptr(), ptr(f.weight), ptr(f.bias), y.data_ptr(), 0)
    torch.cuda.synchronize()
    assert torch.equal(yv, f.y)
