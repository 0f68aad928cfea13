"""GPU: the AdamW step's clipping is the library's: the factor is the one that
ddp_clip_grads scales gradients by, bit for bit, and no bound is applied unless
one is given."""
import math

import pytest

from test_gpu_adamw import Case

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


@pytest.mark.parametrize("bits", [32, 8])
def test_clipping_on_the_way_equals_scaling_first(bits):
    """fp32 gradients, norms and bounds of all sizes."""
    torch = _torch()
    import bucketed_gradient_all_amd as ddp
    s = torch.cuda.current_stream().cuda_stream
    a, b = (Case([1025, 300], bits=bits, seed=2) for _ in range(2))
    grads = ddp.make_grads(b.sizes, [[t.data_ptr() for t in b.g]])
    gen = torch.Generator().manual_seed(1)
    for k in range(64):
        norm = torch.exp(torch.randn(1, generator=gen) * 4.0)
        bound = float(norm * (0.1 + 1.2 * torch.rand(1, generator=gen)))
        norm = norm.cuda()
        for c in (a, b):
            c.restore()
        a.step(1e-3, 10, norm=norm.data_ptr(), max_norm=bound)
        ddp.ddp_clip_grads(grads, bound, norm.data_ptr(), s)
        b.step(1e-3, 10)
        torch.cuda.synchronize()
        for x, y in zip(a.p + a.m + a.v + (a.ms + a.vs if bits == 8 else []),
                        b.p + b.m + b.v + (b.ms + b.vs if bits == 8 else [])):
            assert torch.equal(x, y), (k, float(norm), bound)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_bound_of_the_norm_itself_leaves_gradients_as_they_are(bits):
    """A bound of fl(norm + 1e-6) is a factor of exactly 1."""
    torch = _torch()
    a, b = (Case([1025], bits=bits, seed=3) for _ in range(2))
    b.step(1e-3, 10)
    gen = torch.Generator().manual_seed(2)
    for k in range(32):
        norm = torch.exp(torch.randn(1, generator=gen) * 3.0).cuda()
        a.restore()
        a.step(1e-3, 10, norm=norm.data_ptr(), max_norm=float(norm + 1e-6))
        torch.cuda.synchronize()
        assert torch.equal(a.p[0], b.p[0]) and torch.equal(a.m[0], b.m[0]) and torch.equal(a.v[0], b.v[0]), float(norm)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_norm_without_a_bound_only_decides_whether_to_step(bits):
    torch = _torch()
    a, b = (Case([1025], bits=bits, seed=4) for _ in range(2))
    b.step(1e-3, 10)
    norm = torch.tensor([1e3], device="cuda")
    a.step(1e-3, 10, norm=norm.data_ptr(), skip_nonfinite=True)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a.contents(), b.contents()))
    a.restore()
    norm.fill_(math.nan)
    a.step(1e-3, 10, norm=norm.data_ptr(), skip_nonfinite=True)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a.before, a.contents()))
