"""GPU: the layer norm's forward pass on both sides of the rule that has wide rows
read again instead of kept in registers: widths at its ends, more rows than it
asks for, with and without add, in place. Tolerances are those of the layer
norm's tests.
"""
import pytest

from test_gpu_layernorm import Forward, _torch, say

pytestmark = pytest.mark.gpu

# width, x, y
WIDTHS = [(16385, 1, 1), (20001, 2, 2), (28000, 1, 1), (28001, 1, 1), (8193, 0, 0), (10800, 0, 0), (10801, 0, 0),
          (8195, 0, 1), (16385, 0, 2), (18000, 0, 1), (18001, 0, 1), (16385, 0, 0)]


@pytest.mark.parametrize("width,x,y", WIDTHS)
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("rows", [256, 257])
def test_rows_without_add(width, x, y, kind, rows):
    say("again", width, x, y, kind, rows)
    f = Forward(rows, width, kind, x, y, weight=y, strides=(3, 0, 0, 1), shift=1, seed=width)
    f.run()
    f.check()


@pytest.mark.parametrize("width", [16385, 20800, 20801])
@pytest.mark.parametrize("z", [False, True])
def test_rows_with_add_past_the_caches(width, z):
    rows = (64 << 20) // (2 * width) + 2
    say("again", width, z, rows)
    for kind in (0, 1):
        f = Forward(rows, width, kind, 1, 1, add="rows", z=z, seed=kind)
        f.run()
        f.check()
        del f
        _torch().cuda.empty_cache()


@pytest.mark.parametrize("width,t", [(16391, 1), (20003, 2), (8195, 0)])
@pytest.mark.parametrize("kind", [0, 1])
def test_y_in_the_place_of_x(width, t, kind):
    f = Forward(300, width, kind, t, t, seed=2)
    f.y, f.yb = f.x, None
    apart = Forward(300, width, kind, t, t, seed=2)
    for g in (f, apart):
        g.run()
    _torch().cuda.synchronize()
    assert _torch().equal(f.y, apart.y) and _torch().equal(f.rstd, apart.rstd)
    apart.check()
