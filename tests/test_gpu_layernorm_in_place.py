"""GPU: the layer norm's backward pass in place over many rows: dx where dy or dz
lies, with workgroups that take several turns, so that the next turn's rows are
read before dx is written over the present one's; each plan of threads and rows,
from the caches and past them. Tolerances are those of the layer norm's tests.
"""
import pytest

from test_gpu_layernorm import Backward, _torch, say

pytestmark = pytest.mark.gpu

# rows, width, type; more than 64 MiB of z are read past the caches
SHAPES = [(5001, 61, 0), (9001, 200, 1), (9001, 1024, 0), (9001, 1501, 1), (9001, 2047, 1), (2101, 6143, 1),
          (2101, 12285, 1), (2049, 8191, 0), (600001, 60, 1), (120001, 301, 1), (50001, 750, 1), (25001, 1501, 1),
          (18001, 2047, 1), (9001, 2047, 0), (18001, 2501, 1), (15001, 1277, 0), (9001, 4095, 1), (5001, 8190, 1),
          (3001, 12285, 1), (2501, 16383, 1)]


@pytest.mark.parametrize("rows,width,t", SHAPES)
@pytest.mark.parametrize("where", ["dy", "dz"])
def test_dx_in_the_place_of_an_argument(rows, width, t, where):
    torch = _torch()
    say("in place", rows, width, t, where)
    b = Backward(rows, width, kind=rows % 2 ^ width % 2, x=t, y=t, weight=t, seed=7)
    b.dx, b.dxb = getattr(b, where), None
    b.run()
    b.check()
    del b
    torch.cuda.empty_cache()
