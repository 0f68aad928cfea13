"""GPU: bench.py's clipping with a bound below the norm, on the tiny workload:
the step's clipping scales, and the figure for gradients below the bound is
taken where nothing is scaled."""
import pytest

from test_gpu_bench import _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bound", [0.1, 10.0, 1000.0])
def test_the_figure_below_the_bound_scales_nothing(bound):
    c = _run(["--workload", "tiny", "--steps", "3", "--warmup", "1", "--overlap-steps", "1", "--backward-ms", "0",
              "--no-cpu-baseline", "--no-plain-layout", "--clip-norm", str(bound)])[0]["clip"]
    assert abs(c["norm"] / (31200 / 12) ** 0.5 - 1) < 0.05   # every step's gradients are fresh ones
    b = c["below_bound"]
    # clipped once: the factor's four roundings, a rounding an element, and the norm's own
    want = min(c["norm"], bound * c["norm"] / (c["norm"] + 1e-6))
    assert abs(b["norm"] - want) <= 8 * 2.0 ** -24 * want
    assert b["max_norm"] >= 1.9 * b["norm"]
    assert c["clip_below_bound_ms"] > 0
