"""GPU: bench.py's step with the norm and clipping of its results, on the tiny
workload: the norm it reports is the mean gradient's."""
import pytest

from test_gpu_bench import _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("extra", [[], ["--collective", "reduce_scatter"]])
def test_bench_line_with_clipping(extra):
    lines = _run(["--workload", "tiny", "--steps", "3", "--warmup", "1", "--overlap-steps", "1", "--backward-ms", "0",
                  "--no-cpu-baseline", "--no-plain-layout", "--clip-norm", "1000", *extra])
    assert len(lines) == 1
    c = lines[0]["clip"]
    # 31200 means of four values of U(-1, 1): variance 1/12
    assert abs(c["norm"] / (31200 / 12) ** 0.5 - 1) < 0.05
    assert c["max_norm"] == 1000 and c["step_and_clip_ms"] > 0 and c["clip_below_bound_ms"] > 0
