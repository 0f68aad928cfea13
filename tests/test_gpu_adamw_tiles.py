"""GPU: the AdamW step over tensors around a tile of 1024 elements, at addresses
that cut the first one anywhere. Tolerances are those of the step's tests."""
import pytest

from test_gpu_adamw import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gap", [0, 1, 3, 63, 64])
@pytest.mark.parametrize("param", [0, 1])
def test_sizes_around_a_tile(bits, gap, param):
    c = Case([1023, 1024, 1025, 1151, 1152, 1153, 2047, 2048, 2049, 4097, 896, 897], param=param, bits=bits,
             gap=gap, seed=gap)
    c.step(1e-3, 10)
    c.check(1e-3, 10)
