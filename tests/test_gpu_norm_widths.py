"""Layer norm at both ends of every width class (the threads that share a row change with it) in all type pairs, for
a single row, for few rows in one launch and for rows enough for partial sums."""
import pytest

from tests.test_gpu_layer_norm import I8, TYPES, check  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu
WIDTHS = [128, 129, 512, 513, 1024, 1025, 1400, 2048, 2049, 4096, 4097, 8192, 8193, 16384, 16385]


@pytest.mark.parametrize("dt,wdt", TYPES)
@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("T", [1, 3, 66])
def test_widths(I8, dt, wdt, T, C):  # noqa: F811
    check(I8, dt, wdt, T, C, seed=T + C, eps=1e-6)
