"""CPU tests of the rule that chooses a dense int8 product's kernel: few rows by very many columns."""
import pytest

from i8_cases import KERNELS
from test_i8_host import rules  # noqa: F401  (fixture)


@pytest.mark.parametrize("k", [64, 1024, 4096, 8192])
@pytest.mark.parametrize("n", [8192, 18368, 28672, 49152, 57344, 128256])
def test_few_rows_take_tiles_of_64(rules, n, k):  # noqa: F811
    """Taller tiles hold no more rows than there are: 33 to 64 rows stay with the 64-row tiles that 32 rows take."""
    for m in (17, 32, 33, 48, 64):
        assert KERNELS[rules.dense(m, n, k)] == "I8_TILES_64", m
    assert KERNELS[rules.dense(65, n, k)] != "I8_TILES_64" or n < 18368
