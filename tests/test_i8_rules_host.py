"""CPU tests of the rules that choose an int8 product's kernel: few rows by very many columns, many experts, the
largest weight."""
import pytest

from i8_cases import KERNELS
from i8_many_experts import MANY, counts_of
from test_i8_host import rules  # noqa: F401  (fixture)


@pytest.mark.parametrize("k", [64, 1024, 4096, 8192])
@pytest.mark.parametrize("n", [8192, 18368, 28672, 49152, 57344, 128256])
def test_few_rows_take_tiles_of_64(rules, n, k):  # noqa: F811
    """Taller tiles hold no more rows than there are: 33 to 64 rows stay with the 64-row tiles that 32 rows take."""
    for m in (17, 32, 33, 48, 64):
        assert KERNELS[rules.dense(m, n, k)] == "I8_TILES_64", m
    assert KERNELS[rules.dense(65, n, k)] != "I8_TILES_64" or n < 18368


@pytest.mark.parametrize("case", MANY, ids=lambda c: f"{c.kernel}-{'up' if c.gate_up else 'down'}-{c.experts}")
def test_many_experts_take_their_kernels(rules, case):  # noqa: F811
    pairs = case.t * case.topk
    got = rules.experts(case.t if case.gate_up else 0, pairs, case.n, case.k, case.experts)
    assert KERNELS[got] == case.kernel
    counts = counts_of(case)
    assert len(counts) == case.experts and 0 < sum(counts) < pairs and counts.count(0) and counts[-1]


def test_dense_kernels_at_the_largest_weight(rules):  # noqa: F811
    """One weight's codes end at 2^31 - 24 bytes, the tiles' ranges at 2^31 - 1024: between them is the streaming
    kernel."""
    for m in (20, 64):
        assert KERNELS[rules.dense(m, 33554431, 64)] == "I8_STREAM_32"
        assert KERNELS[rules.dense(m, 33554416, 64)] == "I8_TILES_64"
