"""How many work-groups the norms' backward takes for a few rows, as its workspace
says: one for up to two steps of rows that fit one piece a lane, which then needs no
second launch; more rows, and longer ones, are spread."""
import pytest

from combine_top_route_amd import binding as B
from test_norm_refusals import pytestmark, shape  # noqa: F401

BF16, F32 = 1, 0


def groups(T, d, dtype):
    n = B.norm_workspace_size(shape(T, d, dtype))
    assert n % (8 * d) == 0
    return n // (8 * d)  # two float sums a column


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_long_rows_are_spread(dtype):
    for d in (4104, 8192, 12288, 16384):
        assert [groups(T, d, dtype) for T in (1, 2, 3, 4)] == [1, 2, 3, 4], d


@pytest.mark.parametrize("d,dtype", [(2048, BF16), (4096, BF16), (1024, F32), (2048, F32)])
def test_two_rows_take_one(d, dtype):
    assert [groups(T, d, dtype) for T in (1, 2, 3, 4)] == [1, 1, 3, 4]


def test_short_rows():
    # 32 rows of 64 a step
    assert [groups(T, 64, BF16) for T in (1, 32, 64, 65, 128)] == [1, 1, 1, 3, 4]
