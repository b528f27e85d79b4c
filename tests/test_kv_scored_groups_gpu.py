"""Scored attention at each way that the scores' kernel reads logits: in fours, of several tokens together
(groups of 4 to 16 heads), or one by one; over windows that begin anywhere, and past the last token."""
import pytest

from test_kv_scored_gpu import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [4, 6, 8, 12, 16, 20, 24])
@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("bf16", 256), ("e4m3", 128)])
@pytest.mark.parametrize("in_place", [False, True])
def test_groups(group, dtype, dim, in_place):
    run([1500, 0, 1, 513], 2 * group, 2, dim, 16, dtype=dtype, in_place=in_place, extra=5)
    run([1500, 0, 1, 513], 2 * group, 2, dim, 16, 700, dtype=dtype, in_place=in_place, seed=1)


@pytest.mark.parametrize("group", [12, 16])
def test_longer_rows_than_blocks_at_once(group):
    # One row: a thread comes to its tokens more than once.
    run([50000], group, 1, 64, 64, in_place=True)
    run([30011, 29], group, 1, 128, 16, dtype="e4m3", extra=100)
