"""Cross attention around the bounds at which other kernels take over: rows of a unit (all heads of a group) of the one-pass gradients, rows
of the few-row forward, heads in pairs or one by one, and batches that mix both sides."""
import pytest

from cross_util import Ragged, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [1, 3, 8, 32])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_rows_around_the_one_pass_bound(d, group):
    tiles, tokens = {32: 4, 64: 2, 128: 1}[d], 128 // group
    most = tiles * tokens
    for rows in ([most - 1, most, most + 1], [most], [most + 1], [1, tokens, tokens + 1, most + tokens]):
        check(Ragged(rows, [130, 257, 64, 33][:len(rows)], 2, group, d, padded=True, pad=2, seed=most + len(rows)))


@pytest.mark.parametrize("heads,group", [(1, 1), (2, 1), (1, 4), (3, 2), (2, 16), (1, 32)])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
def test_rows_around_the_few_row_bound(d, heads, group):
    for most in (8, 16, 32):
        n = max(most // group, 1)
        check(Ragged([n, 1, n], [300, 70, 1], heads, group, d, seed=most))
        check(Ragged([n + 1, 1, n, 0], [300, 129, 2, 5], heads, group, d, seed=most))
