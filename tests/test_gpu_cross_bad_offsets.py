"""Cross attention where one offset of a batch names what is not there: the sequences on its two sides are unspecified, all others have to
be right, in both passes (bounds: cross_util)."""
import numpy as np
import pytest
import torch

import tiled_attention_fwd_gb300 as fa
from cross_util import Ragged, check_backward, check_forward

pytestmark = pytest.mark.gpu


def passes(s, cu_rows, cu_keys, key_lens, untouched, code=-11):
    """Both passes with these offsets; the results of the sequences `untouched` of s have to be within their bounds."""
    q, dout, k, v = s.tensors()
    mine_q, mine_k = np.zeros(s.T, dtype=bool), np.zeros(s.K, dtype=bool)
    chosen = [x for b, x in enumerate(s.sequences()) if b in untouched]
    for row0, n, key0, places, _ in chosen:
        mine_q[row0:row0 + n], mine_k[key0:key0 + places] = True, True
    s.sequences, s.mine_q, s.mine_k = lambda: chosen, mine_q, mine_k

    def status():
        with pytest.raises(fa.FAError) as e:
            fa.check_status()
        assert e.value.code == code

    o = torch.full_like(q, 7.0)
    lse = torch.full((q.shape[1], s.T), 7.0, device="cuda")
    fa.cross_forward(q, k, v, cu_rows, cu_keys, key_lens, max_rows=max(s.rows), out=o, lse=lse)
    status()
    # (What the others hold is not looked at.)
    others_q, others_k = torch.from_numpy(~mine_q).cuda(), torch.from_numpy(~mine_k).cuda()
    o[others_q], lse[:, others_q] = 7.0, 7.0
    check_forward(s, o, lse)
    ws = fa.cross_backward_workspace(q, k, len(cu_rows) - 1).fill_(0x7f)  # (large numbers, if they were read)
    grads = [torch.full_like(t, 7.0) for t in (q, k, v)]
    fa.cross_backward(q, k, v, o, lse, dout, cu_rows, cu_keys, key_lens, out=grads, workspace=ws)
    status()
    for t, others in zip(grads, (others_q, others_k, others_k)):
        t[others] = 7.0
    check_backward(s, o, lse, grads)


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("B,n", [(4, 1), (4, 40), (5, 300), (40, 9), (1100, 2)])
def test_a_bad_row_offset_leaves_the_others_right(B, n, d):
    rng = np.random.default_rng(B + d)
    for at, value in ((1, 2 ** 31 - 1), (B // 2, -1), (B - 2, -2 ** 31), (B // 2, None)):
        rows = [max(1, n + int(x)) for x in rng.integers(-n // 2, n // 2 + 1, B)]
        s = Ragged(rows, rng.integers(1, 120 if B < 1000 else 9, B).tolist(), 2 if B < 1000 else 1, 2, d, seed=at, pad=3)
        cu_rows, cu_keys, _ = s.batch()
        cu_rows[at] = s.T + 50 if value is None else value
        passes(s, cu_rows, cu_keys, None, [b for b in range(B) if b not in (at - 1, at)])


def test_a_bad_row_offset_among_thousands():
    """More sequences than a block of the preparing kernel sums up in one go (32 times its threads)."""
    B, rng = 9000, np.random.default_rng(1)
    s = Ragged(rng.integers(0, 3, B).tolist(), rng.integers(0, 4, B).tolist(), 1, 1, 32, seed=1, pad=3)
    cu_rows, cu_keys, _ = s.batch()
    cu_rows[5000] = -3
    passes(s, cu_rows, cu_keys, None, set(range(B)) - {4999, 5000})


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("n", [3, 300])
def test_a_bad_key_offset_or_length_leaves_the_others_right(n, d):
    for at, value in ((1, 2 ** 31 - 1), (2, -7)):
        s = Ragged([n, n + 1, 2, n], [60, 33, 100, 90], 2, 2, d, seed=at, pad=3)
        cu_rows, cu_keys, _ = s.batch()
        cu_keys[at] = value
        passes(s, cu_rows, cu_keys, None, [b for b in range(4) if b not in (at - 1, at)])
    for value in (-1, 104, 2 ** 31 - 1):
        s = Ragged([n, n + 1, 2, n], [60, 33, 100, 90], 2, 2, d, padded=True, seed=5)
        cu_rows, cu_keys, lens = s.batch()
        lens[1] = value
        passes(s, cu_rows, cu_keys, lens, [0, 2, 3])


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("n", [2, 70, 300])
def test_ranges_that_follow_one_another_in_no_order(n, d):
    """Offsets that go back: the range that decreases counts as no rows, and those around it, which share no rows, are right."""
    s = Ragged([n, 1, n], [100, 5, 77], 2, 2, d, seed=n)
    s.rows, s.cu_rows, s.T = [n, 0, n], np.array([n, 2 * n, 0, n]), 2 * n
    s.wide_q = torch.randn(2 * n, 8, d, generator=torch.Generator().manual_seed(d)).bfloat16()
    cu_rows, cu_keys, _ = s.batch()
    passes(s, cu_rows, cu_keys, None, [0, 2])
