"""Cross attention on layouts where heads lie farther apart than rows ([heads, keys, d] seen as [keys, heads, d])."""
import numpy as np
import pytest
import torch

import tiled_attention_fwd_gb300 as fa
from cross_util import Ragged, check_backward, check_forward

pytestmark = pytest.mark.gpu


def heads_first(t):
    """The same values, laid out [heads, rows, d]."""
    return t.transpose(0, 1).contiguous().transpose(0, 1)


@pytest.mark.parametrize("rows,keys", [([1, 5, 0, 2], [333, 60, 9, 1000]), ([17, 120, 40], [100, 33, 260]), ([300, 700, 3], [500, 129, 0])])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("heads,group", [(3, 1), (2, 4), (1, 3)])
def test_heads_before_rows(rows, keys, heads, group, d):
    """Every tensor of both passes, results too, with its heads farther apart than its rows."""
    s = Ragged(rows, keys, heads, group, d, padded=d != 128, lead=2, pad=3, seed=d + group)
    q, dout, k, v = (heads_first(t) for t in s.tensors())
    assert k.stride(0) == d and k.stride(1) == s.K * d or heads == 1
    o, lse = torch.full_like(q, 7.0), torch.full((heads * group, s.T), 7.0, device="cuda")
    assert o.stride() == q.stride()
    fa.cross_forward(q, k, v, *s.batch(), max_rows=max(rows), out=o, lse=lse)
    fa.check_status()
    check_forward(s, o, lse)
    grads = [torch.full_like(t, 7.0) for t in (q, k, v)]
    fa.cross_backward(q, k, v, o, lse, dout, *s.batch(), out=grads)
    fa.check_status()
    check_backward(s, o, lse, grads)


@pytest.mark.parametrize("rows", [[1, 0, 2], [20, 3, 40], [300, 0, 1]])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
def test_no_keys_at_all_with_heads_far_apart(rows, d):
    """k and v of no places, cut from tensors whose heads lie megabytes apart: nothing of them is read, by any of the kernels."""
    heads, group, S = 8, 2, 1 << 16
    k, v = (torch.ones(heads, S, d, dtype=torch.bfloat16, device="cuda").transpose(0, 1)[:0] for _ in range(2))
    assert k.shape == (0, heads, d) and k.stride(1) == S * d
    assert (heads - 1) * k.stride(1) * 2 > fa.cross_workspace(k).numel()  # beyond what stands in for them
    at = torch.tensor([0] + rows).cumsum(0).to(device="cuda", dtype=torch.int32)
    T = sum(rows)
    q = torch.randn(T, heads * group, d, device="cuda").bfloat16()
    o, lse = torch.full_like(q, 7.0), torch.full((heads * group, T), 7.0, device="cuda")
    none = torch.zeros(len(rows) + 1, dtype=torch.int32, device="cuda")
    fa.cross_forward(q, k, v, at, none, max_rows=max(rows), out=o, lse=lse)
    assert not o.any() and torch.isneginf(lse).all()
    dq, dk, dv = fa.cross_backward(q, k, v, o, lse, q, at, none, out=(torch.full_like(q, 7.0), k, v))
    assert not dq.any()
    fa.check_status()


def test_bounds_of_rows_that_pass_32_bits():
    """They are no bounds, whatever their low bits say."""
    q, k = (torch.randn(n, 2, 64, device="cuda").bfloat16() for n in (40, 50))
    i32 = dict(dtype=torch.int32, device="cuda")
    cu, ck = torch.tensor([0, 7, 40], **i32), torch.tensor([0, 30, 50], **i32)
    o, lse = fa.cross_forward(q, k, k, cu, ck, max_rows=2 ** 31 - 1)
    for most in (2 ** 32, 2 ** 32 + 1, 2 ** 40, 2 ** 63 - 1, 2 ** 70, torch.tensor(2 ** 40), np.int64(2 ** 40)):
        again = fa.cross_forward(q, k, k, cu, ck, max_rows=most)
        fa.check_status()
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    for most in (-1, -2 ** 32 + 33):
        with pytest.raises(fa.FAError):
            fa.cross_forward(q, k, k, cu, ck, max_rows=most)
    cache = fa.PagedCache.empty(4, 2, 16, 64)
    cache.k.copy_(torch.randn(cache.k.shape, device="cuda")), cache.v.copy_(torch.randn(cache.v.shape, device="cuda"))
    table, lens = torch.tensor([[0, 1], [2, 3]], **i32), torch.tensor([20, 32], **i32)
    cu = torch.tensor([0, 10, 40], **i32)
    want = fa.paged_forward(q, cache, table, cu, lens, max_rows=2 ** 31 - 1)
    got = fa.paged_forward(q, cache, table, cu, lens, max_rows=2 ** 32 + 1)
    fa.check_status()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
