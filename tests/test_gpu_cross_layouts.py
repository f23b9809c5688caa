"""Cross attention on layouts where heads lie farther apart than rows ([heads, keys, d] seen as [keys, heads, d])."""
import pytest
import torch

import tiled_attention_fwd_gb300 as fa

pytestmark = pytest.mark.gpu


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
