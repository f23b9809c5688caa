"""O of rows that all but copy one key's v, which comes after others of nearly its weight."""
import pytest
import torch

import tiled_attention_fwd_gb300 as fa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("above", [0.3, 2.55, 5.3, 7.3])
@pytest.mark.parametrize("group", [1, 8, 16])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
def test_the_largest_weight_is_exact(d, group, above):
    """The heaviest key's weight is 1 before it is rounded: only the other weights are off by u = 2^-8 (half a step of bf16) each, and O is
    rounded once: |err| <= u sum_{j != max} P_j |v_j| + u |o| + 2^-16 sum_j P_j |v_j| (fp32).  Key 517 is `above` log2 units above key 3
    (one warp reads both, whatever d is), the others lie 14 below it.  The kernels of up to 16 rows are meant."""
    K, late, early = 600, 517, 3
    q = torch.zeros(1, group, d)
    q[..., 0] = 1.0
    k = torch.zeros(K, 1, d)
    k[:, 0, 0] = -14.0
    k[early, 0, 0], k[late, 0, 0] = 0.0, above
    v = torch.randn(K, 1, d, generator=torch.Generator().manual_seed(d + group))
    q, k, v = (t.bfloat16().cuda() for t in (q, k, v))
    scale = 0.6931471805599453  # logits in log2 units
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    ck = torch.tensor([0, K], dtype=torch.int32, device="cuda")
    o, lse = fa.cross_forward(q, k, v, cu, ck, max_rows=1, scale=scale)
    fa.check_status()
    x = (q[0].double() @ k[:, 0].double().T) * scale
    p = torch.softmax(x, -1)
    want, mass = p @ v[:, 0].double(), p @ v[:, 0].double().abs()
    rest = mass - p[:, late:late + 1] * v[late, 0].double().abs()
    u = 2.0 ** -8
    assert ((o[0].double() - want).abs() <= u * rest + u * want.abs() + 2.0 ** -16 * mass).all()
    assert (lse[:, 0].double() - torch.logsumexp(x, -1)).abs().max() <= 2.0 ** -18
