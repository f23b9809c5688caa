"""Units of one or two key tiles, many of them to a CTA: the row statistics of one unit are handed over while the next unit is
under way (the protocol is modelled in test_unit_statistics_protocol.py)."""
import numpy as np
import pytest
import torch

import oracle
from parity_util import TOL_BF16_L, TOL_BF16_O, compare
from test_gpu_fp8 import _check_small
from tiled_attention_fwd_gb300 import check_status, forward
from tiled_attention_fwd_gb300.inputs import Workload, as_f64_numpy

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("Nq,Nk", [(128, 128), (256, 128), (384, 100), (100, 77), (640, 256), (64, 40)])
def test_short_units_match_oracle(d, Nq, Nk, causal):
    g = torch.Generator().manual_seed(d + Nq)
    q, k, v = (torch.randn(2, 400, n, d, generator=g).bfloat16() for n in (Nq, Nk, Nk))
    q, k, v = (t[:, :400 if Nq < 300 and d < 256 else 160] for t in (q, k, v))
    dev = [t.contiguous().cuda() for t in (q, k, v)]
    runs = [forward(*dev, causal=causal) for _ in range(4)]
    check_status()
    o, lse = runs[0]
    for other in runs[1:]:
        assert torch.equal(other[0], o) and torch.equal(other[1], lse)
    heads = np.r_[0:2, -2:0]  # the other heads: by PyTorch in 32 bits on the GPU
    o_ref, l_ref = oracle.attention(*(as_f64_numpy(t[:, heads]) for t in (q, k, v)), d ** -0.5, causal)
    r = compare(as_f64_numpy(o.cpu()[:, heads]), lse.cpu().double().numpy()[:, heads], o_ref, l_ref, "bf16")
    assert r["ok"], r
    for b in range(2):
        x = dev[0][b].float() @ dev[1][b].float().transpose(1, 2) * d ** -0.5
        if causal:
            x.masked_fill_(torch.ones(Nq, Nk, dtype=torch.bool, device="cuda").triu(1), float("-inf"))
        o_ref, l_ref = torch.softmax(x, -1) @ dev[2][b].float(), torch.logsumexp(x, -1)
        floor = (o_ref.bfloat16().float() - o_ref).abs()
        assert ((o[b].float() - o_ref).abs() <= TOL_BF16_O + floor).all() and ((lse[b] - l_ref).abs() <= TOL_BF16_L).all()


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [128, 384])
def test_short_units_of_e4m3_match_oracle(d, N, causal):
    r = _check_small(Workload("fp8_short", 1, 320 if N < 200 else 200, N, d, "fp8", causal, seed=N + d))
    assert r["ok"], r
