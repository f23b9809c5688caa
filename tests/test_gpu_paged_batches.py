"""The paged cache on the GPU: batches of hundreds of sequences, page tables that name what is not there in writes and reads,
and both tensors of pages beyond 2^32 elements."""
import numpy as np
import pytest
import torch

import oracle.paged as ref
import tiled_attention_fwd_gb300 as fa
from paged_util import Setup, check, run
from test_gpu_paged import same, written

pytestmark = pytest.mark.gpu


def stored(s, pages, scales):
    """The rows that a read gives back, [K, V] as fp64 [rows, heads, d]; NaN where a row is no token."""
    out = np.full((2, s.T, s.heads, s.d), np.nan)
    for j in range(2):
        x = ref.dequantise(pages[j], scales[j]) if s.fmt == "e4m3" else pages[j]
        for row, _, _, page, slot in ref.places(s.table, s.cu, s.lens, s.page):
            out[j, row] = x[page, :, slot]
    return out


# More sequences than a CTA has threads (256; d = 256: 128; the chunks' kernel 512 and 384): the plan's sums are taken in turns,
# and a row's sequence is found in more than one step.
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,B,most", [(64, 300, 1), (256, 150, 1), (64, 257, 8), (32, 1100, 3), (64, 600, 40), (256, 400, 30)])
def test_more_sequences_than_threads(fmt, d, B, most):
    rng = np.random.default_rng(B)
    lens = [int(n) for n in rng.integers(0, 70, B)]
    rows = [int(min(n, r)) for n, r in zip(lens, rng.integers(0 if most > 1 else 1, most + 1, B))]
    if most > 20:  # chunks far apart among sequences of few rows and of none
        rows = [r if b % 7 == 3 else min(r, 1) for b, r in enumerate(rows)]
    s = Setup(lens, rows, heads=1, group=2, d=d, page=16, fmt=fmt, seed=B, pad=3)
    check(s, *run(s), d ** -0.5, True)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("B", [31, 32, 33, 257, 1100])
def test_write_and_read_of_many_sequences(fmt, B):
    rng = np.random.default_rng(B)
    lens = [int(n) for n in rng.integers(0, 40, B)]
    rows = [int(min(n, r)) for n, r in zip(lens, rng.integers(0, 9, B))]
    s = Setup(lens, rows, heads=2, d=64, page=16, fmt=fmt, seed=B, pad=4)
    cache = s.cache()
    _, k, v = s.tokens()
    fa.paged_write(cache, k, v, *s.batch())
    pages, scales = written(s, s.k_new, s.v_new)
    got = [torch.full((s.T, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    fa.paged_read(cache, *s.batch(), out=tuple(got))
    fa.check_status()
    for x, want in zip((cache.k, cache.v), pages):
        assert same(x.float().cpu().double().numpy(), want)
    want = stored(s, pages, scales)
    for j in range(2):
        x = got[j].cpu().double().numpy()
        assert same(x[:s.cu[-1]], want[j][:s.cu[-1]]) and (x[s.cu[-1]:] == 7.0).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("entry", [-1, "pages", 2 ** 31 - 1])
def test_writes_and_reads_of_pages_that_are_not_there(fmt, entry):
    """The rows on such a page are not written, nor read into; all others are, and the batch is reported."""
    s = Setup([100, 60], [40, 33], heads=2, group=1, d=64, page=16, fmt=fmt, seed=3)
    cache = s.cache()
    _, k, v = s.tokens()
    table, cu, lens = s.batch()
    bad = table.clone()
    bad[0, 5] = s.kv[0].shape[0] if entry == "pages" else entry  # positions 80 to 95 of sequence 0: its rows 20 to 35
    missing = np.zeros(s.T, dtype=bool)
    missing[20:36] = True
    fa.paged_write(cache, k, v, bad, cu, lens)
    with pytest.raises(fa.FAError) as e:
        fa.check_status()
    assert e.value.code == -11
    pages, scales = written(s, s.k_new, s.v_new)
    gone = s.table[0, 5]
    for j in range(2):
        pages[j][gone] = s.kv[j].float().double().numpy()[gone]
        if fmt == "e4m3":
            scales[j][gone] = s.scale_bytes[j].numpy()[gone]
    for x, want in zip((cache.k, cache.v), pages):
        assert same(x.float().cpu().double().numpy(), want)
    if fmt == "e4m3":
        for x, want in zip((cache.k_scale, cache.v_scale), scales):
            assert np.array_equal(x.cpu().numpy(), want)
    got = [torch.full((s.T, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    fa.paged_read(cache, bad, cu, lens, out=tuple(got))
    with pytest.raises(fa.FAError):
        fa.check_status()
    want = stored(s, pages, scales)
    for j in range(2):
        x = got[j].cpu().double().numpy()
        assert (x[missing] == 7.0).all() and same(x[~missing], want[j][~missing])
    fa.check_status()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_keys_and_values_beyond_32_bits(fmt):
    """Written to and read from the far end of pools of more than 2^32 elements, K as well as V."""
    s = Setup([100, 40], [3, 40], heads=1, group=1, d=256, page=64, fmt=fmt, seed=14)
    far = 2 ** 32 // (64 * 256) + 10
    kv = [torch.empty((far + t.shape[0], 1, 64, 256), dtype=t.dtype, device="cuda") for t in s.kv]
    scales = [None if b is None else torch.empty(kv[0].shape[:3], dtype=torch.uint8, device="cuda") for b in s.scale_bytes]
    cache = fa.PagedCache(*kv, *scales)
    table, cu, lens = s.batch()
    table = torch.where(table >= 0, table + far, table)
    _, k, v = s.tokens()
    fa.paged_write(cache, k, v, table, cu, lens)
    got = fa.paged_read(cache, table, cu, lens, rows=s.T)
    fa.check_status()
    want = stored(s, *written(s, s.k_new, s.v_new))
    for j in range(2):
        assert same(got[j].cpu().double().numpy(), want[j])
