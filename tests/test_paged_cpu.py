"""The paged cache without a GPU: argument checks on the host, and pins of its oracle."""
import math

import numpy as np
import pytest
import torch

import oracle
import oracle.paged as ref
import tiled_attention_fwd_gb300 as fa

FAKE = 1 << 20  # aligned, non-null, never dereferenced by these calls


def cache(**kw):
    c = fa.CPagedCache()
    c.k = c.v = FAKE
    c.k_stride[:] = c.v_stride[:] = (4 * 16 * 64, 16 * 64, 64)
    c.num_pages, c.page_size, c.heads, c.d = 8, 16, 4, 64
    for k, v in kw.items():
        if k.endswith("stride"):
            getattr(c, k)[:] = v
        else:
            setattr(c, k, v)
    return c


def batch(**kw):
    b = fa.CPagedBatch()
    b.page_table = b.cu_rows = b.kv_lens = FAKE
    b.table_stride, b.max_pages, b.B, b.rows = 4, 4, 2, 10
    for k, v in kw.items():
        setattr(b, k, v)
    return b


CACHE_CASES = [(dict(k=0), -1), (dict(v=0), -1), (dict(k_scale=FAKE), -1), (dict(num_pages=0), -2),
               (dict(page_size=24), -2), (dict(page_size=8), -2), (dict(page_size=2048), -2), (dict(heads=0), -2),
               (dict(d=48), -3), (dict(d=512), -3), (dict(k=FAKE + 8), -4), (dict(k_stride=(4096, 1024, 60)), -4),
               (dict(v_stride=(4096, 0, 64)), -2), (dict(v_stride=(1 << 38, 1024, 64)), -2),
               (dict(k_scale=FAKE + 4, v_scale=FAKE), -4),
               (dict(k_scale=FAKE, v_scale=FAKE, k_stride=(4096, 1024, 72)), -4)]  # e4m3 rows are 16-byte units too
BATCH_CASES = [(dict(page_table=0), -1), (dict(cu_rows=0), -1), (dict(kv_lens=0), -1), (dict(B=0), -2),
               (dict(rows=-1), -2), (dict(max_pages=0), -2), (dict(table_stride=3), -2),
               (dict(max_pages=1 << 28, table_stride=1 << 28), -2), (dict(kv_lens=FAKE + 2), -4)]


@pytest.mark.parametrize("kw,code", CACHE_CASES)
def test_bad_caches_are_refused_on_the_host(kw, code):
    c, b = cache(**kw), batch()
    st = (256, 64)
    assert fa.fa_paged_write(c, b, FAKE, st, FAKE, st, None) == code
    assert fa.fa_paged_read(c, b, FAKE, st, FAKE, st, None) == code
    assert fa.fa_paged_fwd(FAKE, (512, 64), c, b, FAKE, (512, 64), FAKE, 8, 1, 0.1, 1, FAKE, 1 << 40, None) == code


@pytest.mark.parametrize("kw,code", BATCH_CASES)
def test_bad_batches_are_refused_on_the_host(kw, code):
    c, b = cache(), batch(**kw)
    st = (256, 64)
    assert fa.fa_paged_write(c, b, FAKE, st, FAKE, st, None) == code
    assert fa.fa_paged_read(c, b, FAKE, st, FAKE, st, None) == code
    assert fa.fa_paged_fwd(FAKE, (512, 64), c, b, FAKE, (512, 64), FAKE, 8, 1, 0.1, 1, FAKE, 1 << 40, None) == code


def test_bad_rows_are_refused_on_the_host():
    c, b, st = cache(), batch(), (256, 64)
    for call in (fa.fa_paged_write, fa.fa_paged_read):
        assert call(c, b, 0, st, FAKE, st, None) == -1
        assert call(c, b, FAKE + 8, st, FAKE, st, None) == -4
        assert call(c, b, FAKE, (252, 64), FAKE, st, None) == -4
        assert call(c, b, FAKE, st, FAKE, (0, 64), None) == -2

    def fwd(q=FAKE, qs=(512, 64), o=FAKE, os=(512, 64), lse=FAKE, heads=8, most=1, scale=0.1, ws=FAKE, n=1 << 40):
        return fa.fa_paged_fwd(q, qs, c, b, o, os, lse, heads, most, scale, 1, ws, n, None)

    assert fwd(q=0) == -1 and fwd(o=0) == -1 and fwd(lse=0) == -1 and fwd(ws=0) == -1
    assert fwd(heads=6) == -2 and fwd(heads=0) == -2 and fwd(heads=4 * 129) == -2 and fwd(most=-1) == -2
    assert fwd(scale=0.0) == -8 and fwd(scale=float("inf")) == -8
    assert fwd(q=FAKE + 8) == -4 and fwd(lse=FAKE + 2) == -4 and fwd(ws=FAKE + 16) == -4 and fwd(qs=(516, 64)) == -4
    need = fa.fa_paged_fwd_workspace_bytes(2, 4, 64)
    assert need > 0 and fwd(n=need - 1) == -9
    assert fa.fa_paged_fwd_workspace_bytes(0, 4, 64) == 0 and fa.fa_paged_fwd_workspace_bytes(2, 4, 48) == 0
    assert "page_table" in fa.fa_strerror(-11)


def test_python_refuses_cpu_tensors():
    k = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.PagedCache(k, k)


# ------------------------------------------------------------------ the oracle's pins
def test_e4m3_rounding_matches_torch():
    x = torch.cat([torch.linspace(-448, 448, 20001), torch.linspace(-0.02, 0.02, 4001), 2.0 ** torch.arange(-12, 9)])
    assert np.array_equal(ref.round_e4m3(x.double().numpy()), x.to(torch.float8_e4m3fn).double().numpy())


def test_scales_are_the_smallest_power_of_two_and_read_back_exactly_in_bf16():
    g = torch.Generator().manual_seed(0)
    x = (torch.randn(200, 64, generator=g) * 2.0 ** torch.randint(-130, 120, (200, 1), generator=g)).bfloat16()
    codes, byte = ref.quantise_rows(x.double().numpy())
    for r, c, e in zip(x.double().numpy(), codes, byte.astype(int)):
        a = np.abs(r).max()
        assert a <= 448 * 2.0 ** (e - 127) and (e == 0 or a > 448 * 2.0 ** (e - 128) or a == 0)
        back = c * 2.0 ** (e - 127)
        assert np.array_equal(torch.from_numpy(back).bfloat16().double().numpy(), back)
        # One rounding: half a step of e4m3 (2^-4 relative) above the subnormals' half step.
        assert (np.abs(back - r) <= np.maximum(2.0 ** -4 * np.abs(r), 2.0 ** (e - 127 - 10))).all()


def test_paged_attention_of_one_page_is_the_contiguous_oracle():
    rng = np.random.default_rng(0)
    n, d = 40, 32
    q, k, v = (rng.standard_normal((1, 1, n, d)) for _ in range(3))
    o_ref, l_ref = oracle.attention(q, k, v, 0.2, True)
    o, lse, absum, _ = ref.attention(q[0, 0][:, None], k, v, [[0]], [0, n], [n], 0.2, True)
    assert np.abs(o[:, 0] - o_ref[0, 0]).max() < 1e-13 and np.abs(lse[0] - l_ref[0, 0]).max() < 1e-13
    assert (absum >= np.abs(o) - 1e-15).all()


def test_paged_attention_takes_pages_heads_and_positions_apart():
    """Two sequences in shuffled pages: rows at the end of their sequences, grouped heads."""
    rng = np.random.default_rng(1)
    ps, d, heads, group = 16, 8, 2, 3
    pages = rng.standard_normal((2, 7, heads, ps, d))
    table = [[4, 1, 6], [0, 3, 5]]
    lens, rows = [35, 20], [3, 2]
    q = rng.standard_normal((5, heads * group, d))
    o, lse, _, _ = ref.attention(q, *pages, table, [0, 3, 5], lens, 0.3, True)
    for row, b, pos, page, slot in ref.places(table, [0, 3, 5], lens, ps):
        for h in range(heads * group):
            k, v = (np.stack([pages[j][table[b][p // ps], h // group, p % ps] for p in range(pos + 1)]) for j in range(2))
            e = [math.exp(0.3 * float(x @ q[row, h])) for x in k]
            assert abs(lse[h, row] - math.log(sum(e))) < 1e-12
            assert np.abs(o[row, h] - sum(a * x for a, x in zip(e, v)) / sum(e)).max() < 1e-12


def test_paged_kernels_fit_their_registers():
    """The chunk kernels' register split (d <= 128) is sized for exactly 128 a thread at launch; the few-row and the
    moving kernels keep their state in registers."""
    from tiled_attention_fwd_gb300 import build

    rep = build.ptxas_report({"fa_paged.cu"} | {f"fa_paged_{k}_d{d}.cu" for k in ("few", "chunk") for d in (32, 64, 128, 256)})
    chunk = {k: r for k, r in rep.items() if "fa_paged_chunk_kernel" in k}
    few = {k: r for k, r in rep.items() if "fa_paged_few_kernel" in k}
    move = {k: r for k, r in rep.items() if "fa_paged_move_kernel" in k}
    # 4 head dimensions x bf16 / e4m3 (x 1, 2 or 4 row tiles, 4 at d <= 128; x write / read)
    assert (len(chunk), len(few), len(move)) == (8, 22, 16)
    for name, r in chunk.items():
        if "ILi256E" in name:
            assert r["registers"] <= 168, (name, r)  # 384 threads, not re-split
        else:
            assert r["registers"] == 128, (name, r)
    for name, r in {**few, **move}.items():
        # Four row tiles of e4m3 at d = 128 need a few registers more than there are (outside the products).
        assert r["spill_stores"] <= (64 if "ILi128ELb1ELi4E" in name else 0), (name, r)


@pytest.mark.parametrize("page_size", [16, 1024])
def test_positions_that_would_pass_32_bits_are_refused(page_size):
    n = 0x7ffff000 // page_size + 1
    c, b = cache(page_size=page_size), batch(max_pages=n, table_stride=n)
    assert fa.fa_paged_write(c, b, FAKE, (256, 64), FAKE, (256, 64), None) == -2
    assert fa.fa_paged_fwd(FAKE, (512, 64), c, b, FAKE, (512, 64), FAKE, 8, 1, 0.1, 1, FAKE, 1 << 40, None) == -2
