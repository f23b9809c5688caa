"""Cross attention and the page tables without a GPU: argument checks on the host, and pins of their oracles."""
import math

import numpy as np
import pytest
import torch

import oracle
import oracle.cross as ref
import oracle.tables as tables
import tiled_attention_fwd_gb300 as fa

FAKE = 1 << 20  # aligned, non-null, never dereferenced by these calls
ST = (256, 64)
MAX = 0x7ffff000


def batch(**kw):
    b = fa.CCrossBatch(FAKE, FAKE, FAKE, 2, 10, 20)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def fwd(b=None, q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, qs=ST, ks=ST, vs=ST, os=ST, q_heads=8, heads=4, d=64, most=1,
        scale=0.1, ws=FAKE, n=1 << 40):
    return fa.fa_cross_fwd(q, qs, k, ks, v, vs, b or batch(), o, os, lse, q_heads, heads, d, most, scale, ws, n, None)


def bwd(b=None, q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, dout=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, st=(ST,) * 8, q_heads=8,
        heads=4, d=64, scale=0.1, ws=FAKE, n=1 << 40):
    return fa.fa_cross_bwd(q, k, v, o, lse, dout, dq, dk, dv, st, b or batch(), q_heads, heads, d, scale, ws, n, None)


@pytest.mark.parametrize("kw,code", [(dict(cu_rows=0), -1), (dict(cu_keys=0), -1), (dict(B=0), -2), (dict(rows=-1), -2),
                                     (dict(keys=-1), -2), (dict(rows=MAX + 1), -2), (dict(keys=MAX + 1), -2),
                                     (dict(cu_rows=FAKE + 2), -4), (dict(cu_keys=FAKE + 1), -4), (dict(key_lens=FAKE + 2), -4)])
def test_bad_batches_are_refused_on_the_host(kw, code):
    assert fwd(batch(**kw)) == code and bwd(batch(**kw)) == code


@pytest.mark.parametrize("kw,code", [(dict(q_heads=6), -2), (dict(q_heads=0), -2), (dict(heads=0), -2), (dict(heads=65536, q_heads=65536), -2),
                                     (dict(q_heads=4 * 33), -2), (dict(d=48), -3), (dict(d=512), -3), (dict(scale=0.0), -8),
                                     (dict(scale=-1.0), -8), (dict(scale=float("nan")), -8), (dict(q=0), -1), (dict(k=0), -1),
                                     (dict(v=0), -1), (dict(o=0), -1), (dict(lse=0), -1), (dict(ws=0), -1), (dict(q=FAKE + 8), -4),
                                     (dict(k=FAKE + 2), -4), (dict(v=FAKE + 4), -4), (dict(o=FAKE + 8), -4), (dict(lse=FAKE + 2), -4),
                                     (dict(ws=FAKE + 16), -4), (dict(n=0), -9)])
def test_bad_arguments_are_refused_on_the_host(kw, code):
    assert fwd(**kw) == code and bwd(**kw) == code


def test_bad_strides_and_gradients_are_refused_on_the_host():
    for bad, code in (((0, 64), -2), ((256, -64), -2), ((1 << 38, 64), -2), ((252, 64), -4), ((256, 60), -4)):
        for name in ("qs", "ks", "vs", "os"):
            assert fwd(**{name: bad}) == code
        for i in range(8):
            assert bwd(st=(ST,) * i + (bad,) + (ST,) * (7 - i)) == code
    for name in ("dout", "dq", "dk", "dv"):
        assert bwd(**{name: 0}) == -1 and bwd(**{name: FAKE + 8}) == -4
    assert fwd(most=-1) == -2
    with pytest.raises(ValueError):
        bwd(st=(ST,) * 7)


def test_workspace_sizes():
    for d in (32, 64, 128, 256):
        need = fa.fa_cross_fwd_workspace_bytes(d)
        assert need > 0 and fwd(d=d, n=need - 1) == -9
        need = fa.fa_cross_bwd_workspace_bytes(2, 10, 8, 4, d)
        assert need > 0 and bwd(d=d, n=need - 1) == -9
    assert fa.fa_cross_fwd_workspace_bytes(48) == 0
    for bad in ((0, 10, 8, 4, 64), (2, -1, 8, 4, 64), (2, 10, 7, 4, 64), (2, 10, 4 * 33, 4, 64), (2, 10, 8, 4, 48), (2, 10, 8, 0, 64),
                (2, MAX + 1, 8, 4, 64)):
        assert fa.fa_cross_bwd_workspace_bytes(*bad) == 0
    # Offsets into the workspace stay in 64 bits.
    assert fa.fa_cross_bwd_workspace_bytes(1, MAX - 1, 64, 64, 128) >= (MAX - 1) * 64 * 8


def pool(**kw):
    p = fa.CPagePool(FAKE, FAKE, 8, 16)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw,code", [(dict(free_pages=0), -1), (dict(free_count=0), -1), (dict(num_pages=0), -2), (dict(page_size=24), -2),
                                     (dict(page_size=8), -2), (dict(page_size=2048), -2), (dict(free_pages=FAKE + 2), -4),
                                     (dict(free_count=FAKE + 1), -4)])
def test_bad_pools_are_refused_on_the_host(kw, code):
    assert fa.fa_paged_extend(pool(**kw), FAKE, 4, 4, FAKE, FAKE, FAKE, FAKE, FAKE, 2, 4, None) == code
    assert fa.fa_paged_release(pool(**kw), FAKE, 4, 4, FAKE, FAKE, 2, None) == code


def test_bad_tables_are_refused_on_the_host():
    def extend(table=FAKE, stride=4, width=4, lens=FAKE, new=FAKE, cu=FAKE, slots=FAKE, pos=FAKE, B=2, rows=4):
        return fa.fa_paged_extend(pool(), table, stride, width, lens, new, cu, slots, pos, B, rows, None)

    def release(table=FAKE, stride=4, width=4, lens=FAKE, done=FAKE, B=2):
        return fa.fa_paged_release(pool(), table, stride, width, lens, done, B, None)

    for call in (extend, release):
        assert call(table=0) == -1 and call(lens=0) == -1 and call(B=0) == -2 and call(width=0) == -2 and call(stride=3) == -2
        assert call(width=1 << 28, stride=1 << 28) == -2 and call(table=FAKE + 2) == -4 and call(lens=FAKE + 2) == -4
    assert extend(new=0) == -1 and extend(cu=0) == -1 and extend(rows=-1) == -2 and extend(rows=MAX + 1) == -2
    assert extend(new=FAKE + 2) == -4 and extend(cu=FAKE + 2) == -4 and extend(slots=FAKE + 8) == -4 and extend(pos=FAKE + 4) == -4
    assert release(done=0) == -1
    assert "pages" in fa.fa_strerror(-12)


def test_python_refuses_cpu_tensors():
    q, cu = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.tensor([0, 3], dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.cross_forward(q, q, q, cu, cu)
    with pytest.raises(ValueError):
        fa.PagePool(cu, cu[:1], 16)


# ------------------------------------------------------------------ the oracles' pins
def test_one_sequence_of_one_head_is_the_contiguous_oracle():
    rng = np.random.default_rng(0)
    q, k, v, do = (rng.standard_normal((1, 1, 30, 32)) for _ in range(4))
    flat = [t[0, 0][:, None] for t in (q, k, v, do)]
    cu = [0, 30]
    o, lse = ref.attention(*flat[:3], cu, cu, None, 0.2)
    o_ref, l_ref = oracle.attention(q, k, v, 0.2, False)
    assert np.abs(o[:, 0] - o_ref[0, 0]).max() < 1e-13 and np.abs(lse[0] - l_ref[0, 0]).max() < 1e-13
    grads = ref.attention_backward(*flat[:3], o, lse, flat[3], cu, cu, None, 0.2)
    for x, y in zip(grads, oracle.attention_backward(q, k, v, do, 0.2, False)):
        assert np.abs(x[:, 0] - y[0, 0]).max() < 1e-12


@pytest.mark.parametrize("padded", [False, True])
def test_gradients_are_autograds_and_those_of_differences(padded):
    rng = np.random.default_rng(1)
    rows, keys = [3, 0, 5, 2], [4, 6, 0, 7]
    places = [9] * 4 if padded else keys
    cu_rows, cu_keys = np.cumsum([1] + rows), np.cumsum([2] + places)
    q, dout = (rng.standard_normal((cu_rows[-1] + 1, 4, 8)) for _ in range(2))
    k, v = (rng.standard_normal((cu_keys[-1] + 1, 2, 8)) for _ in range(2))
    lens = keys if padded else None
    o, lse = ref.attention(q, k, v, cu_rows, cu_keys, lens, 0.4)
    grads = ref.attention_backward(q, k, v, o, lse, dout, cu_rows, cu_keys, lens, 0.4)
    assert np.isnan(grads[0][0]).all() and np.isnan(grads[1][0]).all() and np.isnan(o[0]).all()
    t = [torch.tensor(x, requires_grad=True) for x in (q, k, v)]
    loss = 0.0
    for row0, n, key0, _, length in ref.sequences(cu_rows, cu_keys, lens):
        for h in range(4):
            if n and length:
                x = t[0][row0:row0 + n, h] @ t[1][key0:key0 + length, h // 2].T * 0.4
                y = torch.softmax(x, -1) @ t[2][key0:key0 + length, h // 2]
                assert np.abs(y.detach().numpy() - o[row0:row0 + n, h]).max() < 1e-13
                loss = loss + (y * torch.tensor(dout[row0:row0 + n, h])).sum()
    loss.backward()
    for x, y in zip(grads, t):
        mine = ~np.isnan(x)
        assert np.abs(x[mine] - y.grad.numpy()[mine]).max() < 1e-12
    for which, at in ((0, (2, 1, 3)), (1, (4, 0, 5)), (2, (3, 1, 0))):
        value = []
        for h in (1e-5, -1e-5):
            x = [q.copy(), k.copy(), v.copy()]
            x[which][at] += h
            value.append(np.nansum(ref.attention(*x, cu_rows, cu_keys, lens, 0.4)[0] * dout))
        assert abs((value[0] - value[1]) / 2e-5 - grads[which][at]) < 1e-8


def test_pages_taken_and_given_back_are_a_permutation():
    rng = np.random.default_rng(2)
    ps, width, total = 16, 5, 20
    table = [[-1] * width for _ in range(4)]
    lens, stack, count = [0] * 4, list(range(total)), total
    for _ in range(50):
        new = rng.integers(0, 30, 4).tolist()
        before = list(lens)
        count, cu, slots, pos, why = tables.extend(table, lens, stack, count, new, ps, 100)
        held = [x for row in table for x in row if x >= 0]
        assert sorted(held + stack[:count]) == list(range(total))
        for b in range(4):
            n = cu[b + 1] - cu[b]
            assert n == (new[b] if why[b] is None else 0) and lens[b] == before[b] + n
            for i in range(n):
                p = before[b] + i
                assert pos[cu[b] + i] == p and slots[cu[b] + i] == table[b][p // ps] * ps + p % ps
            assert sum(x >= 0 for x in table[b]) == math.ceil(lens[b] / ps)
        if rng.random() < 0.6:
            count, fine = tables.release(table, lens, stack, count, (rng.random(4) < 0.5).tolist(), ps)
            assert fine


def test_cross_kernels_fit_their_registers():
    """The chunk kernels' register split (d <= 128) is sized for exactly 128 a thread at launch; the gradients' kernels hold a
    tile's S and dP in registers (the one-pass kernel with 16 warps at the limit of 128)."""
    from tiled_attention_fwd_gb300 import build

    rep = build.ptxas_report({f"fa_cross_{k}_d{d}.cu" for k in ("few", "chunk", "bwd") for d in (32, 64, 128, 256)})
    pick = lambda name: {k: r for k, r in rep.items() if name in k}
    chunk, few, short = pick("fa_paged_chunk_kernel"), pick("fa_paged_few_kernel"), pick("fa_cross_bwd_short_kernel")
    long, prep, join = pick("19fa_cross_bwd_kernel"), pick("fa_cross_prep_kernel"), pick("fa_cross_bwd_join_kernel")
    # Chunks: heads one by one, d <= 64 in pairs, too.  Gradients: dK and dV, dQ; d = 256: dV, dK, dQ.
    assert (len(chunk), len(few), len(short), len(long), len(prep), len(join)) == (6, 11, 3, 9, 4, 4)
    for name, r in chunk.items():
        if "ILi256E" in name:
            assert r["registers"] <= 168, (name, r)
        else:
            assert r["registers"] == 128, (name, r)
    for name, r in short.items():
        assert r["registers"] <= 128 and r["spill_stores"] <= 16, (name, r)
    for name, r in {**few, **long, **prep, **join}.items():
        assert r["spill_stores"] == 0, (name, r)


def test_what_stands_in_for_missing_keys_lies_in_the_workspace():
    """Without keys the forward's tensor maps are of the workspace, with dense heads: 65535 of them at most."""
    for d in (32, 64, 128, 256):
        assert fa.fa_cross_fwd_workspace_bytes(d) >= 65535 * d * 2


def test_more_sequences_than_the_kernels_count():
    """They step through the sequences 1024 at a time in 32 bits: beyond 2^31 - 4096 a step would pass the last and wrap."""
    for B in (MAX + 1, 2 ** 31 - 1):
        assert fwd(batch(B=B, rows=0)) == -2 and bwd(batch(B=B, rows=0)) == -2
        assert fa.fa_paged_extend(pool(), FAKE, 4, 4, FAKE, FAKE, FAKE, FAKE, FAKE, B, 4, None) == -2
        assert fa.fa_paged_release(pool(), FAKE, 4, 4, FAKE, FAKE, B, None) == -2
        cache = fa.CPagedCache(FAKE, FAKE, 0, 0, (1024, 512, 64), (1024, 512, 64), 8, 16, 2, 64)
        pages = fa.CPagedBatch(FAKE, FAKE, FAKE, 4, 4, B, 10)
        assert fa.fa_paged_write(cache, pages, FAKE, ST, FAKE, ST, None) == -2
        assert fa.fa_paged_fwd(FAKE, ST, cache, pages, FAKE, ST, FAKE, 4, 1, 0.1, 0, FAKE, 1 << 40, None) == -2


def test_sizes_that_pass_32_bits_stay_too_large():
    """A C int would keep their low bits."""
    from tiled_attention_fwd_gb300 import _lib

    class Tensor:  # as much of one as the batch is made of
        is_cuda, dtype = True, torch.bfloat16

        def __init__(self, *shape, dtype=torch.bfloat16):
            self.shape, self.dtype = shape, dtype

        dim = lambda self: len(self.shape)
        get_device = lambda self: 0
        data_ptr = lambda self: FAKE
        is_contiguous = lambda self: True

    cu = Tensor(3, dtype=torch.int32)
    for n in (2 ** 31, 2 ** 32 + 50):
        b = _lib._cross_batch(Tensor(50, 2, 64), Tensor(n, 2, 64), cu, cu, None)
        assert (b.B, b.rows) == (2, 50) and fwd(b) == -2 and bwd(b) == -2
        b = _lib._cross_batch(Tensor(n, 2, 64), Tensor(50, 2, 64), cu, cu, None)
        assert fwd(b) == -2 and bwd(b) == -2
