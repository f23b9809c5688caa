"""The paged key/value cache on the GPU: writing, reading back, and attention of new tokens over it."""
import numpy as np
import pytest
import torch

import oracle.paged as ref
import tiled_attention_fwd_gb300 as fa
from paged_util import Setup, check, run

pytestmark = pytest.mark.gpu

D = (32, 64, 128, 256)


# ------------------------------------------------------------------ write and read
def written(s, k, v):
    """The pages after the write, by the oracle: fp64 codes (or bf16 values) and scale bytes."""
    pages = [t.float().double().numpy().copy() for t in s.kv]
    scales = [None if b is None else b.numpy().copy() for b in s.scale_bytes]
    for row, _, _, page, slot in ref.places(s.table, s.cu, s.lens, s.page):
        for j, x in enumerate((k, v)):
            if s.fmt == "e4m3":
                pages[j][page, :, slot], scales[j][page, :, slot] = ref.quantise_rows(x[row].double().numpy())
            else:
                pages[j][page, :, slot] = x[row].double().numpy()
    return pages, scales


def same(a, b):
    return np.array_equal(a, b, equal_nan=True)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,heads,page,fused,token_major", [
    (32, 1, 16, False, False), (64, 3, 32, True, False), (128, 2, 16, True, True), (256, 5, 64, False, True)])
def test_write_then_read(fmt, d, heads, page, fused, token_major):
    # New tokens that start and end inside pages, a sequence without rows, rows at negative positions, rows behind the last.
    s = Setup([37, 0, 1, 130, 3, 16], [20, 0, 1, 130, 6, 0], heads=heads, d=d, page=page, fmt=fmt, seed=d, pad=5,
              fused=fused, token_major=token_major)
    cache = s.cache()
    _, k, v = s.tokens()
    fa.paged_write(cache, k, v, *s.batch())
    fa.check_status()
    pages, scales = written(s, s.k_new, s.v_new)
    for got, want in zip((cache.k, cache.v), pages):
        assert same(got.float().cpu().double().numpy(), want)  # every slot, the others as they were
    if fmt == "e4m3":
        for got, want in zip((cache.k_scale, cache.v_scale), scales):
            assert np.array_equal(got.cpu().numpy(), want)
    ko, vo = (torch.full((s.T, heads, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fa.paged_read(cache, *s.batch(), out=(ko, vo))
    fa.check_status()
    for j, got in enumerate((ko, vo)):
        want = np.full((s.T, heads, d), 7.0)
        x = ref.dequantise(pages[j], scales[j]) if fmt == "e4m3" else pages[j]
        for row, _, _, page_, slot in ref.places(s.table, s.cu, s.lens, s.page):
            want[row] = x[page_, :, slot]
        assert same(got.cpu().double().numpy(), want)


def test_quantisation_of_special_rows():
    """Zeros, the smallest and largest bf16, both sides of 1.75 * 2^k, infinities and NaN, signs, ties."""
    big = float(torch.finfo(torch.bfloat16).max)
    rows = [[0.0] * 32, [2.0 ** -133] + [0.0] * 31, [big, -big] + [1.0] * 30, [448.0] + [0.5] * 31,
            [450.0] + [0.5] * 31, [1.75, -1.0] + [2.0 ** -10] * 30, [1.7578125] + [-0.001] * 31,
            [float("inf")] + [1.0] * 31, [1.0] * 31 + [float("nan")], [-float("inf"), float("inf")] + [0.0] * 30,
            [2.0 ** -120, 2.0 ** -126] + [2.0 ** -130] * 30, [1.9921875 * 2.0 ** 127] + [1.5 * 2.0 ** 125] * 31,
            [17.0, 19.0, 21.0, 23.0, -25.0, 27.0, 29.0, 31.0] * 3 + [256.0] * 8, [-0.0] * 32]
    x = torch.tensor(rows).bfloat16().view(len(rows), 1, 32)
    n = len(rows)
    s = Setup([n], [n], heads=1, group=1, d=32, fmt="e4m3")
    s.k_new, s.v_new = x, -x
    cache = s.cache()
    fa.paged_write(cache, x.cuda(), (-x).cuda(), *s.batch())
    pages, scales = written(s, x, -x)
    for got, want in zip((cache.k, cache.v), pages):
        assert same(got.float().cpu().double().numpy(), want)
    for got, want in zip((cache.k_scale, cache.v_scale), scales):
        assert np.array_equal(got.cpu().numpy(), want)
    k, v = fa.paged_read(cache, *s.batch(), rows=n)
    fa.check_status()
    assert same(k.cpu().double().numpy()[:, 0], ref.dequantise(pages[0], scales[0])[s.table[0, 0], 0, :n])
    assert torch.isnan(k[7:10]).all() and torch.isfinite(k[:7]).all() and torch.isfinite(v[10:]).all()


def test_reading_whole_sequences_allocates_zeros_behind_them():
    s = Setup([19, 40], [1, 1], d=64, fmt="e4m3", seed=3)
    table, _, lens = s.batch()
    cu = torch.tensor([0, 19, 59], dtype=torch.int32, device="cuda")
    k, v = fa.paged_read(s.cache(), table, cu, lens, rows=62)
    for j, got in enumerate((k, v)):
        want = np.concatenate([s.values[j][s.table[b, p // 16], :, p % 16][None] for b, n in enumerate(s.lens) for p in range(n)])
        assert same(got[:59].cpu().double().numpy(), want) and (got[59:] == 0).all()


# ------------------------------------------------------------------ attention
LENS = [1, 16, 17, 127, 128, 129, 300, 64]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", D)
@pytest.mark.parametrize("heads,group", [(2, 1), (1, 3), (2, 8)])
def test_single_tokens(fmt, d, heads, group):
    s = Setup(LENS, [1] * len(LENS), heads=heads, group=group, d=d, fmt=fmt, seed=d + group, pad=2, fused=True)
    check(s, *run(s), d ** -0.5, True)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", D)
@pytest.mark.parametrize("causal", [True, False])
def test_few_rows(fmt, d, causal):
    # Rows of all sequences fit 16; some sequences have no rows, some rows no key.
    s = Setup([5, 40, 0, 129, 2, 33, 0], [4, 1, 0, 3, 4, 2, 2], heads=2, group=4, d=d, page=32, fmt=fmt, seed=7, pad=1)
    check(s, *run(s, causal), d ** -0.5, causal)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", D)
@pytest.mark.parametrize("causal", [True, False])
def test_chunks(fmt, d, causal):
    s = Setup([300, 1, 130, 257, 60, 0, 513], [70, 1, 130, 3, 64, 5, 140], heads=2, group=2, d=d, page=16, fmt=fmt, seed=9,
              pad=3, fused=True, token_major=True)
    check(s, *run(s, causal), d ** -0.5, causal)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("group", [1, 3, 5, 7, 16, 24, 128])
def test_group_sizes(fmt, group):
    s = Setup([200, 90, 33], [60 if group < 10 else 7, 1, 2], heads=1, group=group, d=64, page=64, fmt=fmt, seed=group)
    check(s, *run(s), 0.125, True)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 512, 1024])
def test_page_sizes(fmt, page):
    s = Setup([1100, 129, 1024], [1, 40, 300], heads=1, group=2, d=64, page=page, fmt=fmt, seed=page)
    check(s, *run(s), 0.125, True)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("most", [128, 700])
def test_many_units_on_every_sm(fmt, d, most):
    """Several units to a CTA one after another: of one key tile, and of a few with borders inside units."""
    rng = np.random.default_rng(most + d)
    B, heads = (60, 8) if most == 128 else (16, 8)
    lens = rng.integers(1, most + 1, B)
    rows = [int(min(n, r)) for n, r in zip(lens, rng.integers(1, 40 if most == 128 else 90, B))]
    s = Setup([int(n) for n in lens], rows, heads=heads, group=1, d=d, page=32, fmt=fmt, seed=most, pad=4)
    check(s, *run(s), d ** -0.5, True)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("most", [8, 40])
def test_drafts_of_many_sequences(fmt, d, most):
    """Sequences of 0 to 32 rows (e4m3: those of more than 16 are a launch of their own), alone and beside chunks."""
    rng = np.random.default_rng(d + most)
    B = 160
    lens = [int(n) for n in rng.integers(0, 90, B)]
    rows = [int(min(n, r)) for n, r in zip(lens, rng.integers(0, 9, B))]
    if most > 8:
        rows[::20] = [min(n, most) for n in lens[::20]]
    s = Setup(lens, rows, heads=2, group=4, d=d, page=16, fmt=fmt, seed=most, pad=2)
    check(s, *run(s), d ** -0.5, True)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows", [1, 4, 200])
def test_long_sequences_are_split_and_joined(fmt, rows):
    s = Setup([9001, 4097], [rows, 1], heads=1, group=1, d=128, page=64, fmt=fmt, seed=rows)
    check(s, *run(s), 128 ** -0.5, True)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 4, 150])
def test_large_logits_and_late_maxima(fmt, n):
    """Logits with a spread of tens, the largest last: the running maximum moves again and again."""
    s = Setup([700], [n], heads=1, group=2, d=64, fmt=fmt, seed=5)
    ramp = np.linspace(0.2, 6.0, 700)
    k = s.kv[0].float()
    for p in range(700):
        if fmt == "bf16":
            k[s.table[0, p // 16], :, p % 16] *= float(ramp[p])
        else:
            s.scale_bytes[0][s.table[0, p // 16], :, p % 16] += p // 100
    if fmt == "bf16":
        s.kv[0] = k.bfloat16()
        s.values[0] = s.kv[0].double().numpy()
    else:
        s.values[0] = ref.dequantise(s.kv[0].float().double().numpy(), s.scale_bytes[0].numpy())
    check(s, *run(s), 0.125, True)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [4, 100])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_unseen_new_tokens_do_not_reach_earlier_rows(fmt, n, value):
    """A NaN or an infinity in a new token's K or V reaches that token's own row and later ones, no earlier row."""
    s = Setup([150], [n], heads=2, group=2, d=64, fmt=fmt, seed=11)
    bad = 150 - n + n // 2  # position of the bad token
    page, slot = s.table[0, bad // 16], bad % 16
    for j in range(2):
        for h in (0, 1):
            if (j, h) == (0, 0):
                continue  # head 0: only V
            if fmt == "bf16":
                s.kv[j][page, h, slot, 3] = value
                s.values[j][page, h, slot, 3] = value
            else:
                s.kv[j].view(torch.uint8)[page, h, slot] = 0
                s.scale_bytes[j][page, h, slot] = 255
                s.values[j][page, h, slot] = np.nan
    o, lse = run(s)
    o, lse = o.cpu().double().numpy(), lse.cpu().double().numpy()
    clean = Setup([150], [n], heads=2, group=2, d=64, fmt=fmt, seed=11)
    o_ref, l_ref, absum, _ = ref.attention(clean.q.double().numpy(), *clean.values, clean.table, clean.cu, clean.lens, 0.125, True)
    early = n // 2
    assert np.isfinite(o[:early]).all() and np.isfinite(lse[:, :early]).all()
    assert (np.abs(o[:early] - o_ref[:early]) <= 2.0 ** -7 * (absum[:early] + np.abs(o_ref[:early]))).all()
    if fmt == "bf16":  # head 0: V's column 3 alone is touched, with the value's own kind
        late = o[early:, :2]
        assert np.isnan(late[..., 3]).all() if value != value else (late[..., 3] == value).all()
        assert np.isfinite(late[..., :3]).all() and np.isfinite(late[..., 4:]).all() and np.isfinite(lse[:2]).all()
    else:
        assert np.isnan(o[early:]).all() and np.isfinite(lse[:2]).all()
    if fmt == "e4m3" or value != value:  # head 1: K too
        assert np.isnan(o[early:, 2:]).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_offsets_beyond_32_bits(fmt):
    """Pages at the far end of a pool of more than 2^32 elements."""
    s = Setup([100, 40], [3, 40], heads=1, group=2, d=256, page=64, fmt=fmt, seed=13)
    far = 2 ** 32 // (64 * 256) + 10
    kv = [torch.empty((far + s.kv[0].shape[0], 1, 64, 256), dtype=t.dtype, device="cuda") for t in s.kv]
    scales = [None if b is None else torch.empty(kv[0].shape[:3], dtype=torch.uint8, device="cuda") for b in s.scale_bytes]
    for j in range(2):
        kv[j][far:] = s.kv[j].cuda()
        if fmt == "e4m3":
            scales[j][far:] = s.scale_bytes[j].cuda()
    cache = fa.PagedCache(*kv, *scales)
    table, cu, lens = s.batch()
    table = torch.where(table >= 0, table + far, table)
    q, k, v = s.tokens()
    o, lse = fa.paged_forward(q, cache, table, cu, lens, max_rows=40)
    fa.check_status()
    check(s, o, lse, 0.0625, True)
    fa.paged_write(cache, k, v, table, cu, lens)
    k2, v2 = fa.paged_read(cache, table, cu, lens, rows=s.T)
    fa.check_status()
    pages, scale_bytes = written(s, s.k_new, s.v_new)
    want = ref.dequantise(pages[1], scale_bytes[1]) if fmt == "e4m3" else pages[1]
    for row, _, _, page, slot in ref.places(s.table, s.cu, s.lens, s.page):
        assert same(v2[row].cpu().double().numpy(), want[page, :, slot])


# ------------------------------------------------------------------ a run of them together
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_prompt_chunks_and_steps_together(fmt):
    """Two sequences: their prompts in chunks, then single tokens, each call writing and attending; the rows must be
    those of attention over the whole sequences at once, and (bf16) near those of the contiguous forward."""
    heads, group, d, page = 2, 4, 128, 16
    total = [180, 77]
    g = torch.Generator().manual_seed(1)
    q = [torch.randn(n, heads * group, d, generator=g).bfloat16() for n in total]
    k = [torch.randn(n, heads, d, generator=g).bfloat16() for n in total]
    v = [torch.randn(n, heads, d, generator=g).bfloat16() for n in total]
    dtype = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
    cache = fa.PagedCache.empty(24, heads, page, d, dtype=dtype)
    order = torch.randperm(24, generator=g).int()
    table = torch.stack([order[:12], order[12:]]).cuda()
    got = [torch.zeros(n, heads * group, d) for n in total]
    done = [0, 0]
    for chunk in [(100, 0), (61, 50), (1, 20)] + [(1, 1)] * 6 + [(12, 1)]:
        chunk = [min(c, n - a) for c, n, a in zip(chunk, total, done)]
        at = list(done)
        done = [a + c for a, c in zip(done, chunk)]
        rows = [torch.cat([x[b][at[b]:done[b]] for b in range(2)]).cuda() for x in (q, k, v)]
        cu = torch.tensor([0, chunk[0], sum(chunk)], dtype=torch.int32, device="cuda")
        lens = torch.tensor(done, dtype=torch.int32, device="cuda")
        fa.paged_write(cache, rows[1], rows[2], table, cu, lens)
        o, _ = fa.paged_forward(rows[0], cache, table, cu, lens, max_rows=max(chunk))
        for b in range(2):
            got[b][at[b]:done[b]] = o[int(cu[b]):int(cu[b + 1])].float().cpu()
    fa.check_status()
    assert done == total
    for b, n in enumerate(total):
        kr, vr = k[b].double().numpy(), v[b].double().numpy()
        if fmt == "e4m3":
            kr, vr = (ref.dequantise(*ref.quantise_rows(x)) for x in (kr, vr))
        pages = [x.transpose(1, 0, 2)[None] for x in (kr, vr)]  # one page of n tokens
        o_ref, _, absum, _ = ref.attention(q[b].double().numpy(), *pages, [[0]], [0, n], [n], d ** -0.5, True)
        assert (np.abs(got[b].double().numpy() - o_ref) <= 2.0 ** -7 * (absum + np.abs(o_ref))).all()
        if fmt == "bf16":
            whole = [x.transpose(0, 1)[None].contiguous().cuda() for x in
                     (q[b], k[b].repeat_interleave(group, 1), v[b].repeat_interleave(group, 1))]
            o, _ = fa.forward(*whole, causal=True)
            assert (np.abs(got[b].numpy() - o[0].transpose(0, 1).float().cpu().numpy()) <= 2.0 ** -6 * (absum + np.abs(o_ref))).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_captured_step_replays_with_new_contents(fmt):
    """One graph of write and attention, replayed as the sequences grow: lengths, pages and rows are read on the device."""
    heads, group, d, page = 2, 2, 64, 16
    s = Setup([31, 100, 15], [1, 1, 1], heads=heads, group=group, d=d, page=page, fmt=fmt, seed=2, spare=6)
    cache = s.cache()
    table, cu, lens = s.batch()
    q, k, v = (t.clone() for t in s.tokens())
    o, lse = torch.zeros_like(q), torch.zeros(heads * group, 3, device="cuda")
    ws = fa.paged_workspace(cache, 3)

    def step():
        fa.paged_write(cache, k, v, table, cu, lens)
        fa.paged_forward(q, cache, table, cu, lens, max_rows=1, out=o, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    spare = [p for p in range(s.kv[0].shape[0]) if p not in set(s.table.ravel().tolist())]
    g = torch.Generator().manual_seed(4)
    for turn in range(3):
        lens += 1
        for b in range(3):  # a sequence that outgrows its pages gets one of the spare ones
            at = (int(lens[b]) - 1) // page
            if int(table[b, at]) < 0:
                table[b, at] = spare.pop()
        new = [torch.randn(t.shape, generator=g).bfloat16() for t in (q, k, v)]
        for dst, src in zip((q, k, v), new):
            dst.copy_(src)
        graph.replay()
        fa.check_status()
        values = [t.float().cpu().double().numpy() for t in (cache.k, cache.v)]
        if fmt == "e4m3":
            values = [ref.dequantise(c, b.cpu().numpy()) for c, b in zip(values, (cache.k_scale, cache.v_scale))]
        o_ref, l_ref, absum, _ = ref.attention(new[0].double().numpy(), *values, table.tolist(), [0, 1, 2, 3],
                                               lens.tolist(), d ** -0.5, True)
        assert (np.abs(o.cpu().double().numpy() - o_ref) <= 2.0 ** -7 * (absum + np.abs(o_ref))).all()
        assert np.abs(lse.cpu().double().numpy() - l_ref).max() <= 1e-5


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_captured_mixed_batch_replays_with_new_lengths(fmt):
    """A graph of one call over a chunk, drafts and single tokens (every kernel of the attention), replayed with other
    rows to a sequence: what is a chunk in one replay is a single token in another."""
    heads, group, d, page, T, B = 2, 4, 64, 16, 120, 6
    s = Setup([400, 333, 290, 129, 257, 64], [20] * B, heads=heads, group=group, d=d, page=page, fmt=fmt, seed=12)
    cache = s.cache()
    table, cu, lens = s.batch()
    q = s.tokens()[0]
    o, lse = torch.full_like(q, 7.0), torch.full((heads * group, T), 7.0, device="cuda")
    ws = fa.paged_workspace(cache, B)

    def call():
        fa.paged_forward(q, cache, table, cu, lens, max_rows=110, out=o, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for rows in ([1, 8, 2, 100, 0, 6], [70, 1, 1, 1, 1, 1], [1, 5, 8, 4, 3, 1], [9, 9, 9, 9, 9, 64]):
        s.rows, s.cu = rows, np.concatenate([[0], np.cumsum(rows)])
        cu.copy_(torch.tensor(s.cu, dtype=torch.int32))
        o.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        graph.replay()
        fa.check_status()
        check(s, o, lse, d ** -0.5, True)


def test_two_streams_with_workspaces_of_their_own():
    setups = [Setup([2000, 300], [n, 1], heads=2, group=2, d=128, seed=n) for n in (1, 90)]
    jobs = []
    for s in setups:
        cache = s.cache()
        o = torch.full((s.T, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((4, s.T), 7.0, device="cuda")
        jobs.append((s, cache, s.tokens()[0], s.batch(), o, lse, fa.paged_workspace(cache, 2), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, cache, q, batch, o, lse, ws, stream in jobs:
            with torch.cuda.stream(stream):
                fa.paged_forward(q, cache, *batch, max_rows=max(s.rows), out=o, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    fa.check_status()
    for s, _, _, _, o, lse, _, _ in jobs:
        check(s, o, lse, 128 ** -0.5, True)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 80])
def test_same_inputs_give_the_same_bits(fmt, n):
    s = Setup([5000, 700, 81], [n, 1, n], heads=2, group=4, d=128, page=32, fmt=fmt, seed=21)
    cache = s.cache()
    first = run(s, cache=cache)
    for _ in range(3):
        again = run(s, cache=cache)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


# ------------------------------------------------------------------ what is not there
def test_batches_that_name_what_is_not_there_are_reported():
    """Bad pages, lengths and rows are reported once, touch nothing and leave the other sequences right."""
    for n in (1, 40):
        s = Setup([100, 60], [n, n], heads=1, group=2, d=64, page=16, seed=3)
        cache = s.cache()
        q, k, v = s.tokens()
        good = run(s, cache=cache)
        before = cache.k.clone(), cache.v.clone()
        table, cu, lens = s.batch()
        bad = []
        for value in (-1, s.kv[0].shape[0], 2 ** 31 - 1):  # the page of sequence 0's last tokens
            t = table.clone()
            t[0, 6] = value
            bad.append((t, cu, lens))
        for value in (-5, 16 * table.shape[1] + 1, 2 ** 31 - 1):
            x = lens.clone()
            x[0] = value
            bad.append((table, cu, x))
        bad.append((table, torch.tensor([0, n, n - 1], dtype=torch.int32, device="cuda"), lens))
        bad.append((table, torch.tensor([0, n, 10 * n + 50], dtype=torch.int32, device="cuda"), lens))
        for i, (t, c, x) in enumerate(bad):
            o = torch.full_like(good[0], 7.0)
            lse = torch.full_like(good[1], 7.0)
            fa.paged_forward(q, cache, t, c, x, max_rows=n, out=o, lse=lse)
            with pytest.raises(fa.FAError) as e:
                fa.check_status()
            assert e.value.code == -11
            if i < 6:
                assert torch.equal(o[n:], good[0][n:]) and torch.equal(lse[:, n:], good[1][:, n:])
            else:
                assert torch.equal(o[:n], good[0][:n])
            if i >= 3:
                w = fa.PagedCache(before[0].clone(), before[1].clone())
                fa.paged_write(w, k, v, t, c, x)
                with pytest.raises(fa.FAError):
                    fa.check_status()
                moved = (w.k != before[0]) & ~(torch.isnan(w.k) & torch.isnan(before[0]))
                own = {int(p) for p in s.table[0] if p >= 0} if i < 6 else {int(p) for p in s.table[1] if p >= 0}
                assert not moved[sorted(own)].any()
        fa.check_status()  # reported once


def test_more_rows_than_max_rows_are_left_and_reported():
    for n, most in ((3, 2), (70, 1), (70, 60)):
        s = Setup([100, 60], [n, 1], heads=1, group=2, d=64, seed=3)
        cache = s.cache()
        good = run(s, cache=cache)
        o, lse = torch.full_like(good[0], 7.0), torch.full_like(good[1], 7.0)
        fa.paged_forward(s.tokens()[0], cache, *s.batch(), max_rows=most, out=o, lse=lse)
        with pytest.raises(fa.FAError):
            fa.check_status()
        assert (o[:n] == 7.0).all() and torch.equal(o[n:], good[0][n:])


def test_no_rows_is_no_work():
    s = Setup([5], [0], d=64)
    cache = s.cache()
    q, k, v = s.tokens()
    fa.paged_write(cache, k, v, *s.batch())
    fa.paged_read(cache, *s.batch(), rows=0)
    o, lse = fa.paged_forward(q, cache, *s.batch())
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
    fa.check_status()


def test_python_refusals():
    s = Setup([20], [2], d=64, heads=2, group=2)
    cache = s.cache()
    q, k, v = s.tokens()
    table, cu, lens = s.batch()
    for args in ((q, cache, table.long(), cu, lens), (q, cache, table, cu[:1], lens), (q, cache, table.cpu(), cu, lens),
                 (q.float(), cache, table, cu, lens), (q[..., :32], cache, table, cu, lens), (q[0], cache, table, cu, lens),
                 (q, cache, table[:0], cu[:1], lens[:0])):
        with pytest.raises(ValueError):
            fa.paged_forward(*args)
    with pytest.raises(fa.FAError):  # 3 query heads over 2 heads
        fa.paged_forward(q[:, :3], cache, table, cu, lens)
    with pytest.raises(fa.FAError):  # too small a workspace
        fa.paged_forward(q, cache, table, cu, lens, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        fa.paged_write(cache, k[:, :1], v[:, :1], table, cu, lens)
    with pytest.raises(ValueError):
        fa.paged_write(cache, k, v[:1], table, cu, lens)
    with pytest.raises(ValueError):
        fa.paged_read(cache, table, cu, lens)
    with pytest.raises(ValueError):
        fa.PagedCache(cache.k, cache.v, torch.zeros(cache.k.shape[:3], dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        fa.PagedCache(cache.k.cpu(), cache.v.cpu())
    with pytest.raises(fa.FAError):  # pages of 24 tokens
        fa.paged_write(fa.PagedCache.empty(2, 2, 24, 64), k, v, table, cu, lens)
