"""Page tables built on the GPU, against the oracle that takes one token and one page at a time."""
import numpy as np
import pytest
import torch

import oracle.tables as ref
import tiled_attention_fwd_gb300 as fa
from cross_util import Ragged, check_forward

pytestmark = pytest.mark.gpu


class Pool:
    """Tables of sequences with `lens` tokens, on the host and on the device."""

    def __init__(self, lens, width, page, spare, seed=0):
        rng = np.random.default_rng(seed)
        held = [-(-n // page) for n in lens]
        total = sum(held) + spare
        order = rng.permutation(total).tolist()
        self.page, self.lens = page, list(lens)
        self.table = [[-1] * width for _ in lens]
        at = 0
        for b, n in enumerate(held):
            self.table[b][:n] = order[at:at + n]
            at += n
        self.stack, self.count = order[at:] + [-1] * at, spare
        i32 = dict(dtype=torch.int32, device="cuda")
        self.d_table, self.d_lens = torch.tensor(self.table, **i32), torch.tensor(self.lens, **i32)
        self.pool = fa.PagePool(torch.tensor(self.stack, **i32), torch.tensor([self.count], **i32), page)

    def same(self):
        assert self.d_lens.tolist() == self.lens
        assert self.d_table.tolist() == self.table
        assert self.pool.free_count.item() == self.count
        assert self.pool.free_pages.tolist() == self.stack

    def extend(self, new, rows, code=None):
        """One call on both sides; check_status has to say `code`, or what the oracle's reasons come to."""
        self.count, cu, slots, positions, why = ref.extend(self.table, self.lens, self.stack, self.count, new, self.page, rows)
        i32 = dict(dtype=torch.int32, device="cuda")
        out = fa.paged_extend(self.pool, self.d_table, self.d_lens, torch.tensor(new, **i32), rows=rows)
        self.status(code or (-11 if "batch" in why else -12 if "pages" in why else None))
        assert out[0].tolist() == cu
        assert out[1].tolist() == slots + [-1] * (rows - len(slots))
        assert out[2].tolist() == positions + [-1] * (rows - len(slots))
        self.same()
        return out, why

    def release(self, done, code=None, fine=True):
        self.count, ok = ref.release(self.table, self.lens, self.stack, self.count, done, self.page)
        assert ok == fine
        fa.paged_release(self.pool, self.d_table, self.d_lens, torch.tensor(done, dtype=torch.bool, device="cuda"))
        self.status(code)
        self.same()

    def status(self, code):
        if code is None:
            fa.check_status()
        else:
            with pytest.raises(fa.FAError) as e:
                fa.check_status()
            assert e.value.code == code


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 512, 1024])
@pytest.mark.parametrize("pad", [0, 1, 5])
def test_extend_then_release(page, pad):
    rng = np.random.default_rng(page)
    lens = rng.integers(0, 4 * page, 37).tolist()
    new = rng.integers(0, 3 * page, 37).tolist()
    new[3] = new[7] = 0
    p = Pool(lens, 9, page, spare=37 * 4, seed=page)
    p.extend(new, sum(new) + pad)
    p.extend([1] * 37, 37 + pad)
    p.release([b % 3 == 0 for b in range(37)])
    p.extend(new, sum(new) + pad)
    p.release([True] * 37)
    assert p.count == len(p.stack) and sorted(p.stack) == list(range(len(p.stack)))


@pytest.mark.parametrize("B", [1, 2, 31, 33, 255, 257, 1023, 1024, 1025, 3000])
def test_batches_of_any_size(B):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 70, B).tolist()
    p = Pool(lens, 12, 16, spare=B * 6, seed=B)
    for most in (2, 5, 40):
        new = rng.integers(0, most, B).tolist()
        p.extend(new, sum(new) + 3)
        p.release((rng.random(B) < 0.3).tolist())
    p.release([False] * B)
    p.release([True] * B)


@pytest.mark.parametrize("B,most", [(1, 100000), (3, 70000), (40, 5000)])
def test_long_prompts(B, most):
    rng = np.random.default_rng(B)
    new = rng.integers(most // 2, most, B).tolist()
    p = Pool([0] * B, -(-most // 16) + 2, 16, spare=sum(-(-n // 16) for n in new) + 1, seed=B)
    p.extend(new, sum(new))
    p.extend([1] * B, B + 2)
    p.release([b % 2 == 0 for b in range(B)])
    p.release([True] * B)


def test_the_last_token_of_a_page_needs_none_and_the_next_one_does():
    p = Pool([15, 16, 31, 0], 4, 16, spare=2)
    _, why = p.extend([1, 1, 1, 0], 3)
    assert why == [None] * 4 and p.count == 1
    p.extend([0, 0, 0, 0], 0)


# ------------------------------------------------------------------ what does not fit
def test_pages_run_out():
    """Sequences up to the first that the stack cannot serve get theirs; later ones that need none go on."""
    p = Pool([16, 5, 30, 16, 3], 6, 16, spare=3)
    _, why = p.extend([17, 2, 40, 1, 4], 64, code=-12)
    assert why == [None, None, "pages", "pages", None]
    _, why = p.extend([0, 0, 1, 16, 0], 64)
    assert why == [None] * 5


def test_rows_run_out():
    p = Pool([16, 5, 30, 16], 6, 16, spare=30)
    _, why = p.extend([4, 3, 6, 1], 12, code=-11)
    assert why == [None, None, "batch", "batch"]


def test_lengths_and_counts_that_cannot_be():
    for b, old, new in ((0, -1, 2), (1, 5, -3), (2, 90, 10), (1, 2 ** 31 - 1, 2 ** 31 - 1), (0, 5, -2 ** 31)):
        p = Pool([5, 6, 7], 6, 16, spare=9)
        p.lens[b] = old
        p.d_lens[b] = old
        counts = [1, 1, 1]
        counts[b] = new
        _, why = p.extend(counts, 8, code=-11)
        assert [w is None for w in why] == [x != b for x in range(3)]


@pytest.mark.parametrize("value", [-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1])
def test_entries_that_are_no_page(value):
    p = Pool([5, 20, 7], 6, 16, spare=9)
    p.table[1][1] = value
    p.d_table[1, 1] = value
    p.extend([1, 1, 1], 8, code=-11)  # sequence 1's new token lies on it
    p.release([True, True, False], code=-11, fine=False)
    p = Pool([5, 20, 7], 6, 16, spare=9)
    p.stack[8] = value
    p.pool.free_pages[8] = value
    p.extend([16, 1, 1], 20, code=-11)


def test_counts_that_the_stack_cannot_hold():
    for value in (-1, 10 ** 6):
        p = Pool([5], 4, 16, spare=3)
        p.pool.free_count.fill_(value)
        fa.paged_extend(p.pool, p.d_table, p.d_lens, torch.tensor([1], dtype=torch.int32, device="cuda"), rows=1)
        p.status(-11)
    p = Pool([40, 40], 4, 16, spare=1)
    p.pool.free_count.fill_(5)  # three pages too many: room for two of the six
    p.count = 5
    p.release([True, True], code=-11, fine=False)


def test_release_of_a_length_beyond_the_table():
    p = Pool([64, 5], 4, 16, spare=1)
    p.lens[0] = 65
    p.d_lens[0] = 65
    p.release([True, False], code=-11, fine=False)


# ------------------------------------------------------------------ graphs, and the calls that read the tables
def test_captured_extend_and_release_replay():
    p = Pool([3, 40, 0, 77], 12, 16, spare=60)
    i32 = dict(dtype=torch.int32, device="cuda")
    new, done = torch.zeros(4, **i32), torch.zeros(4, dtype=torch.uint8, device="cuda")
    out = torch.zeros(5, **i32), torch.full((64,), -1, dtype=torch.int64, device="cuda"), torch.full((64,), -1, **i32)
    graph = torch.cuda.CUDAGraph()
    fa.paged_extend(p.pool, p.d_table, p.d_lens, new, out=out)
    with torch.cuda.graph(graph):
        fa.paged_release(p.pool, p.d_table, p.d_lens, done)
        fa.paged_extend(p.pool, p.d_table, p.d_lens, new, out=out)
    rng = np.random.default_rng(0)
    for _ in range(6):
        n, d = rng.integers(0, 16, 4).tolist(), (rng.random(4) < 0.4).tolist()
        new.copy_(torch.tensor(n))
        done.copy_(torch.tensor(d))
        p.count, _ = ref.release(p.table, p.lens, p.stack, p.count, d, 16)
        p.count, cu, slots, positions, _ = ref.extend(p.table, p.lens, p.stack, p.count, n, 16, 64)
        graph.replay()
        fa.check_status()
        p.same()
        assert out[0].tolist() == cu and out[1][:cu[-1]].tolist() == slots and out[2][:cu[-1]].tolist() == positions


@pytest.mark.parametrize("fmt", [torch.bfloat16, torch.float8_e4m3fn])
def test_a_decoder_with_an_encoder(fmt):
    """Prompts, then steps of one token: tables extended, K and V written, self attention over the pages and cross attention to the
    encodings, in one captured step; slots agree with where paged_write put the rows, and released pages serve a new request."""
    d, heads, group, page, B = 64, 2, 2, 16, 3
    g = torch.Generator(device="cuda").manual_seed(0)
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = fa.PagedCache.empty(40, heads, page, d, dtype=fmt)
    pool = fa.PagePool.full(40, page)
    table, lens = torch.full((B, 8), -1, **i32), torch.zeros(B, **i32)
    enc = Ragged([1] * B, [50, 0, 130], heads, group, d, seed=1)
    _, _, ek, ev = enc.tensors()
    _, cu_keys, _ = enc.batch()

    def tokens(n):
        return (torch.randn(n, heads * h, d, generator=g, device="cuda").bfloat16() for h in (group, 1, 1))

    def step(q, k, v, new, out, o, most):
        fa.paged_extend(pool, table, lens, new, out=out)
        fa.paged_write(cache, k, v, table, out[0], lens)
        fa.paged_forward(q, cache, table, out[0], lens, max_rows=most, out=o[0], lse=o[1])
        fa.cross_forward(q, ek, ev, out[0], cu_keys, max_rows=most, out=o[2], lse=o[3])

    def buffers(n):
        out = torch.zeros(B + 1, **i32), torch.full((n,), -1, dtype=torch.int64, device="cuda"), torch.full((n,), -1, **i32)
        o = [torch.full((n, heads * group, d), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((heads * group, n), 7.0, device="cuda")]
        return out, o + [t.clone() for t in o]

    held = []  # every sequence's k and v, as they were given
    new = torch.tensor([33, 5, 16], **i32)
    q, k, v = tokens(54)
    out, o = buffers(54)
    step(q, k, v, new, out, o, 33)
    fa.check_status()
    at = out[0].tolist()
    for b in range(B):
        held.append([k[at[b]:at[b + 1]], v[at[b]:at[b + 1]]])

    q1, k1, v1 = tokens(B)
    new.fill_(1)
    out1, o1 = buffers(B)
    saved = [t.clone() for t in (table, lens, pool.free_pages, pool.free_count)]
    step(q1, k1, v1, new, out1, o1, 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(q1, k1, v1, new, out1, o1, 1)
    for t, x in zip((table, lens, pool.free_pages, pool.free_count), saved):
        t.copy_(x)
    for _ in range(20):
        for dst, src in zip((q1, k1, v1), tokens(B)):
            dst.copy_(src)
        graph.replay()
        fa.check_status()
        for b in range(B):
            held[b] = [torch.cat([x, y[b:b + 1]]) for x, y in zip(held[b], (k1, v1))]
        assert lens.tolist() == [x[0].shape[0] for x in held]
        assert out1[2].tolist() == [n - 1 for n in lens.tolist()]
        # The rows lie where the slots say.
        where = [t.transpose(1, 2).reshape(-1, heads, d) if fmt == torch.bfloat16 else None for t in (cache.k, cache.v)]
        if fmt == torch.bfloat16:
            assert torch.equal(where[0][out1[1]], k1) and torch.equal(where[1][out1[1]], v1)
        # Self attention of the step is cross attention to the sequence's own tokens, which lie packed here.
        cu = torch.tensor(np.cumsum([0] + lens.tolist()), **i32)
        ks, vs = (torch.cat([x[j] for x in held]) for j in range(2))
        if fmt == torch.float8_e4m3fn:
            ks, vs = fa.paged_read(cache, table, cu, lens, rows=int(cu[-1]))
        o2, l2 = fa.cross_forward(q1, ks, vs, out1[0], cu, max_rows=1)
        # Both round P and O to 16 bits once: 4 half steps of |O| and sums of at most |v| < 8 of weight 1 apart.
        assert (o1[0].float() - o2.float()).abs().max() <= 4 * 2.0 ** -8 * 8 and (o1[1] - l2).abs().max() <= 1e-4
        enc.wide_q[:, :heads * group] = q1.cpu()
        check_forward(enc, o1[2], o1[3])
    done = torch.tensor([True, False, False], device="cuda")
    fa.paged_release(pool, table, lens, done)
    assert lens[0].item() == 0 and pool.free_count.item() == 40 - sum(-(-n // page) for n in lens.tolist())
    fa.paged_extend(pool, table, lens, torch.tensor([20, 0, 0], **i32), rows=20)
    fa.check_status()
    used = [x for row in table.tolist() for x in row if x >= 0]
    assert len(set(used)) == len(used) and lens[0].item() == 20


def test_python_refusals():
    p = Pool([5, 6], 4, 16, spare=4)
    i32 = dict(dtype=torch.int32, device="cuda")
    new = torch.tensor([1, 1], **i32)
    for args in ((p.d_table.long(), p.d_lens, new), (p.d_table, p.d_lens[:1], new), (p.d_table, p.d_lens, new.long()),
                 (p.d_table.cpu(), p.d_lens, new), (p.d_table[:0], p.d_lens[:0], new[:0]), (p.d_table.t(), p.d_lens, new)):
        with pytest.raises(ValueError):
            fa.paged_extend(p.pool, *args, rows=4)
    with pytest.raises(ValueError):
        fa.paged_extend(p.pool, p.d_table, p.d_lens, new)
    slots, pos, cu = torch.zeros(8, dtype=torch.int64, device="cuda"), torch.zeros(8, **i32), torch.zeros(3, **i32)
    for out in ((cu[:2], slots, pos), (cu, slots[:4], pos), (cu, pos, pos), (cu, slots, slots)):
        with pytest.raises(ValueError):
            fa.paged_extend(p.pool, p.d_table, p.d_lens, new, out=out)
    with pytest.raises(fa.FAError):  # slots that are not 16-byte aligned
        fa.paged_extend(p.pool, p.d_table, p.d_lens, new, out=(cu, slots[1:], pos[:7]))
    with pytest.raises(ValueError):
        fa.paged_release(p.pool, p.d_table, p.d_lens, new)
    with pytest.raises(ValueError):
        fa.PagePool(p.pool.free_pages.cpu(), p.pool.free_count.cpu(), 16)
    with pytest.raises(fa.FAError):
        fa.paged_release(fa.PagePool(p.pool.free_pages, p.pool.free_count, 24), p.d_table, p.d_lens,
                         torch.zeros(2, dtype=torch.bool, device="cuda"))
    p.same()
    fa.check_status()
