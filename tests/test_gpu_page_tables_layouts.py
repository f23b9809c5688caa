"""Page tables whose rows lie farther apart than they are wide, and calls that want no slots or no positions."""
import pytest
import torch

import oracle.tables as ref
import tiled_attention_fwd_gb300 as fa
from test_gpu_page_tables import Pool

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


def widen(p, left, right):
    """p's table as columns of a wider one, whose others hold 12345."""
    B, width = p.d_table.shape
    wide = torch.full((B, left + width + right), 12345, **I32)
    wide[:, left:left + width] = p.d_table
    p.d_table = wide[:, left:left + width]
    return lambda: (wide[:, :left] == 12345).all() and (wide[:, left + width:] == 12345).all()


@pytest.mark.parametrize("B", [1, 2, 37, 1030])
@pytest.mark.parametrize("left,right", [(0, 3), (2, 0), (5, 20)])
def test_rows_farther_apart_than_they_are_wide(B, left, right):
    p = Pool([(7 * b) % 70 for b in range(B)], 12, 16, spare=B * 7, seed=B)
    others_are_left = widen(p, left, right)
    assert p.d_table.stride(0) == 12 + left + right
    new = [(11 * b) % 60 for b in range(B)]
    p.extend(new, sum(new) + 1)
    p.extend([1] * B, B)
    assert others_are_left()
    p.release([b % 3 != 1 for b in range(B)])
    p.extend(new, sum(new) + 1)
    p.release([True] * B)
    assert others_are_left()


@pytest.mark.parametrize("wanted", [(True, False), (False, True), (False, False)])
def test_slots_and_positions_that_are_not_wanted(wanted):
    """The library takes NULL for either; the rest of the call is the same, what it reports too."""
    p = Pool([5, 20, 7, 0], 6, 16, spare=9)
    for new, code in (([1, 20, 0, 33], 0), ([1, 1, 1, 1], 0), ([30, 90, 2, 1], -11)):
        rows = 64
        slots, positions = torch.full((rows,), -7, dtype=torch.int64, device="cuda"), torch.full((rows,), -7, **I32)
        cu, counts = torch.zeros(5, **I32), torch.tensor(new, **I32)
        stream = torch.cuda.current_stream().cuda_stream
        p.count, want_cu, want_slots, want_positions, _ = ref.extend(p.table, p.lens, p.stack, p.count, new, 16, rows)
        assert fa.fa_paged_extend(p.pool._c, p.d_table.data_ptr(), 6, 6, p.d_lens.data_ptr(), counts.data_ptr(), cu.data_ptr(),
                                  slots.data_ptr() if wanted[0] else None, positions.data_ptr() if wanted[1] else None, 4, rows,
                                  stream) == 0
        assert fa.fa_status(stream) == code
        p.same()
        assert cu.tolist() == want_cu
        n = want_cu[-1]
        assert slots.tolist() == (want_slots + [-7] * (rows - n) if wanted[0] else [-7] * rows)
        assert positions.tolist() == (want_positions + [-7] * (rows - n) if wanted[1] else [-7] * rows)


def shorten(pool, table, lens, new_lens):
    """Sequences lose their last tokens (a rejected draft): the pages behind the new length go back as a table of their own, on the GPU."""
    ps, width = pool.page_size, table.shape[1]
    held, kept = (lens + ps - 1) // ps, (new_lens + ps - 1) // ps
    k = torch.arange(width, device=table.device)
    behind = table.gather(1, (kept.view(-1, 1) + k).clamp(max=width - 1).long()).contiguous()
    table.masked_fill_(k >= kept.view(-1, 1), -1)
    fa.paged_release(pool, behind, ((held - kept) * ps).int(), torch.ones_like(lens, dtype=torch.bool))
    lens.copy_(new_lens)


def test_shortened_sequences_give_their_pages_back():
    """As the header says: whoever lowers a length across a page's border gives the pages behind it back; none is lost then, in a captured
    loop either."""
    ps, width, total = 16, 6, 20
    pool = fa.PagePool.full(total, ps)
    table, lens = torch.full((3, width), -1, **I32), torch.zeros(3, **I32)
    counts, keep = torch.zeros(3, **I32), torch.zeros(3, **I32)
    cu, slots, positions = torch.zeros(4, **I32), torch.full((64,), -1, dtype=torch.int64, device="cuda"), torch.full((64,), -1, **I32)

    def step():
        fa.paged_extend(pool, table, lens, counts, out=(cu, slots, positions))
        shorten(pool, table, lens, lens - keep)

    step()  # (of no tokens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    want = [0] * 3
    for new, dropped in (([17, 5, 30], [0, 0, 0]), ([8, 30, 1], [7, 28, 1]), ([16, 16, 1], [16, 1, 0]), ([2, 2, 18], [0, 0, 17]),
                         ([0, 16, 4], [0, 16, 4])):
        counts.copy_(torch.tensor(new)), keep.copy_(torch.tensor(dropped))
        graph.replay()
        fa.check_status()
        want = [a + b - c for a, b, c in zip(want, new, dropped)]
        assert lens.tolist() == want
        free = pool.free_pages[:pool.free_count.item()].tolist()
        used = [x for row, n in zip(table.tolist(), want) for x in row[:-(-n // ps)]]
        assert sorted(used + free) == list(range(total))
        assert all(x == -1 for row, n in zip(table.tolist(), want) for x in row[-(-n // ps):])
    fa.paged_release(pool, table, lens, torch.ones(3, dtype=torch.bool, device="cuda"))
    fa.check_status()
    assert sorted(pool.free_pages.tolist()) == list(range(total)) and pool.free_count.item() == total
