"""How fa_cross_prep_kernel (csrc/fa_cross_bwd.cuh) deals out and places the rows' vectors, stepped on the CPU: for offsets of any kind
every index lies within the vectors, and where sequences share no rows each tile is made once, in a place of its own."""
import random

import pytest

THREADS = 256


def sequences(cu, rows, keys):
    """(first row, rows or 0) as cross_seq cuts them; no rows where there are no keys."""
    out = []
    for b in range(len(cu) - 1):
        lo, hi = cu[b], cu[b + 1]
        fine = 0 <= lo <= hi <= rows
        out.append((lo, hi - lo) if fine and keys[b] else (0, 0))
    return out


def prep(seqs, t0, heads, most, grid):
    """The kernel's steps, block by block: {(sequence, tile, head): place} and tile0."""
    B = len(seqs)
    add = lambda x, y: min(x + y, most)
    tiles_at = lambda b: -(-seqs[b][1] // t0) if b < B else 0

    def scan(xs):
        out, x = [], 0
        for y in xs:
            x = add(x, y)
            out.append(x)
        return out

    per = -(-B // THREADS)
    mine = []
    for t in range(THREADS):
        x = 0
        for b in range(t * per, min((t + 1) * per, B)):
            x = add(x, tiles_at(b))
        mine.append(x)
    upto = []
    below = 0
    firsts = []
    for w in range(THREADS // 32):
        s = scan(mine[32 * w:32 * w + 32])
        upto += [add(x, below) for x in s]
        firsts += [add(x, below) for x in [0] + s[:-1]]
        below = add(below, s[-1])
    places = below * heads
    share = 1 if places <= grid else -(-places // grid)
    made, tile0 = {}, {}
    for block in range(grid):
        start = share * block
        end = min(start + share, places)
        if start >= end:
            continue
        tile_at = start // heads
        who = [t for t in range(THREADS) if firsts[t] <= tile_at < upto[t]]
        assert len(who) == 1
        b, before = who[0] * per, firsts[who[0]]
        while per > 1:
            y = scan([tiles_at(b + i) for i in range(32)])
            hit = [i for i in range(32) if add(before, y[i]) > tile_at]
            at = hit[0] if hit else 31
            before = add(before, ([0] + y)[at] if hit else y[31])
            b += at if hit else 32
            assert b < B
            if hit:
                break
        tile, head = tile_at - before, start - tile_at * heads
        tiles = tiles_at(b)
        assert 0 <= tile < tiles and 0 <= head < heads
        for x in range(start, end):
            first = min(before, most - tiles)
            if tile == 0 and head == 0:
                tile0[b] = first
            assert 0 <= first and first + tile < most
            assert (b, tile, head) not in made
            made[b, tile, head] = first + tile
            head += 1
            if head < heads:
                continue
            head, tile = 0, tile + 1
            if tile < tiles:
                continue
            tile = 0
            before = add(before, tiles)
            if x + 1 == end:
                break
            while True:
                b += 1
                assert b < B
                tiles = tiles_at(b)
                if tiles:
                    break
    return made, tile0


def check(cu, rows, keys, t0, heads, grid, shared):
    seqs, B = sequences(cu, rows, keys), len(cu) - 1
    most = rows // t0 + B
    made, tile0 = prep(seqs, t0, heads, most, grid)
    for b, (_, n) in enumerate(seqs):  # what the products' kernels read
        need = -(-n // t0)
        if need == 0:
            continue
        vec0 = min(tile0.get(b, 0xffffffff), most)
        assert (heads - 1) * most + vec0 + need <= (heads + 1) * most  # (of the last head; there is room for one more)
        if not shared:
            assert all(made[b, t, h] == vec0 + t for t in range(need) for h in range(heads))
    if not shared:
        assert len({(p, h) for (_, _, h), p in made.items()}) == len(made)


@pytest.mark.parametrize("B", [1, 3, 31, 200, 256, 257, 700, 9000])
def test_tiles_are_made_once(B):
    rng = random.Random(B)
    for t0, heads, grid in ((64, 3, 1216), (2, 1, 7), (21, 5, 64)):
        n = [rng.choice([0, 1, 2, rng.randrange(1, 200 if B < 1000 else 9)]) for _ in range(B)]
        cu = [rng.randrange(5)]
        for x in n:
            cu.append(cu[-1] + x)
        rows = cu[-1] + rng.randrange(4)
        keys = [rng.random() < 0.9 for _ in range(B)]
        check(cu, rows, keys, t0, heads, grid, False)
        for bad in (-1, -2 ** 31, 2 ** 31 - 1, rows + 1):  # an offset that names what is not there
            x = list(cu)
            x[rng.randrange(B + 1)] = bad
            check(x, rows, keys, t0, heads, grid, False)


def test_ranges_in_no_order():
    rng = random.Random(0)
    for _ in range(200):
        n = rng.randrange(1, 90)
        cu = [n, 2 * n, 0, n, 5 * n, 6 * n, 2 * n, 4 * n]  # (the ranges that go back count as no rows; [n, 5n) shares rows: cut it)
        cu = cu[:4] + [-1] + cu[4:]
        check(cu, 6 * n, [True] * (len(cu) - 1), rng.choice([2, 21, 64]), rng.choice([1, 4]), rng.choice([3, 64, 1216]), False)


@pytest.mark.parametrize("B", [2, 40, 300, 2000])
def test_ranges_that_share_rows_stay_within_the_vectors(B):
    """They may not, but nothing is touched that is not there."""
    rng = random.Random(B)
    for t0, heads, grid in ((64, 3, 1216), (2, 1, 7), (21, 5, 64)):
        rows = 300
        for cu in ([0, rows] * B, [rng.randrange(-5, rows + 5) for _ in range(B + 1)], [0, 7] * B):
            check(cu[:B + 1], rows, [True] * B, t0, heads, grid, True)
