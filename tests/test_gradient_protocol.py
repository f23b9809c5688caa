"""The barriers of cross attention's gradient kernels (csrc/fa_cross_bwd_short.cuh, csrc/fa_cross_bwd.cuh), stepped on the CPU: their
warps as coroutines that run in any order, the tensor core's completions late but in the order of each issuing warp.  A wait is for a phase's
parity, so it must never be made two phases early or late: every wait that passes is checked to be for the phase meant, and
no order may leave every warp waiting."""
import random

import pytest

RING = 4


class Barrier:
    def __init__(self, count):
        self.count, self.arrived, self.phase = count, 0, 0

    def arrive(self):
        self.arrived += 1
        if self.arrived == self.count:
            self.arrived, self.phase = 0, self.phase + 1


class Items:
    """ShortItem: key tiles of a segment, items of a key tile (SUBS to a row tile)."""

    def __init__(self, subs):
        self.subs, self.tile, self.slot0, self.k = subs, 0, 0, 0

    def enter(self, seg):
        self.n, rows, qt = seg[0], seg[1], 128 // self.subs
        self.items = (len(rows) - 1) * self.subs + -(-rows[-1] // qt)
        self.j = self.m = 0

    sub = property(lambda s: s.m % s.subs)
    slot = property(lambda s: s.slot0 + s.m // s.subs)
    last = property(lambda s: s.m == s.items - 1)
    last_sub = property(lambda s: s.sub == s.subs - 1 or s.last)

    def next(self):
        self.m += 1
        if self.m < self.items:
            return True
        self.m, self.tile, self.j = 0, self.tile + 1, self.j + 1
        if self.j < self.n:
            return True
        self.slot0 += -(-self.items // self.subs)
        self.k += 1
        return False


def schedule(rng, bars, commits, warps):
    """Steps the warps in a random order until all have ended."""
    waits = {}

    def step(name):
        try:
            waits[name] = next(warps[name])
        except StopIteration:
            del warps[name]
            waits.pop(name, None)

    for name in list(warps):
        step(name)
    while warps:
        pending = [q for q in commits.values() if q]
        ready = [w for w in warps if (bars[waits[w][0]].phase & 1) != (waits[w][1] & 1)]
        assert ready or pending, {w: waits[w] for w in warps}  # a deadlock
        if pending and (not ready or rng.random() < 0.3):
            bars[rng.choice(pending).pop(0)].arrive()
            continue
        name = rng.choice(ready)
        bar, phase = waits[name]
        assert bars[bar].phase == phase + 1, (name, bar, phase, bars[bar].phase)
        step(name)


def run(units, stages, slots, subs, seed):
    rng = random.Random(seed)
    apart = subs == 2  # dQ has a warp of its own
    names = ["kv_done", "kv_free", "dq_done", "dq_free"]
    bars = {x: Barrier(1) for x in names + [(name, b) for name in ("s", "p", "free", "ds") for b in range(2)]}
    for i in range(stages):
        bars[("st_full", i)], bars[("st_empty", i)] = Barrier(1), Barrier(1)
    for i in range(slots):
        bars[("q_full", i)], bars[("q_empty", i)] = Barrier(1), Barrier(1)
    for i in range(RING):
        bars[("seg_full", i)], bars[("seg_empty", i)] = Barrier(1), Barrier(6 if apart else 5)
    ring = [None] * RING
    commits = {"s": [], "kv": [], "dq": []}  # completions under way, in order

    def load():
        tiles = rows = 0
        for k, unit in enumerate(units + [None]):
            yield ("seg_empty", k % RING), k // RING - 1
            ring[k % RING] = unit
            bars[("seg_full", k % RING)].arrive()
            if unit is None:
                return
            for t in range(unit[0]):
                yield ("st_empty", tiles % stages), tiles // stages - 1
                bars[("st_full", tiles % stages)].arrive()
                tiles += 1
                for _ in unit[1] if t == 0 else ():
                    yield ("q_empty", rows % slots), rows // slots - 1
                    bars[("q_full", rows % slots)].arrive()
                    rows += 1

    def segment(it):
        yield ("seg_full", it.k % RING), it.k // RING
        seg = ring[it.k % RING]
        bars[("seg_empty", it.k % RING)].arrive()
        if seg is not None:
            it.enter(seg)
        return seg

    def items(it):
        """Every item in turn: the body runs at each value yielded as None."""
        begun = False
        while True:
            if not begun and (yield from segment(it)) is None:
                return
            yield None
            begun = it.next()

    def mma_s():
        it, n = Items(subs), 0
        for wait in items(it):
            if wait is not None:
                yield wait
                continue
            if it.m == 0:
                yield ("st_full", it.tile % stages), it.tile // stages
            if it.j == 0 and it.sub == 0:
                yield ("q_full", it.slot % slots), it.slot // slots
            if n >= 2:
                yield ("free", n & 1), (n >> 1) - 1
            commits["s"].append(("s", n & 1))
            n += 1

    def issue_dq(it, row_tiles, queue):
        if it.j == 0 and it.m < subs and it.k > 0:
            yield "dq_free", it.k - 1
        queue.append(("ds", row_tiles & 1))
        if it.last:
            queue.append(("st_empty", it.tile % stages))
            if it.j == it.n - 1:
                queue.append("dq_done")

    def mma_kv():
        it, n, tiles, row_tiles = Items(subs), 0, 0, 0
        for wait in items(it):
            if wait is not None:
                yield wait
                continue
            yield ("p", n & 1), n >> 1
            if it.m == 0:
                if tiles:
                    yield "kv_free", tiles - 1
                tiles += 1
            commits["kv"].append(("free", n & 1))
            n += 1
            if it.last:
                commits["kv"].append("kv_done")
            if it.last_sub and it.j == it.n - 1:
                commits["kv"].append(("q_empty", it.slot % slots))
            if it.last_sub and not apart:
                yield from issue_dq(it, row_tiles, commits["kv"])
                row_tiles += 1

    def mma_dq():
        it, n, row_tiles = Items(subs), 0, 0
        for wait in items(it):
            if wait is not None:
                yield wait
                continue
            if it.last_sub:
                for x in range(n - (it.sub > 0), n + 1):
                    yield ("p", x & 1), x >> 1
                yield from issue_dq(it, row_tiles, commits["dq"])
                row_tiles += 1
            n += 1

    def elementwise(group):
        it, n, row_tiles = Items(subs), 0, 0
        for wait in items(it):
            if wait is not None:
                yield wait
                continue
            if n & 1 == group:
                yield ("s", group), n >> 1
                yield ("q_full", it.slot % slots), it.slot // slots
                if row_tiles:
                    yield ("ds", row_tiles - 1 & 1), row_tiles - 1 >> 1
                bars[("p", group)].arrive()
            n += 1
            row_tiles += it.last_sub

    def output():
        it, tiles = Items(subs), 0
        while (yield from segment(it)) is not None:
            for _ in range(it.n):
                yield "kv_done", tiles
                tiles += 1
                bars["kv_free"].arrive()
            yield "dq_done", it.k
            bars["dq_free"].arrive()
            it.k += 1

    warps = {"load": load(), "s": mma_s(), "kv": mma_kv(), "ew0": elementwise(0), "ew1": elementwise(1), "out": output()}
    if apart:
        warps["dq"] = mma_dq()
    schedule(rng, bars, commits, warps)


# (stages, slots, items to a row tile, row tiles of a unit at most) at d = 32, 64, 128, and other rings.
@pytest.mark.parametrize("stages,slots,subs,most", [(4, 6, 2, 4), (3, 2, 2, 2), (2, 1, 4, 1), (2, 2, 2, 2), (2, 2, 4, 2)])
def test_every_order_ends_and_no_wait_is_for_another_phase(stages, slots, subs, most):
    for seed in range(400):
        rng = random.Random(seed)
        units = [(rng.randint(1, 4), [128] * rng.randint(0, most - 1) + [rng.randint(1, 128)]) for _ in range(rng.randint(0, 12))]
        run(units, stages, slots, subs, seed)


def run_long(segments, stages, apart, dp, seed):
    """fa_cross_bwd_kernel over segments of so many streamed tiles: one issuing warp and one ring of `stages`; or (d = 256, `apart`) the
    accumulations by a warp of their own, (`dp`) dP, too, and `stages` slots of the rings A and B (`dp`: a tile's regions, each slot holds its own)."""
    rng = random.Random(seed)
    names = ["fix_full", "out_done", "drain"] + [(x, b) for x in ("p", "free") for b in range(2)]
    rings = {"a": stages[0], "b": stages[1]} if apart else {"a": stages}
    acc_ring = "a" if dp or not apart else "b"  # what the accumulations read
    bars = {x: Barrier(1) for x in names + [(r, e, i) for r in rings for e in ("full", "empty") for i in range(rings[r])]}
    first = 2 if dp else 1  # warps whose products make a tile's S and dP
    bars.update({"fix_empty": Barrier(first), ("s", 0): Barrier(first), ("s", 1): Barrier(first), "out_free": Barrier(2)})
    for i in range(RING):
        bars[("seg_full", i)], bars[("seg_empty", i)] = Barrier(1), Barrier(2 + first + apart)
    ring = [None] * RING
    commits = {0: [], 1: [], "acc": []}

    def regions(r, pos):
        """Slots of tile `pos` and their phases."""
        return [(i, pos) for i in range(rings[r])] if dp and r == "b" else [(pos % rings[r], pos // rings[r])]

    def load():
        pos = 0
        for k, n in enumerate(segments + [None]):
            yield ("seg_empty", k % RING), k // RING - 1
            ring[k % RING] = n
            bars[("seg_full", k % RING)].arrive()
            if n is None:
                return
            yield "fix_empty", k - 1
            bars["fix_full"].arrive()
            for _ in range(n):
                for r in sorted(rings, reverse=dp):
                    for slot, phase in regions(r, pos):
                        yield (r, "empty", slot), phase - 1
                        bars[(r, "full", slot)].arrive()
                pos += 1

    def segment(k):
        yield ("seg_full", k % RING), k // RING
        bars[("seg_empty", k % RING)].arrive()
        return ring[k % RING]

    def one():
        pos, ready = 0, [0, 0]
        queue, k = commits["acc"], 0
        while (n := (yield from segment(k))) is not None:
            yield "fix_full", k
            for t in range(-2, n):
                if t >= 0:
                    yield ("p", t & 1), ready[t & 1]
                    ready[t & 1] += 1
                    if t == 0 and k > 0:
                        yield "out_free", k - 1
                    queue.append(("a", "empty", (pos + t) % stages))
                if t + 2 < n:
                    yield ("a", "full", (pos + t + 2) % stages), (pos + t + 2) // stages
                    queue.append(("s", t & 1))
                    if t + 2 == n - 1:
                        queue.append("fix_empty")
            pos, k = pos + n, k + 1
            queue.append("out_done")

    def sdp(x):
        pos, used, k = 0, [0, 0], 0
        while (n := (yield from segment(k))) is not None:
            yield "fix_full", k
            for t in range(n):
                r = "ab"[x]
                if used[t & 1]:
                    yield ("free", t & 1), used[t & 1] - 1
                used[t & 1] += 1
                for slot, phase in regions(r, pos):
                    yield (r, "full", slot), phase
                    if r != acc_ring:
                        commits[x].append((r, "empty", slot))
                commits[x].append(("s", t & 1))
                if t == n - 1:
                    commits[x].append("fix_empty")
                pos += 1
            k += 1

    def acc():
        pos, ready, k = 0, [0, 0], 0
        while (n := (yield from segment(k))) is not None:
            for t in range(n):
                slot = pos % rings[acc_ring]
                yield (acc_ring, "full", slot), pos // rings[acc_ring]
                yield ("p", t & 1), ready[t & 1]
                ready[t & 1] += 1
                if t == 0 and k > 0:
                    yield "out_free", k - 1
                commits["acc"] += [("free", t & 1), (acc_ring, "empty", slot)]
                pos += 1
            commits["acc"].append("out_done")
            k += 1

    def elementwise(b):
        pos, done, k = 0, 0, 0
        while (n := (yield from segment(k))) is not None:
            for t in range(b, n, 2):
                yield ("s", b), done
                done += 1
                yield (acc_ring, "full", (pos + t) % rings[acc_ring]), (pos + t) // rings[acc_ring]
                bars[("p", b)].arrive()
            pos += n
            yield "out_done", k
            bars["out_free"].arrive()
            k += 1

    warps = {"load": load(), "ew0": elementwise(0), "ew1": elementwise(1)}
    warps.update({"s": sdp(0), "acc": acc()} if apart else {"mma": one()})
    if dp:
        warps["dp"] = sdp(1)
    schedule(rng, bars, commits, warps)


@pytest.mark.parametrize("stages,apart,dp", [(2, False, False), (3, False, False), (4, False, False), ((2, 3), True, False), ((2, 4), True, True)])
def test_the_kernel_of_longer_sequences(stages, apart, dp):
    for seed in range(400):
        rng = random.Random(seed)
        run_long([rng.choice((1, 1, 2, 3, 4, 7)) for _ in range(rng.randint(0, 12))], stages, apart, dp, seed)
