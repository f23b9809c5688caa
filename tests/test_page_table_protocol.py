"""The cluster of fa_paged_release_kernel (csrc/fa_paged_tables.cu), stepped on the CPU: its CTAs start one by one, their warps run in any
order.  A store to another CTA's shared memory may only meet one that has started and not ended, and a round's counts may only be
overwritten when every CTA has read them."""
import random
from pathlib import Path

import pytest

WARPS = 2  # of a CTA here (32 there); a round is of 4 units a warp of 16 CTAs


class Cluster:
    """barrier.cluster: a phase ends when every warp of every CTA has arrived."""

    def __init__(self, ctas):
        self.ctas, self.arrived, self.phase = ctas, 0, 0
        self.started, self.ended = [False] * ctas, [0] * ctas
        self.count = [{} for _ in range(ctas)]  # s_count of each CTA: unit of the round -> round

    def arrive(self):
        self.arrived += 1
        if self.arrived == self.ctas * WARPS:
            self.arrived, self.phase = 0, self.phase + 1

    def store(self, cta, at, value):
        assert self.started[cta], "a store to a CTA that has not started"
        assert self.ended[cta] == 0, "a store to a CTA that has ended"
        self.count[cta][at] = value


def warp(c, rank, w, rounds, synced, entry):
    """One warp of CTA `rank`; yields where it may be interrupted, or what it waits for (a function)."""
    phase = 0  # cluster phases that this warp has arrived at

    def wait():
        mine = phase
        return lambda: c.phase >= mine

    units = 4 * 16 * WARPS
    if entry:
        c.arrive()
        phase += 1
    all_started = not entry
    for r in range(rounds):
        for i0 in range(rank * WARPS + w, units, 4 * c.ctas * WARPS):
            yield None  # the loads
            if not all_started:
                yield wait()
                all_started = True
            for e in range(4):
                for cta in range(c.ctas):
                    if i0 + e * c.ctas * WARPS < units:
                        c.store(cta, i0 + e * c.ctas * WARPS, r)
                yield None
        c.arrive()
        phase += 1
        yield wait()
        assert len(c.count[rank]) == units and all(x == r for x in c.count[rank].values()), (rank, r)
        yield None
        # block_scan and the barrier behind it: every warp of the CTA has read its counts.
        synced[rank] += 1
        goal = (r + 1) * WARPS
        yield lambda: synced[rank] >= goal
        yield None  # the stack and the table
        if r + 1 < rounds:
            c.arrive()
            phase += 1
            yield wait()
    c.ended[rank] += 1


def run(ctas, rounds, seed, entry=True):
    rng = random.Random(seed)
    c, synced = Cluster(ctas), [0] * ctas
    warps, waits = [], {}
    order = rng.sample(range(ctas), ctas)
    while warps or order:
        if order and (not warps or rng.random() < 0.1):
            rank = order.pop()
            c.started[rank] = True
            for w in range(WARPS):
                warps.append(warp(c, rank, w, rounds, synced, entry))
            continue
        ready = [x for x in warps if x not in waits or waits[x] is None or waits[x]()]
        if not ready:
            assert order, "every warp waits"
            continue
        x = rng.choice(ready)
        try:
            waits[x] = next(x)
        except StopIteration:
            warps.remove(x)
            waits.pop(x, None)


@pytest.mark.parametrize("ctas", [16, 8])
@pytest.mark.parametrize("rounds", [1, 3])
def test_release_touches_its_neighbours_when_they_are_there(ctas, rounds):
    for seed in range(6):
        run(ctas, rounds, seed)


def test_the_barrier_at_the_beginning_is_what_sees_to_it():
    with pytest.raises(AssertionError, match="not started"):
        for seed in range(6):
            run(16, 1, seed, entry=False)


def test_the_kernel_waits_before_its_first_store_to_a_neighbour():
    text = (Path(__file__).parent.parent / "tiled_attention_fwd_gb300" / "csrc" / "fa_paged_tables.cu").read_text()
    text = text[text.index("fa_paged_release_kernel(const TableArgs"):]
    assert text.index("cluster_arrive();") < text.index("cluster_wait();") < text.index("st_cluster(")
