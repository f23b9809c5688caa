"""The hand-over of a unit's row statistics in the forward kernels (csrc/fa_fwd_tc.cuh, csrc/fa_paged_chunk.cuh), as a model:
every interleaving of the MMA warp, the two softmax warpgroups and the correction warpgroup of one CTA, for units of one key
tile.  An mbarrier's parity wait passes once the phase of that parity is over, so a barrier that is two phases ahead looks as
if nothing had arrived."""
import pytest


def explore(units, barriers, slot_by_unit, order=("l_full", "o_done")):
    """(deadlocks, wrong reads) reachable; units: the tiles each unit has, [(1, 1), ..]; `barriers` per tile (1 or 2);
    statistics in slot (unit's index & 1) or (number of the tile's finished units & 1); order: of the correction's waits."""
    mine = [[k for k, has in enumerate(units) if has[t]] for t in range(2)]  # units of tile t

    def mma():  # (kind, tile): S of the first unit, then every unit's P V, then the next unit's S
        for t in range(2):
            if units[0][t]:
                yield "s", t
        for k, has in enumerate(units):
            for t in range(2):
                if has[t]:
                    yield "pv", t
            for t in range(2):
                if k + 1 < len(units) and units[k + 1][t]:
                    yield "s", t

    mma = list(mma())
    correction = [("free", t, None) for t in range(2)]
    for k, has in enumerate(units):
        for t in range(2):
            if has[t]:
                correction += [(order[0], t, k), (order[1], t, k), ("read", t, k), ("free", t, k)]

    # State: program counters (MMA, softmax 0, softmax 1, correction); per tile the phases of s_full, o_done, the softmax's and
    # the correction's arrivals on pv_go, l_full; the units whose statistics the slots hold.
    start = ((0, 0, 0, 0), ((0, 0, 0, 0), (0, 0, 0, 0)), ((0,) * barriers,) * 2, ((-1, -1), (-1, -1)))

    def passed(phases, parity):
        return (phases & 1) != parity

    def steps(state):
        pc, count, l_full, slots = state

        def put(tup, i, v):
            return tup[:i] + (v,) + tup[i + 1:]

        def bump(t, i):
            return put(count, t, put(count[t], i, count[t][i] + 1))

        if pc[0] < len(mma):
            kind, t = mma[pc[0]]
            s, o, p, f = count[t]
            if kind == "s":
                yield put(pc, 0, pc[0] + 1), bump(t, 0), l_full, slots
            elif min(p, f) > o:  # P V number o: P posted and O free
                yield put(pc, 0, pc[0] + 1), bump(t, 1), l_full, slots
        for t in range(2):  # softmax: two steps a unit (P posted; statistics written and announced)
            i = pc[1 + t]
            if i < 2 * len(mine[t]):
                n = i // 2
                if i % 2 == 0:
                    if passed(count[t][0], n & 1):
                        yield put(pc, 1 + t, i + 1), bump(t, 2), l_full, slots
                else:
                    unit = mine[t][n]
                    slot = (unit if slot_by_unit else n) & 1
                    bar = n % barriers
                    yield (put(pc, 1 + t, i + 1), count, put(l_full, t, put(l_full[t], bar, l_full[t][bar] + 1)),
                           put(slots, t, put(slots[t], slot, unit)))
        if pc[3] < len(correction):
            kind, t, k = correction[pc[3]]
            n = None if k is None else mine[t].index(k)
            on = put(pc, 3, pc[3] + 1)
            if kind == "free":
                yield on, bump(t, 3), l_full, slots
            elif kind == "o_done":
                if passed(count[t][1], n & 1):
                    yield on, count, l_full, slots
            elif kind == "l_full":
                if passed(l_full[t][n % barriers], n // barriers & 1):
                    yield on, count, l_full, slots
            else:
                if slots[t][(k if slot_by_unit else n) & 1] != k:
                    wrong.add((t, k))
                yield on, count, l_full, slots

    seen, todo, wrong, stuck = {start}, [start], set(), 0
    last = (len(mma), 2 * len(mine[0]), 2 * len(mine[1]), len(correction))
    while todo:
        state = todo.pop()
        after = list(steps(state))
        if not after and state[0] != last:
            stuck += 1
        for s in after:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return stuck, wrong


BOTH, FIRST = (1, 1), (1, 0)  # a unit at the end of an odd number of query tiles has the first alone


@pytest.mark.parametrize("order", [("l_full", "o_done"), ("o_done", "l_full")])  # fa_fwd_tc.cuh, fa_paged_chunk.cuh
@pytest.mark.parametrize("units", [[BOTH] * 5, [BOTH, FIRST] * 3, [FIRST, BOTH, BOTH, FIRST, BOTH], [FIRST] * 4])
def test_two_barriers_hand_over_every_unit(units, order):
    assert explore(units, 2, False, order) == (0, set())


@pytest.mark.parametrize("order", [("l_full", "o_done"), ("o_done", "l_full")])
def test_one_barrier_can_be_overrun(order):
    """What the two barriers are for: with one, a correction that comes late waits for a phase that is long over."""
    stuck, _ = explore([BOTH] * 4, 1, False, order)
    assert stuck > 0


def test_slots_by_the_units_index_can_be_overwritten():
    """What counting a tile's own units is for: where a unit has no second tile, units k and k + 2 share a slot."""
    _, wrong = explore([BOTH, FIRST] * 3, 2, True)
    assert wrong
