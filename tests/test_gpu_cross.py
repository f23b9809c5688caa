"""Cross attention of ragged batches on the GPU, forward and backward, against the fp64 oracle (bounds: cross_util)."""
import numpy as np
import pytest
import torch

import oracle.cross as ref
import tiled_attention_fwd_gb300 as fa
from cross_util import Ragged, backward, check, check_backward, check_forward, forward

pytestmark = pytest.mark.gpu

D = (32, 64, 128, 256)


# ------------------------------------------------------------------ shapes
@pytest.mark.parametrize("d", D)
@pytest.mark.parametrize("heads,group", [(1, 1), (3, 1), (2, 4), (1, 8), (2, 3), (1, 32)])
def test_single_rows(d, heads, group):
    check(Ragged([1, 1, 1, 1], [1, 333, 64, 1000], heads, group, d, seed=d + group))


@pytest.mark.parametrize("d", D)
@pytest.mark.parametrize("rows,keys", [([1], [1]), ([2, 5, 8], [15, 16, 17]), ([31, 33], [127, 129]),
                                       ([63, 64, 65], [128, 95, 97]), ([127, 128, 129], [255, 256, 257]),
                                       ([300, 1], [1, 700])])
def test_lengths_around_the_tiles(d, rows, keys):
    check(Ragged(rows, keys, 2, 1, d, seed=sum(rows)))
    check(Ragged(rows, keys, 1, 3, d, seed=sum(rows) + 1, padded=True, lead=5, pad=7))


@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 7, 8, 12, 16, 24, 31, 32])
@pytest.mark.parametrize("d", [64, 128])
def test_group_sizes(group, d):
    check(Ragged([40, 3, 150], [100, 333, 200], 1, group, d, seed=group))


def test_group_sizes_of_wide_heads():
    for group in (1, 3, 8, 20, 32):
        check(Ragged([40, 3, 70], [100, 133, 200], 1, group, 256, seed=group))


@pytest.mark.parametrize("d", D)
@pytest.mark.parametrize("padded", [False, True])
def test_fused_projections_and_offsets(d, padded):
    check(Ragged([20, 0, 130], [77, 50, 260], 2, 2, d, padded=padded, fused=True, lead=3, pad=11, seed=d))


@pytest.mark.parametrize("d", D)
@pytest.mark.parametrize("padded", [False, True])
def test_sequences_without_rows_or_keys(d, padded):
    check(Ragged([0, 4, 0, 90, 1, 40], [50, 0, 0, 0, 7, 300], 2, 2, d, padded=padded, pad=2, seed=d))
    check(Ragged([3, 60], [0, 0], 1, 2, d, padded=padded, pad=2, seed=d))
    check(Ragged([0, 0], [9, 140], 1, 2, d, padded=padded, pad=2, seed=d))


@pytest.mark.parametrize("d", D)
def test_many_units_on_every_sm(d):
    rng = np.random.default_rng(d)
    B = 120
    rows, keys = rng.integers(0, 90, B).tolist(), rng.integers(0, 260, B).tolist()
    check(Ragged(rows, keys, 2, 2, d, padded=False, seed=d))


@pytest.mark.parametrize("B", [1023, 1025, 1700])
def test_more_sequences_than_threads(B):
    rng = np.random.default_rng(B)
    rows, keys = rng.integers(0, 3, B).tolist(), rng.integers(0, 9, B).tolist()
    rows[B // 2], keys[B // 2] = 200, 150
    check(Ragged(rows, keys, 1, 2, 32, seed=B))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows,keys", [([1], [20000]), ([8], [9001]), ([130], [9001]), ([3001], [200]), ([700], [3000])])
def test_few_long_sequences_are_split_and_joined(d, rows, keys):
    check(Ragged(rows, keys, 1, 2, d, seed=rows[0]))


# ------------------------------------------------------------------ values
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("rows", [[3, 1], [100, 70]])
def test_large_logits_and_late_maxima(d, rows):
    s = Ragged(rows, [400, 130], 2, 2, d, seed=1, gain=6.0)
    s.wide_k[350:, :] *= 3
    check(s)
    check(Ragged(rows, [400, 130], 2, 2, d, seed=2), scale=1e-6)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -3e38])
@pytest.mark.parametrize("rows", [[2, 3], [90, 70]])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_padding_and_neighbours_are_never_seen(value, rows, d):
    """What lies between the sequences' keys and behind their rows, and a whole neighbour, hold anything."""
    s = Ragged(rows + rows, [37, 130, 61, 5], 2, 2, d, padded=True, lead=2, pad=3, seed=4)
    want = forward(s)
    grads = backward(s, *want)
    for row0, n, key0, places, length in s.sequences():
        s.wide_k[key0 + length:key0 + places] = value
    s.wide_q[torch.from_numpy(~s.mine_q)] = value
    row0, n, key0, places, length = s.sequences()[1]  # the neighbour
    s.wide_k[key0:key0 + length] = value
    s.wide_q[row0:row0 + n] = value
    got = forward(s)
    keep_q, keep_k = torch.from_numpy(s.mine_q.copy()), torch.from_numpy(s.mine_k.copy())
    keep_q[row0:row0 + n] = False
    keep_k[key0:key0 + places] = False
    assert torch.equal(got[0][keep_q.cuda()], want[0][keep_q.cuda()])
    assert torch.equal(got[1][:, keep_q.cuda()], want[1][:, keep_q.cuda()])
    again = backward(s, *got)
    for x, y, keep in zip(again, grads, (keep_q, keep_k, keep_k)):
        assert torch.equal(x[keep.cuda()], y[keep.cuda()])


@pytest.mark.parametrize("rows", [[2], [90]])
def test_a_nan_reaches_its_own_sequence_only(rows):
    s = Ragged(rows + rows, [200, 130], 1, 2, 64, seed=5)
    s.wide_k[50, 1, 3] = float("nan")  # of v: one column of O
    o, lse = forward(s)
    n = rows[0]
    assert torch.isnan(o[:n, :, 3]).all() and not torch.isnan(o[:n, :, 4:]).any() and not torch.isnan(o[n:]).any()
    assert torch.isfinite(lse).all()
    dq, dk, dv = backward(s, o, lse)
    assert torch.isnan(dq[:n]).all() and torch.isfinite(dq[n:]).all()
    assert torch.isnan(dk[:200]).all() and torch.isfinite(dk[200:]).all()
    assert torch.isfinite(dv).all()  # dV = P^T dO does not read V


# ------------------------------------------------------------------ gradients
def test_gradients_are_those_of_differences():
    """A loss sum(w o) moved along random directions of q, k and v: differences of the forward's fp64 oracle (step 2^-10, whose
    own error is its square times a third derivative) against the kernel's gradients.  Four roundings of half a step of bf16
    (O, P, dS, the result), independent, leave an error of norm 2 * 2^-8 of the gradient's at most; along a random direction that is
    a normal variable's deviation, and 4 of those are allowed."""
    s = Ragged([20, 60], [50, 33], 2, 2, 64, seed=9)
    o, lse = forward(s)
    grads = [t.cpu().double().numpy() for t in backward(s, o, lse)]
    q, dout, k, v = (t.double().numpy() for t in s.host)
    rng = np.random.default_rng(0)
    for which in range(3):
        x = [q, k, v]
        way = rng.standard_normal(x[which].shape)
        loss = []
        for sign in (1, -1):
            y = list(x)
            y[which] = x[which] + sign * 2.0 ** -10 * way
            loss.append((ref.attention(*y, s.cu_rows, s.cu_keys, None, 64 ** -0.5)[0] * dout).sum())
        slope = (loss[0] - loss[1]) * 2.0 ** 9
        size = np.linalg.norm(grads[which])
        assert abs((grads[which] * way).sum() - slope) <= 4 * 2 * 2.0 ** -8 * size, which


def test_a_batch_of_one_length_is_the_plain_backward():
    """Heads of their own and one length: fa_bwd_strided's gradients, to both sides' bounds."""
    B, n, m, h, d = 2, 100, 160, 3, 64
    s = Ragged([n] * B, [m] * B, h, 1, d, seed=3)
    q, dout, k, v = s.tensors()
    o, lse = forward(s)
    mine = backward(s, o, lse)

    def batched(t, length):
        return t.view(B, length, h, d).transpose(1, 2)

    ob, lb = fa.forward(batched(q, n), batched(k, m), batched(v, m))
    assert torch.allclose(ob, batched(o, n), atol=2.0 ** -7)
    plain = fa.backward(batched(q, n), batched(k, m), batched(v, m), ob, lb, batched(dout, n).contiguous())
    for x, y, length in zip(mine, plain, (n, m, m)):
        assert (batched(x, length).float() - y.float()).norm() <= 2.0 ** -7 * y.float().norm()


@pytest.mark.parametrize("d", [64, 128])
def test_same_inputs_give_the_same_bits(d):
    s = Ragged([700, 81, 3], [500, 1700, 900], 2, 4, d, seed=21)
    o, lse = forward(s)
    grads = backward(s, o, lse)
    for _ in range(3):
        again = forward(s)
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)
        assert all(torch.equal(a, b) for a, b in zip(backward(s, o, lse), grads))


# ------------------------------------------------------------------ graphs, streams, workspaces
@pytest.mark.parametrize("rows", [[1, 2, 0], [60, 3, 200]])
def test_captured_calls_replay_with_new_lengths(rows):
    """One capture of both passes; replays with other offsets, lengths and contents."""
    first = Ragged(rows, [50, 300, 120], 2, 2, 64, seed=1, padded=True, pad=100)
    q, dout, k, v = first.tensors()
    cu_rows, cu_keys, lens = first.batch()
    o = torch.full((first.T, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, first.T), 7.0, device="cuda")
    grads = [torch.full(t.shape, 7.0, dtype=torch.bfloat16, device="cuda") for t in (q, k, v)]
    ws, wsb = fa.cross_workspace(k), fa.cross_backward_workspace(q, k, 3)

    def calls():
        fa.cross_forward(q, k, v, cu_rows, cu_keys, lens, max_rows=300, out=o, lse=lse, workspace=ws)
        fa.cross_backward(q, k, v, o, lse, dout, cu_rows, cu_keys, lens, out=grads, workspace=wsb)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        calls()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for seed, new_rows, keys in ((1, rows, [50, 300, 120]), (2, rows[::-1], [303, 0, 41]), (3, [0] * 3, [1, 2, 3]),
                                 (4, [sum(rows), 0, 0], [200, 10, 303])):
        s = Ragged(new_rows, keys, 2, 2, 64, seed=seed)
        s.key_lens, s.cu_keys, s.T, s.K = keys, first.cu_keys, first.T, first.K
        s.wide_q = torch.full_like(first.wide_q, float("nan"))
        s.wide_k = torch.full_like(first.wide_k, float("nan"))
        g = torch.Generator().manual_seed(seed)
        s.wide_q[:sum(new_rows)] = torch.randn(sum(new_rows), 8, 64, generator=g).bfloat16()
        s.mine_q = np.arange(s.T) < sum(new_rows)
        s.mine_k = first.mine_k
        for row0, n, key0, places, length in s.sequences():
            s.wide_k[key0:key0 + length] = torch.randn(length, 4, 64, generator=g).bfloat16()
        for dst, src in zip((q, dout, k, v), s.host):
            dst.copy_(src)
        cu_rows.copy_(torch.tensor(s.cu_rows))
        lens.copy_(torch.tensor(keys))
        for t in (o, lse, *grads):
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        fa.check_status()
        check_forward(s, o, lse)
        check_backward(s, o, lse, grads)


def test_two_streams_with_workspaces_of_their_own():
    setups = [Ragged([n, 300], [2000, 90], 2, 2, 128, seed=n) for n in (1, 90)]
    jobs = []
    for s in setups:
        q, dout, k, v = s.tensors()
        o, lse = torch.empty_like(q), torch.empty(4, s.T, device="cuda")
        grads = [torch.full(t.shape, 7.0, dtype=torch.bfloat16, device="cuda") for t in (q, k, v)]
        jobs.append((s, (q, dout, k, v), s.batch(), o, lse, grads, fa.cross_workspace(k),
                     fa.cross_backward_workspace(q, k, 2), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (q, dout, k, v), batch, o, lse, grads, ws, wsb, stream in jobs:
            with torch.cuda.stream(stream):
                fa.cross_forward(q, k, v, *batch, out=o, lse=lse, workspace=ws)
                fa.cross_backward(q, k, v, o, lse, dout, *batch, out=grads, workspace=wsb)
    torch.cuda.synchronize()
    fa.check_status()
    for s, _, _, o, lse, grads, _, _, _ in jobs:
        check_forward(s, o, lse)
        check_backward(s, o, lse, grads)


def test_workspaces_of_any_contents():
    s = Ragged([40, 3], [100, 900], 2, 2, 64, seed=2)
    q, _, k, _ = s.tensors()
    for fill in (0, 0xff, 0x7f):
        ws = fa.cross_workspace(k).fill_(fill)
        o, lse = forward(s, workspace=ws)
        check_forward(s, o, lse)
        wsb = fa.cross_backward_workspace(q, k, 2).fill_(fill)
        check_backward(s, o, lse, backward(s, o, lse, workspace=wsb))


# ------------------------------------------------------------------ large offsets
def test_keys_beyond_2_to_the_32_elements():
    """k and v are views into 17 GB each of padded places; the last sequence lies behind 2^32 elements."""
    heads, d, S = 8, 128, 2_100_000
    B = 4
    k, v = (torch.zeros(B * S, heads, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert k.numel() > 2 ** 32
    keys, rows = [60, 0, 33, 200], [2, 1, 0, 70]
    s = Ragged(rows, keys, heads, 1, d, seed=6)
    q, dout, ks, vs = s.tensors()
    cu_keys = torch.arange(B + 1, dtype=torch.int32, device="cuda") * S
    for b in range(B):
        at = slice(int(s.cu_keys[b]), int(s.cu_keys[b + 1]))
        k[b * S:b * S + keys[b]], v[b * S:b * S + keys[b]] = ks[at], vs[at]
    lens = torch.tensor(keys, dtype=torch.int32, device="cuda")
    cu_rows = s.batch()[0]
    o, lse = fa.cross_forward(q, k, v, cu_rows, cu_keys, lens)
    fa.check_status()
    check_forward(s, o, lse)
    dk, dv = (torch.empty_like(t) for t in (k, v))
    dq = torch.empty_like(q)
    fa.cross_backward(q, k, v, o, lse, dout, cu_rows, cu_keys, lens, out=(dq, dk, dv))
    fa.check_status()
    mine = [torch.cat([t[b * S:b * S + keys[b]] for b in range(B)]) for t in (dk, dv)]
    check_backward(s, o, lse, (dq, *mine))
    for t in (dk, dv):
        assert all(not t[b * S + keys[b]:(b + 1) * S].any() for b in range(B))  # zeros behind the keys


# ------------------------------------------------------------------ what is not there
@pytest.mark.parametrize("n", [1, 40])
def test_batches_that_name_what_is_not_there_are_reported(n):
    """Bad offsets and lengths are reported once, and sequences that do not touch them stay right."""
    s = Ragged([n, n, n], [100, 60, 80], 1, 2, 64, padded=True, seed=3)
    q, dout, k, v = s.tensors()
    good = forward(s)
    want = backward(s, *good)
    cu_rows, cu_keys, lens = s.batch()
    big = 2 ** 31 - 1
    bad = []
    for i, value in ((1, -1), (1, big), (1, 3 * n + 50), (2, n - 1)):
        x = cu_rows.clone()
        x[i] = value
        bad.append((x, cu_keys, lens))
    for i, value in ((1, -7), (1, big), (2, 5)):
        x = cu_keys.clone()
        x[i] = value
        bad.append((cu_rows, x, lens))
    for value in (-1, 104, big):
        x = lens.clone()
        x[1] = value
        bad.append((cu_rows, cu_keys, x))
    for i, (a, b, c) in enumerate(bad):
        o, lse = (torch.full_like(t, 7.0) for t in good)
        fa.cross_forward(q, k, v, a, b, c, max_rows=3 * n, out=o, lse=lse)
        with pytest.raises(fa.FAError) as e:
            fa.check_status()
        assert e.value.code == -11
        grads = [torch.full_like(t, 7.0) for t in (q, k, v)]
        fa.cross_backward(q, k, v, *good, dout, a, b, c, out=grads)
        with pytest.raises(fa.FAError):
            fa.check_status()
        if i >= 7:  # a length: the other sequences are as they were
            other = torch.tensor([True] * n + [False] * n + [True] * n, device="cuda")
            assert torch.equal(o[other], good[0][other]) and torch.equal(grads[0][other], want[0][other])
            S = s.sequences()[1][2:4]
            other = torch.ones(s.K, dtype=torch.bool, device="cuda")
            other[S[0]:S[0] + S[1]] = False
            assert torch.equal(grads[1][other], want[1][other]) and torch.equal(grads[2][other], want[2][other])
    fa.check_status()  # reported once


def test_more_rows_than_max_rows_are_left_and_reported():
    for n, most in ((3, 2), (70, 1), (70, 60)):
        s = Ragged([n, 1], [100, 60], 1, 2, 64, seed=3)
        good = forward(s)
        q, _, k, v = s.tensors()
        o, lse = (torch.full_like(t, 7.0) for t in good)
        fa.cross_forward(q, k, v, *s.batch(), max_rows=most, out=o, lse=lse)
        with pytest.raises(fa.FAError):
            fa.check_status()
        assert (o[:n] == 7.0).all() and torch.equal(o[n:], good[0][n:])


def test_no_rows_or_keys_at_all():
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(30, 2, 64, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    none, some = torch.tensor([0, 0], **i32), torch.tensor([0, 30], **i32)
    o, lse = fa.cross_forward(q, k, k, none, some)
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
    out = (torch.full_like(q, 7.0), torch.full_like(k, 7.0), torch.full_like(k, 7.0))
    fa.cross_backward(q, k, k, o, lse, q, none, some, out=out)
    assert not out[1].any() and not out[2].any()
    q = torch.ones(30, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = k[:0]
    o, lse = fa.cross_forward(q, k, k, some, none)
    assert not o.any() and torch.isneginf(lse).all()
    dq, dk, dv = fa.cross_backward(q, k, k, o, lse, q, some, none)
    assert not dq.any() and dk.shape == (0, 2, 64)
    q = q[:0]
    fa.cross_backward(q, k, k, *fa.cross_forward(q, k, k, none, none), q, none, none)
    fa.check_status()


def test_python_refusals():
    s = Ragged([2], [20], 2, 2, 64)
    q, dout, k, v = s.tensors()
    cu_rows, cu_keys, _ = s.batch()
    lens = cu_keys[1:].clone()
    for args in ((q.float(), k, v, cu_rows, cu_keys), (q, k, v, cu_rows.long(), cu_keys), (q, k, v, cu_rows, cu_keys[:1]),
                 (q, k, v[:3], cu_rows, cu_keys), (q, k[..., :32], v, cu_rows, cu_keys), (q, k, v, cu_rows.cpu(), cu_keys),
                 (q[0], k, v, cu_rows, cu_keys), (q, k, v, cu_rows, cu_keys, cu_keys), (q, k, v, cu_rows[:1], cu_keys[:1]),
                 (q, k.transpose(1, 2), v, cu_rows, cu_keys), (q.cpu(), k, v, cu_rows, cu_keys), (q, k.cpu(), v, cu_rows, cu_keys)):
        with pytest.raises(ValueError):
            fa.cross_forward(*args)
    with pytest.raises(fa.FAError):  # 3 query heads over 2 heads
        fa.cross_forward(q[:, :3], k, v, cu_rows, cu_keys)
    with pytest.raises(fa.FAError):  # a stride of 0
        fa.cross_forward(q, k[:, :1].expand(-1, 2, -1), v, cu_rows, cu_keys, lens)
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    o, lse = fa.cross_forward(q, k, v, cu_rows, cu_keys)
    with pytest.raises(fa.FAError):
        fa.cross_forward(q, k, v, cu_rows, cu_keys, workspace=small[:0])
    with pytest.raises(fa.FAError):
        fa.cross_backward(q, k, v, o, lse, dout, cu_rows, cu_keys, workspace=small)
    with pytest.raises(ValueError):
        fa.cross_backward(q, k, v, o, lse[:1], dout, cu_rows, cu_keys)
    with pytest.raises(ValueError):
        fa.cross_backward(q, k, v, o[:1], lse, dout, cu_rows, cu_keys)
    with pytest.raises(ValueError):
        fa.cross_backward(q, k, v, o, lse, dout, cu_rows, cu_keys, out=(q, k, v[:1]))
    fa.check_status()


# ------------------------------------------------------------------ paddings, wide heads, first calls
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("rows,keys", [([2], [3]), ([300], [3]), ([0], [5]), ([4, 0, 90], [0, 7, 2000])])
def test_long_paddings_are_cleared(rows, keys, d):
    """Many blocks clear one sequence's places."""
    s = Ragged(rows, keys, 2, 2, d, padded=True, lead=2, pad=3, seed=d)
    s.cu_keys = np.cumsum([2] + [6001] * len(rows))
    s.K = int(s.cu_keys[-1]) + 3
    g = torch.Generator().manual_seed(d)
    s.wide_k = torch.full((s.K, 4, d), float("nan"), dtype=torch.bfloat16)
    s.mine_k = (np.arange(s.K) >= 2) & (np.arange(s.K) < s.K - 3)
    for _, _, key0, _, length in s.sequences():
        s.wide_k[key0:key0 + length] = torch.randn(length, 4, d, generator=g).bfloat16()
    check(s)


def test_many_padded_sequences_are_cleared():
    """Each block clears several sequences' places."""
    rng = np.random.default_rng(5)
    rows, keys = rng.integers(0, 6, 500).tolist(), rng.integers(0, 40, 500).tolist()
    check(Ragged(rows, keys, 1, 2, 32, padded=True, pad=4, seed=5))


@pytest.mark.parametrize("d", [32, 256])
def test_same_inputs_give_the_same_bits_captured_or_not(d):
    s = Ragged([700, 81, 3], [500, 1700, 900], 2, 4, d, seed=22, padded=True)
    tensors, batch = s.tensors(), s.batch()
    q, dout, k, v = tensors
    o, lse = forward(s, tensors=tensors)
    grads = backward(s, o, lse, tensors=tensors)
    ws = fa.cross_backward_workspace(q, k, 3)
    out = [torch.empty_like(t) for t in (q, k, v)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]  # with one workspace
    for graph in graphs:
        with torch.cuda.graph(graph):
            fa.cross_backward(q, k, v, o, lse, dout, *batch, out=out, workspace=ws)
    for graph in graphs * 2:
        ws.fill_(255)
        for t, x in zip(out, grads):
            t.copy_(torch.full_like(t, 7.0))
        graph.replay()
        fa.check_status()
        assert all(torch.equal(a, b) for a, b in zip(out, grads))


def test_first_calls_may_be_captured():
    """Kernels' attributes and cluster sizes are set by a first call of theirs; it may be a captured one (the device's own state is made
    by the process' first call of any, which may not: include/fa_gb300.h)."""
    import subprocess
    import sys

    code = """
import torch
import tiled_attention_fwd_gb300 as fa
i32 = dict(dtype=torch.int32, device="cuda")
pool = fa.PagePool.full(40, 16)
table, lens, new = torch.full((3, 8), -1, **i32), torch.zeros(3, **i32), torch.tensor([5, 0, 33], **i32)
done = torch.tensor([False, True, True], device="cuda")
out = torch.zeros(4, **i32), torch.full((38,), -1, dtype=torch.int64, device="cuda"), torch.full((38,), -1, **i32)
cu = torch.tensor([0, 5, 40], **i32)
q, k = (torch.randn(40, 4, d, device="cuda").bfloat16() for d in (64, 64))
o, dq, dk, dv = (torch.empty_like(q) for _ in range(4))
lse = torch.empty(4, 40, device="cuda")
ws, wsb = fa.cross_workspace(k), fa.cross_backward_workspace(q, k, 2)
fa.check_status()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    fa.paged_extend(pool, table, lens, new, out=out)
    fa.paged_release(pool, table, lens, done)
    fa.cross_forward(q, k, k, cu, cu, out=o, lse=lse, workspace=ws)
    fa.cross_backward(q, k, k, o, lse, o, cu, cu, out=(dq, dk, dv), workspace=wsb)
graph.replay()
fa.check_status()
assert lens.tolist() == [5, 0, 0] and out[0].tolist() == [0, 5, 5, 38] and pool.free_count.tolist() == [39]
x, l = fa.cross_forward(q, k, k, cu, cu)
assert torch.equal(o, x) and torch.equal(lse, l)
assert all(torch.equal(a, b) for a, b in zip((dq, dk, dv), fa.cross_backward(q, k, k, o, lse, o, cu, cu)))
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300, cwd=str(__import__("pathlib").Path(__file__).parent.parent))


# ------------------------------------------------------------------ heads in pairs (d <= 64)
@pytest.mark.parametrize("d", [32, 64])
@pytest.mark.parametrize("heads,group", [(2, 1), (3, 1), (5, 3), (3, 32), (7, 5)])
def test_heads_in_pairs_and_the_odd_one(heads, group, d):
    s = Ragged([40, 1, 0, 150, 17, 3], [100, 333, 50, 129, 0, 64], heads, group, d, padded=True, fused=True, lead=2, pad=3, seed=heads)
    o, lse = forward(s)
    check_forward(s, o, lse)


@pytest.mark.parametrize("rows,keys", [([1, 20], [20000, 9001]), ([130], [9001]), ([3001], [200])])
def test_pairs_that_are_split_and_joined(rows, keys):
    s = Ragged(rows, keys, 3, 2, 64, seed=rows[0])
    o, lse = forward(s)
    check_forward(s, o, lse)
    for _ in range(2):
        again = forward(s)
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)


def test_pairs_leave_and_report_what_is_not_there():
    s = Ragged([18, 40, 2], [70, 90, 33], 3, 1, 64, seed=4)
    q, _, k, v = s.tensors()
    cu_rows, cu_keys, _ = s.batch()
    o = torch.full((s.T, 3, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((3, s.T), 7.0, device="cuda")
    fa.cross_forward(q, k, v, cu_rows, cu_keys, max_rows=39, out=o, lse=lse)
    with pytest.raises(fa.FAError):
        fa.check_status()
    want, want_lse = forward(s)
    mine = torch.ones(s.T, dtype=torch.bool, device="cuda")
    mine[18:58] = False
    assert torch.equal(o[mine], want[mine]) and torch.equal(lse[:, mine], want_lse[:, mine])
    assert (o[~mine] == 7.0).all() and (lse[:, ~mine] == 7.0).all()
    bad = cu_keys.clone()
    bad[-1] = s.K + 1
    fa.cross_forward(q, k, v, cu_rows, bad, max_rows=40, out=o, lse=lse)
    with pytest.raises(fa.FAError):
        fa.check_status()
    assert torch.equal(o[:58], want[:58]) and (o[58:] == 0).all() and torch.isneginf(lse[:, 58:]).all()
