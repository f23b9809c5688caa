"""The paged cache on the GPU with values that a cache may hold and random tokens do not show: scales far apart, NaN codes,
scales near the end of the range, very small queries over very large keys.  Bounds are those of paged_util."""
import numpy as np
import pytest
import torch

import oracle.paged as ref
import tiled_attention_fwd_gb300 as fa
from paged_util import Setup, U, check, run

pytestmark = pytest.mark.gpu

D = (32, 64, 128, 256)


def place(s, b, pos):
    return s.table[b, pos // s.page], pos % s.page


def refresh(s):
    """The oracle's values after codes or scale bytes of s (e4m3) were changed."""
    s.values = [ref.dequantise(c.float().double().numpy(), b.numpy()) for c, b in zip(s.kv, s.scale_bytes)]


# ------------------------------------------------------------------ V's scales
@pytest.mark.parametrize("d", D)
@pytest.mark.parametrize("n,group", [(4, 1), (4, 4), (4, 8), (100, 2)])
@pytest.mark.parametrize("up", [12, 16, 24, 40, 80, 125])
def test_an_unseen_token_of_any_size_leaves_earlier_rows(d, n, group, up):
    """A new token's V is 2^up times the others'; rows before it do not see it."""
    s = Setup([150, 70], [n, 3], heads=2, group=group, d=d, fmt="e4m3", seed=d + up)
    page, slot = place(s, 0, 150 - n // 2)
    byte = s.scale_bytes[1][page, :, slot]
    byte.copy_((byte.int() + up).clamp(max=247).to(torch.uint8))
    refresh(s)
    check(s, *run(s), d ** -0.5, True)


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("light,up", [(20, 24), (45, 32), (60, 40), (64, 64), (90, 95), (120, 110)])
def test_a_visible_token_of_small_weight_and_large_value(d, light, up):
    """One of 300 tokens has a weight of about 2^-light of the others' and a V 2^up times theirs."""
    s = Setup([300], [1], heads=1, group=1, d=d, fmt="e4m3", seed=light)
    q = s.q[0, 0].double().numpy()
    page, slot = place(s, 0, 37)
    codes, byte = ref.quantise_rows(-q / (q @ q) * d ** 0.5 * light * np.log(2.0))
    s.kv[0][page, 0, slot] = torch.from_numpy(codes).float().to(torch.float8_e4m3fn)
    s.scale_bytes[0][page, 0, slot] = int(byte)
    s.scale_bytes[1][page, 0, slot] += up
    refresh(s)
    check(s, *run(s), d ** -0.5, True)


@pytest.mark.parametrize("d", D)
@pytest.mark.parametrize("n,group", [(1, 1), (1, 8), (4, 4), (4, 8)])
@pytest.mark.parametrize("spread", [6, 20, 60, 90])
def test_scales_of_values_that_are_far_apart(d, n, group, spread):
    s = Setup([333, 40], [n, n], heads=2, group=group, d=d, page=32, fmt="e4m3", seed=spread)
    g = torch.Generator().manual_seed(spread + d)
    s.scale_bytes[1] = (127 + torch.randint(-spread, spread + 1, s.scale_bytes[1].shape, generator=g)).to(torch.uint8)
    s.scale_bytes[1][~s.held[:, None, :].expand_as(s.scale_bytes[1])] = 255
    refresh(s)
    check(s, *run(s), d ** -0.5, True)


@pytest.mark.parametrize("n,group", [(1, 4), (4, 2), (4, 8)])
@pytest.mark.parametrize("byte", [0, 20, 70, 200, 240])
@pytest.mark.parametrize("tokens", ["all", "first 200", "last 200"])
def test_values_all_small_or_all_large(n, group, byte, tokens):
    """Whole runs of tokens with tiny (byte 20: 2^-107), zero (0: codes are zeros, too) or huge values."""
    s = Setup([333], [n], heads=2, group=group, d=64, page=16, fmt="e4m3", seed=byte + n)
    for pos in range(333):
        if (tokens == "first 200" and pos >= 200) or (tokens == "last 200" and pos < 133):
            continue
        page, slot = place(s, 0, pos)
        s.scale_bytes[1][page, :, slot] = byte
        if byte == 0:
            s.kv[1][page, :, slot] = 0.0
    refresh(s)
    check(s, *run(s), 0.125, True)


# ------------------------------------------------------------------ logits from the ends of the range
@pytest.mark.parametrize("d", D)
@pytest.mark.parametrize("n,group", [(1, 2), (4, 2), (4, 8), (100, 2)])
@pytest.mark.parametrize("small,large,shrink", [(60, 60, 0), (100, 100, 0), (112, 112, 0), (121, 121, 0), (-60, -60, 0),
                                                (-100, -100, 0), (100, 112, 12), (100, 118, 18)])
def test_small_queries_over_large_keys(d, n, group, small, large, shrink):
    """q is 2^-small, K 2^large and the scale 2^-shrink of the usual: the logits are ordinary, a code's product with the key's
    scale is not."""
    s = Setup([150, 70], [n, 3], heads=2, group=group, d=d, fmt="e4m3", seed=d + n)
    s.wide *= 2.0 ** -small  # (q, k and v rows are views of it)
    b = s.scale_bytes[0]
    s.scale_bytes[0] = torch.where(b == 255, b, (b.int() + large).to(torch.uint8))
    refresh(s)
    scale = d ** -0.5 * 2.0 ** -shrink
    check(s, *run(s, scale=scale), scale, True)


# ------------------------------------------------------------------ parts that count for nothing
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 4, 100])
def test_a_nan_of_negligible_weight_is_a_nan_however_the_keys_are_split(fmt, n):
    """Every row sees a token whose V is NaN and whose weight, like that of its 1600 neighbours, is below 2^-150."""
    s = Setup([9001], [n], heads=1, group=1, d=64, page=64, fmt=fmt, seed=n)
    far = np.zeros(64)
    far[0] = -1000.0
    codes, byte = ref.quantise_rows(far)
    s.q[:, 0, 0] = 4.0  # so these tokens' logits are near -500
    for pos in range(1600):
        page, slot = place(s, 0, pos)
        if fmt == "bf16":
            s.kv[0][page, 0, slot] = torch.from_numpy(far).bfloat16()
        else:
            s.kv[0][page, 0, slot] = torch.from_numpy(codes).float().to(torch.float8_e4m3fn)
            s.scale_bytes[0][page, 0, slot] = int(byte)
    page, slot = place(s, 0, 5)
    if fmt == "bf16":
        s.kv[1][page, 0, slot, 3] = float("nan")
        s.values = [t.double().numpy() for t in s.kv]
    else:
        s.scale_bytes[1][page, 0, slot] = 255
        refresh(s)
    check(s, *run(s), 0.125, True)


# ------------------------------------------------------------------ NaN codes
@pytest.mark.parametrize("d", D)
@pytest.mark.parametrize("n,group", [(1, 2), (4, 2), (4, 8), (100, 2)])
@pytest.mark.parametrize("code", [0x7f, 0xff])
@pytest.mark.parametrize("new", [True, False])
def test_nan_codes_under_a_finite_scale(d, n, group, code, new):
    """A code that is e4m3's NaN, in one column of K or V: NaN for the rows that see it, nothing for the others."""
    s = Setup([150, 70], [n, 3], heads=3, group=group, d=d, fmt="e4m3", seed=d + n)
    page, slot = place(s, 0, 150 - n + n // 2 if new else 21)
    s.kv[0].view(torch.uint8)[page, 1, slot, 3] = code
    s.kv[1].view(torch.uint8)[page, 2, slot, d - 5] = code
    refresh(s)
    check(s, *run(s), d ** -0.5, True)


# ------------------------------------------------------------------ scales beyond bf16's range
@pytest.mark.parametrize("d", D)
@pytest.mark.parametrize("n,group", [(4, 2), (4, 8), (100, 2)])
@pytest.mark.parametrize("byte", [248, 250, 254])
def test_unseen_values_beyond_bf16_leave_earlier_rows(d, n, group, byte):
    """448 times 2^121 and more is no bf16: a token that holds it (not from paged_write) reaches the rows that see it."""
    s = Setup([150, 70], [n, 3], heads=2, group=group, d=d, fmt="e4m3", seed=d + n)
    o_ref, l_ref, absum, size = ref.attention(s.q.double().numpy(), *s.values, s.table, s.cu, s.lens, d ** -0.5, True)
    page, slot = place(s, 0, 149)
    for j in range(2):
        s.kv[j].view(torch.uint8)[page, 1, slot] = 0x7e
        s.scale_bytes[j][page, 1, slot] = byte
    o, lse = (t.cpu().double().numpy() for t in run(s))
    keep = np.r_[0:n - 1, n:n + 3]
    e_s = (d + 8) * 2.0 ** -24 * size
    tol_o = U * (absum + 2 * np.abs(o_ref)) + (2.0 ** -16 + 2 * e_s.T[:, :, None]) * absum
    assert (np.abs(o - o_ref) <= tol_o)[keep].all()
    tol_l = 2 * e_s + 150 / 16 * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -22 * np.abs(l_ref)
    assert (np.abs(lse - l_ref) <= tol_l)[:, keep].all()


# ------------------------------------------------------------------ pools of one page or one head
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("pages,heads", [(1, 1), (1, 2), (5, 1)])
def test_strides_of_one_element_dimensions_are_not_looked_at(fmt, pages, heads):
    """torch may report any stride for a dimension of one element: 7 here, which no row of 16 bytes could have."""
    lens = [64 * pages - 9]
    s = Setup(lens, [3], heads=heads, group=2, d=64, page=64, fmt=fmt, seed=heads, spare=0)
    cache = s.cache()
    odd = [torch.as_strided(t, t.shape, (7 if pages == 1 else t.stride(0), 7 if heads == 1 else t.stride(1), 64, 1))
           for t in (cache.k, cache.v)]
    check(s, *run(s, cache=fa.PagedCache(*odd, cache.k_scale, cache.v_scale)), 0.125, True)


# ------------------------------------------------------------------ one NaN among many rows
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_a_nan_in_one_sequence_leaves_the_others_and_most_of_the_time(fmt):
    """Prompts, one token's V a NaN: the rows of other sequences and heads keep their bits, and the rows that need no
    mending are not searched (that made this call 186 and 68 times as long; 40 leaves room for a busy GPU)."""
    B, n, heads, d, page = 4, 3000, 8, 128, 16
    pages = -(-n // page)
    g = torch.Generator(device="cuda").manual_seed(0)
    table = torch.randperm(B * pages, device="cuda", generator=g).int().view(B, pages)
    cu = torch.arange(B + 1, device="cuda", dtype=torch.int32) * n
    lens = torch.full((B,), n, device="cuda", dtype=torch.int32)
    cache = fa.PagedCache.empty(B * pages, heads, page, d, dtype=torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn)
    q, k, v = (torch.randn(B * n, heads, d, device="cuda", generator=g).bfloat16() for _ in range(3))
    fa.paged_write(cache, k, v, table, cu, lens)
    ws = fa.paged_workspace(cache, B)

    def timed():
        out, times = None, []
        for _ in range(4):
            begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            begin.record()
            out = fa.paged_forward(q, cache, table, cu, lens, max_rows=n, workspace=ws)
            end.record()
            fa.check_status()
            times.append(begin.elapsed_time(end))
        return out, min(times)

    (o, lse), clean = timed()
    at, head = 50, 3  # of sequence 1
    if fmt == "bf16":
        cache.v[int(table[1, at // page]), head, at % page, 7] = float("nan")
    else:
        cache.v_scale[int(table[1, at // page]), head, at % page] = 255
    (o2, lse2), spoiled = timed()
    other = torch.ones(o.shape[:2], dtype=torch.bool, device="cuda")
    other[n:2 * n, head] = False
    assert torch.equal(o2[other], o[other]) and torch.equal(lse2.t()[other], lse.t()[other])
    # (Rows computed again: each side within 2 (d + 8) 2^-24 sum_c |q_c k_c| scale, a sum of about 128 * 0.64 / 11 = 7.)
    assert ((lse2 - lse).abs() <= 4 * (d + 8) * 2.0 ** -24 * 20).all()
    assert torch.isnan(o2[n + at:2 * n, head, 7]).all() and torch.isfinite(o2[n:n + at, head]).all()
    assert ((o2[n:n + at, head].float() - o[n:n + at, head].float()).abs() <= 2.0 ** -6 * (1 + o[n:n + at, head].float().abs())).all()
    assert spoiled <= 40 * clean, (spoiled, clean)
