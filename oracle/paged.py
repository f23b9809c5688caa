"""fp64 NumPy oracle of the paged key/value cache: quantisation of rows to e4m3 with power-of-two scales, the place of
a row's token in the pages, and attention of rows over their sequences' cached tokens, one row at a time."""
from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0
LARGEST_POWER = 120  # 448 * 2^120 is the last power of two times e4m3's largest value below 2^129


def round_e4m3(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 values (ties to even) of |x| <= 448: steps of 2^(floor(log2 |x|) - 3), 2^-9 below 2^-6."""
    _, exp = np.frexp(np.abs(x))
    step = np.ldexp(1.0, np.maximum(exp - 1, -6) - 3)
    return np.rint(x / step) * step


def quantise_rows(x: np.ndarray):
    """(codes as fp64 e4m3 values, scale bytes) of the rows (last axis) of x."""
    rows = x.reshape(-1, x.shape[-1])
    codes = np.zeros(rows.shape)
    byte = np.zeros(rows.shape[0], dtype=np.uint8)
    for i, r in enumerate(rows):
        if not np.isfinite(r).all():
            byte[i] = 255
            continue
        a = float(np.abs(r).max())
        if a == 0.0:
            continue
        e = math.frexp(a)[1] - 10
        while a > E4M3_MAX * 2.0 ** e:
            e += 1
        e = min(max(e, -127), LARGEST_POWER)
        limit = 240.0 if e == LARGEST_POWER else E4M3_MAX
        codes[i] = np.clip(round_e4m3(np.clip(r * 2.0 ** -e, -E4M3_MAX, E4M3_MAX)), -limit, limit)
        byte[i] = e + 127
    return codes.reshape(x.shape), byte.reshape(x.shape[:-1])


def dequantise(codes: np.ndarray, byte: np.ndarray) -> np.ndarray:
    power = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127.0))
    return codes * power[..., None]


def places(page_table, cu_rows, kv_lens, page_size):
    """[(row, sequence, position, page, slot)] of every row that stands for a token."""
    out = []
    for b in range(len(kv_lens)):
        n = int(cu_rows[b + 1]) - int(cu_rows[b])
        for i in range(n):
            pos = int(kv_lens[b]) - n + i
            if pos >= 0:
                out.append((int(cu_rows[b]) + i, b, pos, int(page_table[b][pos // page_size]), pos % page_size))
    return out


def attention(q, k_pages, v_pages, page_table, cu_rows, kv_lens, scale, causal):
    """O [rows, q_heads, d], L [q_heads, rows] and two figures for error bounds: A = sum_j p_j |v_j| (as O) and the
    largest sum_c |q_c k_jc| * scale of the row's visible keys (as L).  k_pages, v_pages: fp64 [num_pages, heads,
    page_size, d].  Rows of no sequence keep NaN."""
    rows, hq, d = q.shape
    heads, ps = k_pages.shape[1], k_pages.shape[2]
    o = np.full(q.shape, np.nan)
    absum = np.full(q.shape, np.nan)
    lse = np.full((hq, rows), np.nan)
    size = np.zeros((hq, rows))
    for b in range(len(kv_lens)):
        lo, hi, length = int(cu_rows[b]), int(cu_rows[b + 1]), int(kv_lens[b])
        pages = [int(page_table[b][p]) for p in range(-(-length // ps))]
        k = k_pages[pages].transpose(1, 0, 2, 3).reshape(heads, -1, d)[:, :length]
        v = v_pages[pages].transpose(1, 0, 2, 3).reshape(heads, -1, d)[:, :length]
        for i in range(hi - lo):
            see = length - (hi - lo) + i + 1 if causal else length
            for h in range(hq):
                g = h // (hq // heads)
                if see <= 0:
                    o[lo + i, h], absum[lo + i, h], lse[h, lo + i] = 0.0, 0.0, -np.inf
                    continue
                s = (k[g, :see] @ q[lo + i, h]) * scale
                m = s.max()
                p = np.exp(s - m)
                total = p.sum()
                o[lo + i, h] = p @ v[g, :see] / total
                absum[lo + i, h] = p @ np.abs(v[g, :see]) / total
                lse[h, lo + i] = m + np.log(total)
                size[h, lo + i] = (np.abs(k[g, :see]) @ np.abs(q[lo + i, h])).max() * scale
    return o, lse, absum, size
