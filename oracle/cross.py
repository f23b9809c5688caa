"""fp64 NumPy oracle of cross attention over ragged batches: sequence b has the rows cu_rows[b] .. cu_rows[b + 1] of q and the
first key_lens[b] of the places cu_keys[b] .. cu_keys[b + 1] of k and v; query head h reads key/value head h // group."""
from __future__ import annotations

import numpy as np


def sequences(cu_rows, cu_keys, key_lens):
    """[(first row, rows, first place, places, keys)]."""
    out = []
    for b in range(len(cu_rows) - 1):
        places = int(cu_keys[b + 1]) - int(cu_keys[b])
        out.append((int(cu_rows[b]), int(cu_rows[b + 1]) - int(cu_rows[b]), int(cu_keys[b]), places,
                    places if key_lens is None else int(key_lens[b])))
    return out


def attention(q, k, v, cu_rows, cu_keys, key_lens, scale):
    """O [rows, q_heads, d] and L [q_heads, rows]; rows of no sequence keep NaN."""
    o = np.full(q.shape, np.nan)
    lse = np.full(q.shape[1::-1], np.nan)
    group = q.shape[1] // k.shape[1]
    for row0, n, key0, _, length in sequences(cu_rows, cu_keys, key_lens):
        i, j = slice(row0, row0 + n), slice(key0, key0 + length)
        for h in range(q.shape[1]):
            if length == 0:
                o[i, h], lse[h, i] = 0.0, -np.inf
                continue
            s = q[i, h] @ k[j, h // group].T * scale
            m = s.max(axis=1, keepdims=True)
            p = np.exp(s - m)
            total = p.sum(axis=1, keepdims=True)
            o[i, h] = p @ v[j, h // group] / total
            lse[h, i] = (m + np.log(total))[:, 0]
    return o, lse


def attention_backward(q, k, v, o, lse, dout, cu_rows, cu_keys, key_lens, scale):
    """dQ, dK, dV from the inputs and the forward's o and lse; NaN for rows and places of no sequence."""
    dq, dk, dv = (np.full(x.shape, np.nan) for x in (q, k, v))
    group = q.shape[1] // k.shape[1]
    for row0, n, key0, places, length in sequences(cu_rows, cu_keys, key_lens):
        i, j = slice(row0, row0 + n), slice(key0, key0 + length)
        dq[i] = 0.0
        dk[key0:key0 + places] = 0.0
        dv[key0:key0 + places] = 0.0
        for h in range(q.shape[1] if length > 0 and n > 0 else 0):
            g = h // group
            p = np.exp(q[i, h] @ k[j, g].T * scale - lse[h, i][:, None])
            dsum = (dout[i, h] * o[i, h]).sum(axis=1, keepdims=True)
            ds = p * (dout[i, h] @ v[j, g].T - dsum)
            dq[i, h] = scale * (ds @ k[j, g])
            dk[j, g] += scale * (ds.T @ q[i, h])
            dv[j, g] += p.T @ dout[i, h]
    return dq, dk, dv
