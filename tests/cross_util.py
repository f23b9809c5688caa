"""Shared helpers of the cross-attention tests: ragged batches and the error bounds.

u = 2^-8 is half a step of bf16 relative to the value.  Of one row i, e_i bounds the relative error of P: the dot product's
and the scaled exponent's fp32 error, (d + 8) 2^-24 times the largest sum_c |q_c k_jc| scale (2 e_S in paged_util's terms, twice
for the exponent of a difference), 2^-22 |L|, and 2^-20 of the exponential and the fp32 sums.
  O, L: as paged_util's.
  dV = sum P dO: P is rounded once (u) and carries e; the sum over rows in fp32 2^-16; dV is rounded once.
     |err| <= sum_i (u + e_i + 2^-16) P_ij |dO_i| + u |dV|.
  dS = P (dP - D): dP and D carry (d + 8) 2^-24 of their sums of magnitudes, w_i at most; dS is rounded once:
     err(dS) <= (u + e_i) |dS| + P w_i.
  dQ = scale dS K, dK = scale sum dS^T Q: err(dS) and 2^-16 |dS| (fp32 sums) times |K| or |Q|, and u of the result.
Parts of a sum that several blocks make are joined in fp32: in the 2^-16.
"""
from __future__ import annotations

import numpy as np
import torch

import oracle.cross as ref
import tiled_attention_fwd_gb300 as fa

U = 2.0 ** -8
F32 = 2.0 ** -24


class Ragged:
    """A batch of random sequences; rows and places of none, and places behind the keys, hold NaN."""

    def __init__(self, rows, keys, heads=2, group=2, d=64, padded=False, fused=False, lead=0, pad=0, seed=0, gain=1.0):
        g = torch.Generator().manual_seed(seed)
        self.rows, self.keys, self.heads, self.group, self.d, self.fused = rows, keys, heads, group, d, fused
        places = [max(keys + [1]) + 3] * len(keys) if padded else keys
        self.cu_rows = np.cumsum([lead] + list(rows))
        self.cu_keys = np.cumsum([lead] + list(places))
        self.key_lens = list(keys) if padded else None
        self.T, self.K = int(self.cu_rows[-1]) + pad, int(self.cu_keys[-1]) + pad
        hq = heads * group
        self.wide_q = (gain * torch.randn(self.T, 2 * hq, d, generator=g)).bfloat16()
        self.wide_k = torch.randn(self.K, 2 * heads, d, generator=g).bfloat16()
        self.mine_q = np.zeros(self.T, dtype=bool)   # rows of sequences
        self.mine_k = np.zeros(self.K, dtype=bool)   # places of sequences
        seen = np.zeros(self.K, dtype=bool)
        for row0, n, key0, m, length in self.sequences():
            self.mine_q[row0:row0 + n] = True
            self.mine_k[key0:key0 + m] = True
            seen[key0:key0 + length] = True
        self.wide_q[torch.from_numpy(~self.mine_q)] = float("nan")
        self.wide_k[torch.from_numpy(~seen)] = float("nan")

    def sequences(self):
        return ref.sequences(self.cu_rows, self.cu_keys, self.key_lens)

    @property
    def host(self):
        """q, dout, k, v (views, bf16, CPU)."""
        hq = self.heads * self.group
        return (self.wide_q[:, :hq], self.wide_q[:, hq:], self.wide_k[:, :self.heads], self.wide_k[:, self.heads:])

    def tensors(self):
        """q, dout, k, v on the device: views into two tensors, or contiguous."""
        if self.fused:
            hq = self.heads * self.group
            wq, wk = self.wide_q.cuda(), self.wide_k.cuda()
            return wq[:, :hq], wq[:, hq:], wk[:, :self.heads], wk[:, self.heads:]
        return tuple(t.contiguous().cuda() for t in self.host)

    def batch(self):
        i32 = dict(dtype=torch.int32, device="cuda")
        return (torch.tensor(self.cu_rows, **i32), torch.tensor(self.cu_keys, **i32),
                None if self.key_lens is None else torch.tensor(self.key_lens, **i32))


def forward(s: Ragged, scale=None, max_rows=None, workspace=None, tensors=None):
    """cross_forward into buffers of 7.0."""
    q, _, k, v = tensors or s.tensors()
    o = torch.full((s.T, s.heads * s.group, s.d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((s.heads * s.group, s.T), 7.0, device="cuda")
    fa.cross_forward(q, k, v, *s.batch(), max_rows=max(s.rows + [0]) if max_rows is None else max_rows, scale=scale, out=o,
                     lse=lse, workspace=workspace)
    fa.check_status()
    return o, lse


def backward(s: Ragged, o, lse, scale=None, workspace=None, tensors=None):
    """cross_backward into buffers of 7.0."""
    q, dout, k, v = tensors or s.tensors()
    out = tuple(torch.full(t.shape, 7.0, dtype=torch.bfloat16, device="cuda") for t in (q, k, v))
    fa.cross_backward(q, k, v, o, lse, dout, *s.batch(), scale=scale, out=out, workspace=workspace)
    fa.check_status()
    return out


def _near(x, y, tol):
    """x is y to within tol; the same NaN and infinities."""
    fine = np.isfinite(y)
    assert np.array_equal(np.isnan(x), np.isnan(y)), (np.isnan(x).sum(), np.isnan(y).sum())
    assert np.array_equal(x[~fine & ~np.isnan(y)], y[~fine & ~np.isnan(y)])
    err = np.abs(x - y)[fine]
    assert (err <= tol[fine]).all(), float((err - tol[fine]).max())


def _heads(s: Ragged, scale):
    """For each sequence with rows and keys and each query head: (row slice, key slice, h, g, S, size)."""
    q, _, k, _ = (t.double().numpy() for t in s.host)
    for row0, n, key0, _, length in s.sequences():
        if n == 0 or length == 0:
            continue
        i, j = slice(row0, row0 + n), slice(key0, key0 + length)
        for h in range(s.heads * s.group):
            g = h // s.group
            size = (np.abs(q[i, h]) @ np.abs(k[j, g]).T).max(axis=1) * scale
            yield i, j, h, g, q[i, h] @ k[j, g].T * scale, size


def check_forward(s: Ragged, o, lse, scale=None):
    scale = s.d ** -0.5 if scale is None else scale
    q, _, k, v = (t.double().numpy() for t in s.host)
    o, lse = o.cpu().double().numpy(), lse.cpu().double().numpy()
    assert (o[~s.mine_q] == 7.0).all() and (lse[:, ~s.mine_q] == 7.0).all()
    o_ref, l_ref = ref.attention(q, k, v, s.cu_rows, s.cu_keys, s.key_lens, scale)
    tol_o, tol_l = np.zeros(o_ref.shape), np.zeros(l_ref.shape)
    for i, j, h, g, x, size in _heads(s, scale):
        e = 2 * (s.d + 8) * F32 * size
        with np.errstate(all="ignore"):
            absum = np.exp(x - l_ref[h, i][:, None]) @ np.abs(v[j, g])
        tol_o[i, h] = U * (absum + 2 * np.abs(o_ref[i, h])) + (2.0 ** -16 + e[:, None]) * absum
        tol_l[h, i] = e + x.shape[1] / 16 * F32 + 2.0 ** -21 + 2.0 ** -22 * np.abs(l_ref[h, i])
    _near(o[s.mine_q], o_ref[s.mine_q], tol_o[s.mine_q])
    _near(lse[:, s.mine_q], l_ref[:, s.mine_q], tol_l[:, s.mine_q])


def check_backward(s: Ragged, o, lse, grads, scale=None):
    """`o` and `lse`: what was given to cross_backward."""
    scale = s.d ** -0.5 if scale is None else scale
    q, dout, k, v = (t.double().numpy() for t in s.host)
    o, lse = o.cpu().double().numpy(), lse.cpu().double().numpy()
    got = [t.cpu().double().numpy() for t in grads]
    want = ref.attention_backward(q, k, v, o, lse, dout, s.cu_rows, s.cu_keys, s.key_lens, scale)
    tol = [U * np.abs(w) for w in want]
    for i, j, h, g, x, size in _heads(s, scale):
        with np.errstate(all="ignore"):
            p = np.exp(x - lse[h, i][:, None])
            e = (2 * (s.d + 8) * F32 * size + 2.0 ** -22 * np.abs(lse[h, i]) + 2.0 ** -20)[:, None]
            mag_dp = np.abs(dout[i, h]) @ np.abs(v[j, g]).T
            mag_d = (np.abs(dout[i, h]) * np.abs(o[i, h])).sum(axis=1, keepdims=True)
            ds = np.abs(p * (dout[i, h] @ v[j, g].T - (dout[i, h] * o[i, h]).sum(axis=1, keepdims=True)))
            err = (U + e + 2.0 ** -16) * ds + p * (s.d + 8) * F32 * (mag_dp + mag_d)
            tol[0][i, h] += scale * (err @ np.abs(k[j, g]))
            tol[1][j, g] += scale * (err.T @ np.abs(q[i, h]))
            tol[2][j, g] += (p * (U + e + 2.0 ** -16)).T @ np.abs(dout[i, h])
    for x, y, t, mine in zip(got, want, tol, (s.mine_q, s.mine_k, s.mine_k)):
        assert (x[~mine] == 7.0).all()
        _near(x[mine], y[mine], t[mine])


def check(s: Ragged, scale=None, **kw):
    o, lse = forward(s, scale, **kw)
    check_forward(s, o, lse, scale)
    check_backward(s, o, lse, backward(s, o, lse, scale), scale)
