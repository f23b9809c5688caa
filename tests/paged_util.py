"""Shared helpers of the paged-cache tests: caches and batches of chosen lengths, and the error bounds.

Bounds of one output row against the fp64 oracle on the same (bf16 or dequantised) values.  u = 2^-8 is half a step
of bf16 relative to the value.
  O: P is rounded once to 16 bits (at most u a term, so u * A in all, A = sum p |v|), O once (u |O|), and where the
     largest P's rounding is moved into the normaliser that shifts O by at most u |O| more.  The logits carry the
     fp32 error e_S of the dot product and of the scaled exponent: (d + 8) 2^-24 times the row's largest
     sum_c |q_c k_c| scale, which changes p by e_S relative, O by at most 2 e_S A; the exponential and the fp32 sums
     add 2^-16 A at the lengths tested.
  L: 2 e_S + the sum's relative error (len / 16 additions in a row at most, 2^-24 each, and 2^-21 of the exponential)
     + 2^-22 |L|.
"""
from __future__ import annotations

import numpy as np
import torch

import oracle.paged as ref
import tiled_attention_fwd_gb300 as fa

U = 2.0 ** -8


class Setup:
    """A cache whose pages hold random tokens in shuffled order, everything else NaN, and a batch over it."""

    def __init__(self, lens, rows, heads=2, group=2, d=64, page=16, fmt="bf16", seed=0, pad=0, fused=False,
                 token_major=False, spare=2, spread=0.5):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.rows, self.heads, self.group, self.d, self.page, self.fmt = lens, rows, heads, group, d, page, fmt
        need = [-(-n // page) for n in lens]
        total = sum(need) + spare
        order = torch.randperm(total, generator=g).tolist()
        width = max(need + [1]) + 1
        table = np.full((len(lens), width), -1, dtype=np.int64)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = table
        self.cu = np.concatenate([[0], np.cumsum(rows)])
        self.T = int(self.cu[-1]) + pad
        x = torch.randn(2, total, heads, page, d, generator=g)
        x = x * torch.exp(spread * torch.randn(2, total, heads, page, 1, generator=g))
        x = x.bfloat16()
        held = torch.zeros(total, page, dtype=torch.bool)
        for b, n in enumerate(lens):
            for p in range(n):
                held[table[b, p // page], p % page] = True
        x[:, ~held[:, None, :].expand(total, heads, page)] = float("nan")
        self.held = held
        kv = [x[0], x[1]]
        if fmt == "e4m3":
            codes, byte = zip(*[ref.quantise_rows(t.double().numpy()) for t in kv])
            self.scale_bytes = [torch.from_numpy(b) for b in byte]
            kv = [torch.from_numpy(c).to(torch.float32).to(torch.float8_e4m3fn) for c in codes]
            # An empty slot's codes are NaN as well as its scale.
            for t in kv:
                t.view(torch.uint8)[~held[:, None, :].expand(total, heads, page)] = 0x7f
            self.values = [ref.dequantise(c, b) for c, b in zip(codes, byte)]
        else:
            self.scale_bytes = [None, None]
            self.values = [t.double().numpy() for t in kv]
        self.kv = kv
        self.token_major = token_major
        hq = heads * group
        wide = torch.randn(self.T, hq + 2 * heads, d, generator=g).bfloat16()
        self.q, self.k_new, self.v_new = wide[:, :hq], wide[:, hq:hq + heads], wide[:, hq + heads:]
        self.fused = fused
        self.wide = wide

    def cache(self, kv=None, scales=None):
        kv = [t.cuda() for t in (kv or self.kv)]
        if self.token_major:  # [pages, page_size, heads, d] storage
            kv = [t.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(t.dtype) if t.element_size() == 1
                  else t.transpose(1, 2).contiguous().transpose(1, 2) for t in kv]
        scales = [None if s is None else s.cuda() for s in (scales or self.scale_bytes)]
        return fa.PagedCache(*kv, *scales)

    def batch(self):
        i32 = dict(dtype=torch.int32, device="cuda")
        return (torch.tensor(self.table, **i32), torch.tensor(self.cu, **i32), torch.tensor(self.lens, **i32))

    def tokens(self):
        """q, k, v on the device: views into one tensor, or contiguous."""
        if self.fused:
            w = self.wide.cuda()
            hq = self.heads * self.group
            return w[:, :hq], w[:, hq:hq + self.heads], w[:, hq + self.heads:]
        return tuple(t.contiguous().cuda() for t in (self.q, self.k_new, self.v_new))


def reference(s: Setup, scale, causal, values=None):
    k, v = values or s.values
    return ref.attention(s.q.double().numpy(), k, v, s.table, s.cu, s.lens, scale, causal)


def check(s: Setup, o, lse, scale, causal, values=None):
    """Compare with the oracle; rows behind the last sequence must still hold the 7.0 they were given."""
    o_ref, l_ref, absum, size = reference(s, scale, causal, values)
    o, lse = o.cpu().double().numpy(), lse.cpu().double().numpy()
    T = int(s.cu[-1])
    assert (o[T:] == 7.0).all() and (lse[:, T:] == 7.0).all()
    o, lse, o_ref, l_ref, absum, size = o[:T], lse[:, :T], o_ref[:T], l_ref[:, :T], absum[:T], size[:, :T]
    e_s = (s.d + 8) * 2.0 ** -24 * size
    tol_o = U * (absum + 2 * np.abs(o_ref)) + (2.0 ** -16 + 2 * e_s.T[:, :, None]) * absum
    seen = np.isfinite(l_ref)
    assert np.array_equal(np.isneginf(lse), np.isneginf(l_ref))
    assert np.array_equal(np.isnan(lse), np.isnan(l_ref))
    assert np.array_equal(np.isnan(o), np.isnan(o_ref))
    fine = ~np.isnan(o_ref)
    err = np.abs(o - o_ref)
    assert (err[fine] <= tol_o[fine]).all(), float((err[fine] - tol_o[fine]).max())
    tol_l = 2 * e_s + max(s.lens) / 16 * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -22 * np.abs(np.where(seen, l_ref, 0))
    err = np.abs(lse[seen] - l_ref[seen])
    assert (err <= tol_l[seen]).all(), float((err - tol_l[seen]).max())


def run(s: Setup, causal=True, scale=None, max_rows=None, cache=None, workspace=None):
    """paged_forward into buffers of 7.0; (o, lse)."""
    cache = s.cache() if cache is None else cache
    q = s.tokens()[0]
    o = torch.full((s.T, s.heads * s.group, s.d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((s.heads * s.group, s.T), 7.0, device="cuda")
    fa.paged_forward(q, cache, *s.batch(), max_rows=max(s.rows) if max_rows is None else max_rows, causal=causal,
                     scale=scale, out=o, lse=lse, workspace=workspace)
    fa.check_status()
    return o, lse
