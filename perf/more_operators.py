"""Cases of two kinds of operators on ragged batches whose lengths are held on the GPU.

Cross attention of a decoder's rows to an encoder's states, and its gradient.  Sequence b has the rows
cu_rows[b] .. cu_rows[b + 1] of q [rows, Hq, d] and the places cu_keys[b] .. cu_keys[b + 1] of k and v [keys, Hkv, d], of which
the first key_lens[b] are keys: all of them in a packed batch, fewer in a padded one, whose other places hold anything (NaN
here).  Every row sees every key of its sequence; a sequence without keys has o = 0, lse = -inf and no gradient.

The tables of the paged key/value cache: extending requests by new tokens (pages taken from a stack of free ones, row offsets,
each new token's slot and position) and releasing the pages of requests that are done.
"""
import math

import torch

own = False


def _cross(name, op, B, rows, keys, Hq, Hkv, d, padded=False, fused=False, pad=0, holes=0):
    return {"name": name, "op": op, "B": B, "n_lo": rows[0], "n_hi": rows[1], "k_lo": keys[0], "k_hi": keys[1], "Hq": Hq,
            "Hkv": Hkv, "d": d, "padded": padded, "fused": fused, "pad": pad, "holes": holes}


def _pages(name, op, B, ctx, new, page, done=0, pad=0):
    return {"name": name, "op": op, "B": B, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "n_lo": new[0], "n_hi": new[1], "page": page,
            "done": done, "pad": pad}


def listed():
    return [
        # One sequence's next token over a short encoding: the smallest call, where latency is all.
        _cross("cross_step_small", "forward", 1, (1, 1), (333, 333), 16, 16, 64),
        # A serving step: one to five hypotheses a sequence, grouped heads, a padded batch of encodings: bound by reading them.
        _cross("cross_step", "forward", 64, (1, 5), (512, 4096), 32, 8, 128, padded=True, fused=True),
        # A batch of ordinary sentences, every head with keys of its own.
        _cross("cross_batch", "forward", 32, (17, 200), (100, 1024), 16, 16, 64, pad=3),
        # Long targets over long encodings: bound by the tensor cores.
        _cross("cross_long", "forward", 4, (1024, 4096), (2048, 8192), 16, 4, 128),
        # Gradients: a few short sequences, some of them without an encoding.
        _cross("grad_small", "backward", 5, (5, 64), (33, 300), 8, 8, 64, holes=4),
        # A training batch of ordinary sentences, padded encodings.
        _cross("grad_batch", "backward", 32, (17, 200), (100, 1024), 16, 16, 64, padded=True, pad=3),
        # Long targets over long encodings; shared heads.
        _cross("grad_long", "backward", 4, (1024, 4096), (2048, 8192), 16, 4, 128, fused=True),
        # Wide heads.
        _cross("grad_wide", "backward", 6, (100, 700), (256, 2048), 8, 2, 256),
        # A serving step of a full batch: a token each, few of them on a new page.
        _pages("extend_step", "extend", 256, (1, 8192), (1, 1), 16),
        # Prompts arrive: thousands of pages and 200 thousand slots.
        _pages("extend_prompts", "extend", 48, (0, 0), (333, 8192), 32, pad=5),
        # The few requests of a batch that are done give their pages back.
        _pages("release_few", "release", 256, (1, 8192), (0, 0), 16, done=17),
        # Every request ends.
        _pages("release_all", "release", 128, (1000, 32768), (0, 0), 16, done=1),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _range(rng, lo, hi, ratio):
    top = _log_int(rng, lo, hi)
    return _log_int(rng, max(lo, top // ratio), top), top


def draw(rng):
    most = {k: max(_cost(c) for c in listed() if (c["op"] in ("forward", "backward")) == k) for k in (True, False)}
    while True:
        op = rng.choice(["forward", "forward", "forward", "backward", "backward", "backward", "extend", "release"])
        if op in ("forward", "backward"):
            step = op == "forward" and rng.random() < 0.4
            rows = (1, rng.choice([1, 1, 2, 5, 8])) if step else _range(rng, 2, 4096, 8)
            Hkv = rng.choice([1, 2, 3, 4, 8, 16])
            c = _cross("drawn", op, _log_int(rng, 1, 128 if step else 48), rows, _range(rng, 1, 16384 if step else 8192, 8),
                       Hkv * rng.choice([1, 1, 2, 3, 4, 8]), Hkv, rng.choice([32, 64, 64, 128, 128, 256]),
                       padded=rng.random() < 0.4, fused=rng.random() < 0.4, pad=rng.choice([0, 0, 3, 11]),
                       holes=rng.choice([0, 0, 2, 5]))
            scores = c["B"] * c["Hq"] * c["n_hi"] * c["k_hi"]
            held = c["B"] * max(c["k_hi"] * c["Hkv"], c["n_hi"] * c["Hq"]) * c["d"]
            if _cost(c) > most[True] or scores > 2 ** 31 or held > 2 ** 30 or c["Hq"] > 64:
                continue
        else:
            prompts = op == "extend" and rng.random() < 0.5
            new = (0, 0) if op == "release" else _range(rng, 1, 8192, 16) if prompts else (rng.choice([0, 1]), rng.choice([1, 1, 4]))
            c = _pages("drawn", op, _log_int(rng, 1, 64 if prompts else 1024),
                       rng.choice([(0, 0), (0, 700)]) if prompts else _range(rng, 1, 32768, 16), new,
                       rng.choice([16, 16, 32, 64, 128, 256]), done=rng.choice([1, 2, 5, 17]) if op == "release" else 0,
                       pad=rng.choice([0, 0, 5]))
            if _cost(c) > most[False]:
                continue
        del c["name"]
        return c


def _spread(b, lo, hi, turn):
    return hi if b == 0 else lo + int(round((hi - lo) * (((b + 1) * turn) % 1.0)))


def _rows(c):
    return [_spread(b, c["n_lo"], c["n_hi"], 0.7548776662) for b in range(c["B"])]


def _keys(c):
    return [0 if c["holes"] and b % c["holes"] == 1 else _spread(b, c["k_lo"], c["k_hi"], 0.6180339887) for b in range(c["B"])]


def _ctx(c):
    return [_spread(b, c["ctx_lo"], c["ctx_hi"], 0.6180339887) for b in range(c["B"])]


def _done(c):
    return [b % c["done"] == 0 for b in range(c["B"])]


def work(case):
    c = case
    if c["op"] in ("forward", "backward"):
        rows, keys = _rows(c), _keys(c)
        pairs, T, K = sum(n * k for n, k in zip(rows, keys)), sum(rows), sum(keys)
        if c["op"] == "forward":  # q, o and lse; k and v; two products
            return {"bytes": T * c["Hq"] * (4 * c["d"] + 4) + 4 * K * c["Hkv"] * c["d"], "flops": 4 * c["d"] * c["Hq"] * pairs}
        # q, o, dO, dq and lse; k, v, dk and dv; five products
        return {"bytes": T * c["Hq"] * (8 * c["d"] + 4) + 8 * K * c["Hkv"] * c["d"], "flops": 10 * c["d"] * c["Hq"] * pairs}
    ps, lens = c["page"], _ctx(c)
    if c["op"] == "extend":
        # Lengths and counts, both ways; new pages off the stack and into the table; slots and positions, and their pages.
        new = _rows(c)
        fresh = sum(-(-(a + n) // ps) - -(-a // ps) for a, n in zip(lens, new))
        seen = sum(-(-(a + n) // ps) - a // ps for a, n in zip(lens, new) if n)
        return {"bytes": 16 * c["B"] + 8 * fresh + 4 * seen + 12 * sum(new), "flops": 0}
    # Marks and lengths; pages out of the table, onto the stack, and the table's entries marked.
    return {"bytes": 9 * c["B"] + 12 * sum(-(-a // ps) for a, d in zip(lens, _done(c)) if d), "flops": 0}


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


def _offsets(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def _prepare_cross(c, g, dev):
    rows, keys = _rows(c), _keys(c)
    places = [max(keys + [1])] * c["B"] if c["padded"] else keys
    cu_rows, cu_keys = _offsets(rows), _offsets(places)
    T, K, Hq, Hkv, d = cu_rows[-1] + c["pad"], cu_keys[-1] + c["pad"], c["Hq"], c["Hkv"], c["d"]
    i32 = {"dtype": torch.int32, "device": dev}
    s = {"case": dict(c), "cu_rows": torch.tensor(cu_rows, **i32), "cu_keys": torch.tensor(cu_keys, **i32),
         "key_lens": torch.tensor(keys, **i32) if c["padded"] else None, "T": cu_rows[-1], "K": cu_keys[-1],
         "max_rows": max(rows), "max_places": max(places)}
    # Keys have channels that are larger than others; states differ in size.  Both are views of one projection, or apart.
    wide = torch.randn(K, 2 * Hkv, d, generator=g, device=dev)
    wide *= torch.exp(0.5 * torch.randn(1, 2 * Hkv, d, generator=g, device=dev))
    wide *= torch.exp(0.3 * torch.randn(K, 2 * Hkv, 1, generator=g, device=dev))
    wide = wide.bfloat16()
    place = torch.arange(K, device=dev, dtype=torch.int32)
    b = torch.searchsorted(s["cu_keys"][1:].contiguous(), place, right=True).clamp(max=c["B"] - 1)
    wide[place - s["cu_keys"][b] >= torch.tensor(keys, **i32)[b]] = float("nan")  # padding, and what lies behind the last
    s["k"], s["v"] = (x if c["fused"] else x.contiguous() for x in (wide[:, :Hkv], wide[:, Hkv:]))
    s["q"] = torch.randn(T, Hq, d, generator=g, device=dev, dtype=torch.bfloat16)
    s["o"] = torch.zeros(T, Hq, d, dtype=torch.bfloat16, device=dev)
    s["lse"] = torch.zeros(Hq, T, device=dev)
    if c["op"] == "backward":  # the forward's results, and the gradient that comes down
        _plain_forward(s)
        s["dout"] = torch.randn(T, Hq, d, generator=g, device=dev, dtype=torch.bfloat16)
        s["dq"] = torch.zeros_like(s["q"])
        s["dk"], s["dv"] = (torch.zeros(K, Hkv, d, dtype=torch.bfloat16, device=dev) for _ in range(2))
    return s


def _prepare_pages(c, g, dev):
    lens, ps, B = _ctx(c), c["page"], c["B"]
    new = _rows(c) if c["op"] == "extend" else [0] * B
    held = [-(-a // ps) for a in lens]
    want = [-(-(a + n) // ps) for a, n in zip(lens, new)]
    width, used = max(want + [1]) + 1, sum(held)
    total = sum(want) + 7
    order = torch.randperm(total, generator=g, device=dev).int()
    k = torch.arange(width, device=dev)
    first = torch.tensor(_offsets(held)[:-1], device=dev).view(-1, 1)
    taken = k.view(1, -1) < torch.tensor(held, device=dev).view(-1, 1)
    table = torch.where(taken, order[(first + k).clamp(max=total - 1)], torch.full((), -1, dtype=torch.int32, device=dev))
    i32 = {"dtype": torch.int32, "device": dev}
    # The stack of free pages: the first `count` entries, the last of them taken first.  Behind it: anything.
    stack = torch.cat([order[used:], torch.full((used,), -1, **i32)])
    kept = torch.cat([table.reshape(-1), torch.tensor(lens, **i32), stack, torch.tensor([total - used], **i32)])
    rows = sum(new) + c["pad"]
    s = {"case": dict(c), "kept": kept, "now": kept.clone(), "sizes": [B * width, B, total, 1], "width": width}
    if c["op"] == "extend":
        s |= {"new": torch.tensor(new, **i32), "cu_rows": torch.zeros(B + 1, **i32),
              "slots": torch.full((rows,), -1, dtype=torch.int64, device=dev), "positions": torch.full((rows,), -1, **i32)}
    else:
        s["done"] = torch.tensor(_done(c), device=dev)
    return s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    return (_prepare_cross if case["op"] in ("forward", "backward") else _prepare_pages)(case, g, dev)


# ------------------------------------------------------------------ plain forms
def _batched(s):
    """q's rows as [B, Hkv, rows x group, d] (an index of them and whether they are there), k and v as [B, Hkv, places, d] in 32 bits,
    zeros where no key is."""
    c = s["case"]
    B, Hkv, G, d, n, m = c["B"], c["Hkv"], c["Hq"] // c["Hkv"], c["d"], s["max_rows"], s["max_places"]
    dev = s["q"].device
    i, j = torch.arange(n, device=dev), torch.arange(m, device=dev)
    row = s["cu_rows"][:-1].view(B, 1) + i
    there = row < s["cu_rows"][1:].view(B, 1)
    row = row.clamp(max=s["q"].shape[0] - 1).long()
    there = there.view(B, 1, n, 1).expand(B, 1, n, G).reshape(B, 1, n * G, 1)

    def rows_of(x):
        x = x[row].float().view(B, n, Hkv, G, -1).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, -1)
        return torch.where(there, x, torch.zeros_like(x))

    place = (s["cu_keys"][:-1].view(B, 1) + j).clamp(max=max(s["k"].shape[0] - 1, 0)).long()
    lens = s["cu_keys"][1:] - s["cu_keys"][:-1] if s["key_lens"] is None else s["key_lens"]
    key = (j < lens.view(B, 1)).view(B, 1, m, 1)

    def keys_of(x):
        x = x[place].float().transpose(1, 2) if x.shape[0] else torch.zeros(B, Hkv, m, d, device=dev)
        return torch.where(key, x, torch.zeros_like(x))

    return rows_of, there, keys_of, key


def _ragged(s, x):
    """[B, Hkv, rows x group, e] back to [T, Hq, e]."""
    c = s["case"]
    x = x.view(c["B"], c["Hkv"], s["max_rows"], c["Hq"] // c["Hkv"], -1)
    t = torch.arange(s["T"], device=x.device, dtype=torch.int32)
    b = torch.searchsorted(s["cu_rows"][1:].contiguous(), t, right=True)
    return x[b, :, (t - s["cu_rows"][b]).long()].reshape(s["T"], c["Hq"], -1)


def _ragged_keys(s, x):
    """[B, Hkv, places, d] back to [K, Hkv, d]."""
    t = torch.arange(s["K"], device=x.device, dtype=torch.int32)
    b = torch.searchsorted(s["cu_keys"][1:].contiguous(), t, right=True)
    return x[b, :, (t - s["cu_keys"][b]).long()]


def _plain_forward(s):
    rows_of, _, keys_of, key = _batched(s)
    x = torch.matmul(rows_of(s["q"]), keys_of(s["k"]).transpose(2, 3))
    x *= s["case"]["d"] ** -0.5
    x.masked_fill_(~key.transpose(2, 3), float("-inf"))
    top = x.amax(-1, keepdim=True)
    x -= torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = x.exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, keys_of(s["v"])) / torch.where(total == 0, torch.ones_like(total), total)
    s["o"][:s["T"]] = _ragged(s, o)
    s["lse"][:, :s["T"]] = _ragged(s, top + total.log()).squeeze(-1).t()
    return {"o": s["o"], "lse": s["lse"]}


def _plain_backward(s):
    rows_of, there, keys_of, key = _batched(s)
    scale = s["case"]["d"] ** -0.5
    q, k, v, dout = rows_of(s["q"]), keys_of(s["k"]), keys_of(s["v"]), rows_of(s["dout"])
    lse = rows_of(s["lse"].t().unsqueeze(-1))
    D = (dout * rows_of(s["o"])).sum(-1, keepdim=True)
    p = torch.matmul(q, k.transpose(2, 3))
    p *= scale
    p -= lse
    p.exp_().masked_fill_(~(there & key.transpose(2, 3)), 0.0)
    dv = torch.matmul(p.transpose(2, 3), dout)
    ds = torch.matmul(dout, v.transpose(2, 3))
    ds -= D
    ds *= p
    del p
    s["dq"][:s["T"]] = _ragged(s, torch.matmul(ds, k) * scale)
    s["dk"][:s["K"]] = _ragged_keys(s, torch.matmul(ds.transpose(2, 3), q) * scale)
    s["dv"][:s["K"]] = _ragged_keys(s, dv)
    return {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}


def _tables(s):
    """Table, lengths, stack and count as views of the copy that this pass works on: the scheduler keeps the accepted ones."""
    s["now"].copy_(s["kept"])
    table, lens, stack, count = s["now"].split(s["sizes"])
    return table.view(-1, s["width"]), lens, stack, count


def _plain_extend(s):
    table, lens, stack, count = _tables(s)
    ps, new, width = s["case"]["page"], s["new"].long(), s["width"]
    old = lens.long()
    fits = (old >= 0) & (new >= 0) & (old + new <= width * ps)
    rows = torch.where(fits, new, 0)
    held, want = (old + ps - 1) // ps, (old + rows + ps - 1) // ps
    need = torch.where(fits, want - held, 0)
    upto = need.cumsum(0)
    served = fits & ((need == 0) | (upto <= count)) & (rows.cumsum(0) <= s["slots"].shape[0])
    rows = torch.where(served, rows, 0)
    need = torch.where(served, need, 0)
    cu = torch.cat([torch.zeros_like(rows[:1]), rows.cumsum(0)])
    k = torch.arange(width, device=table.device).view(1, -1)
    fresh = (k >= held.view(-1, 1)) & (k < (held + need).view(-1, 1))
    at = (count - 1).view(1, 1) - ((upto - need).view(-1, 1) + k - held.view(-1, 1))
    table.copy_(torch.where(fresh, stack[at.clamp(0, stack.shape[0] - 1)], table))
    lens += rows.int()
    count -= need.sum().int()
    s["cu_rows"].copy_(cu)
    t = torch.arange(s["slots"].shape[0], device=table.device)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=s["case"]["B"] - 1)
    pos = (old[b] + t - cu[b]).clamp(min=0)
    there = t < cu[-1]
    slot = table[b, (pos // ps).clamp(max=width - 1)].long() * ps + pos % ps
    s["slots"].copy_(torch.where(there, slot, s["slots"]))
    s["positions"].copy_(torch.where(there, pos.int(), s["positions"]))
    return {"table": table, "lens": lens, "stack": stack, "count": count, "cu_rows": s["cu_rows"], "slots": s["slots"],
            "positions": s["positions"]}


def _plain_release(s):
    table, lens, stack, count = _tables(s)
    ps, total = s["case"]["page"], stack.shape[0]
    k = torch.arange(s["width"], device=table.device).view(1, -1)
    given = s["done"].view(-1, 1) & (k < ((lens.long() + ps - 1) // ps).view(-1, 1))
    back = (given & (table >= 0) & (table < total)).view(-1)
    at = torch.where(back, count + back.cumsum(0) - 1, total)  # (the last place: not kept)
    stack.copy_(torch.cat([stack, stack[:1]]).scatter(0, at.clamp(max=total), table.view(-1))[:total])
    count += back.sum().int()
    table.masked_fill_(given, -1)
    lens.masked_fill_(s["done"], 0)
    return {"table": table, "lens": lens, "stack": stack, "count": count}


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"forward": _plain_forward, "backward": _plain_backward, "extend": _plain_extend, "release": _plain_release}[op](s)
    import tiled_attention_fwd_gb300 as fa

    if op == "forward":
        if "workspace" not in s:
            s["workspace"] = fa.cross_workspace(s["k"])
        o, lse = fa.cross_forward(s["q"], s["k"], s["v"], s["cu_rows"], s["cu_keys"], s["key_lens"], max_rows=s["max_rows"],
                                  out=s["o"], lse=s["lse"], workspace=s["workspace"])
        return {"o": o, "lse": lse}
    if op == "backward":
        if "workspace" not in s:
            s["workspace"] = fa.cross_backward_workspace(s["q"], s["k"], s["case"]["B"])
        dq, dk, dv = fa.cross_backward(s["q"], s["k"], s["v"], s["o"], s["lse"], s["dout"], s["cu_rows"], s["cu_keys"],
                                       s["key_lens"], out=(s["dq"], s["dk"], s["dv"]), workspace=s["workspace"])
        return {"dq": dq, "dk": dk, "dv": dv}
    table, lens, stack, count = _tables(s)
    pool = fa.PagePool(stack, count, s["case"]["page"])
    if op == "extend":
        cu, slots, positions = fa.paged_extend(pool, table, lens, s["new"], out=(s["cu_rows"], s["slots"], s["positions"]))
        return {"table": table, "lens": lens, "stack": stack, "count": count, "cu_rows": cu, "slots": slots,
                "positions": positions}
    fa.paged_release(pool, table, lens, s["done"])
    return {"table": table, "lens": lens, "stack": stack, "count": count}


# ------------------------------------------------------------------ definitions, in 64 bits
def _exact_cross(c, s):
    G, scale = c["Hq"] // c["Hkv"], 1.0 / math.sqrt(c["d"])
    out = {n: torch.zeros(s[n].shape, dtype=torch.float64, device=s["q"].device)
           for n in (("o", "lse") if c["op"] == "forward" else ("dq", "dk", "dv"))}
    cu_rows, cu_keys = s["cu_rows"].tolist(), s["cu_keys"].tolist()
    for b, m in enumerate(_keys(c)):
        i, j = slice(cu_rows[b], cu_rows[b + 1]), slice(cu_keys[b], cu_keys[b] + m)
        for h in range(c["Hq"]):
            if m == 0:
                if c["op"] == "forward":
                    out["lse"][h, i] = float("-inf")
                continue
            q, k, v = s["q"][i, h].double(), s["k"][j, h // G].double(), s["v"][j, h // G].double()
            x = q @ k.t() * scale
            if c["op"] == "forward":
                out["lse"][h, i] = torch.logsumexp(x, -1)
                out["o"][i, h] = torch.softmax(x, -1) @ v
                continue
            dout = s["dout"][i, h].double()
            p = torch.exp(x - s["lse"][h, i].double().unsqueeze(-1))
            ds = p * (dout @ v.t() - (dout * s["o"][i, h].double()).sum(-1, keepdim=True))
            out["dq"][i, h] = ds @ k * scale
            out["dk"][j, h // G] += ds.t() @ q * scale
            out["dv"][j, h // G] += p.t() @ dout
    return out


def _exact_pages(c, s):
    B, ps, width = c["B"], c["page"], s["width"]
    at = _offsets(s["sizes"])
    kept = s["kept"].tolist()
    table = [kept[b * width:(b + 1) * width] for b in range(B)]
    lens, stack, count = kept[at[1]:at[2]], kept[at[2]:at[3]], kept[at[3]]
    out = {}
    if c["op"] == "extend":
        slots, positions, cu = s["slots"].tolist(), s["positions"].tolist(), [0]
        for b, n in enumerate(s["new"].tolist()):
            for x in range(n):
                if lens[b] % ps == 0:
                    count -= 1
                    table[b][lens[b] // ps] = stack[count]
                slots[cu[-1] + x] = table[b][lens[b] // ps] * ps + lens[b] % ps
                positions[cu[-1] + x] = lens[b]
                lens[b] += 1
            cu.append(cu[-1] + n)
        out = {"cu_rows": torch.tensor(cu, dtype=torch.int32), "slots": torch.tensor(slots, dtype=torch.int64),
               "positions": torch.tensor(positions, dtype=torch.int32)}
    else:
        for b, done in enumerate(s["done"].tolist()):
            for k in range(-(-lens[b] // ps) if done else 0):
                stack[count] = table[b][k]
                count += 1
                table[b][k] = -1
            lens[b] = 0 if done else lens[b]
    whole = {"table": table, "lens": lens, "stack": stack, "count": [count]}
    return {n: torch.tensor(x, dtype=torch.int32) for n, x in whole.items()} | out


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_cross if case["op"] in ("forward", "backward") else _exact_pages)(case, s)
