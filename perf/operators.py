"""Cases of the paged key/value cache operators: writing new tokens' K and V into the pages, reading them back, and
attention of a chunk of new tokens (down to a single one) over the pages.

A batch is described the same way to all three.  ``page_table[b]`` names the pages of sequence b in the order of its
positions, ``kv_lens[b]`` counts its tokens (the new ones included) and ``cu_rows[b] .. cu_rows[b + 1]`` are its rows in
the token-major tensors: row cu_rows[b] + i stands for position kv_lens[b] - n_b + i, where n_b is the number of rows.
Pages hold [heads, page_size, d]; in an e4m3 cache a token's row of one head has a power-of-two scale of its own, kept
as its biased exponent in a byte.  Slots that no token has reached yet hold NaN here, and page-table entries behind a
sequence's last page hold -1: neither may be seen in an output.
"""
import math

import torch

own = False

SM_SCALE_D = {32: 32 ** -0.5, 64: 0.125, 128: 128 ** -0.5, 256: 0.0625}


def _case(name, op, fmt, B, ctx, rows, Hq, Hkv, d, page, causal=True, pad=0, fused=False):
    return {"name": name, "op": op, "fmt": fmt, "B": B, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "n_lo": rows[0],
            "n_hi": rows[1], "Hq": Hq, "Hkv": Hkv, "d": d, "page": page, "causal": causal, "pad": pad, "fused": fused}


WHOLE = (0, 0)  # rows of a sequence: all of its tokens


def listed():
    return [
        # One token of each running sequence is appended: a serving step's smallest call, where latency is all.
        _case("write_step_bf16", "write", "bf16", 16, (100, 4096), (1, 1), 16, 8, 128, 16, fused=True),
        # Ragged prompts are quantised into the cache.
        _case("write_prompt_e4m3", "write", "e4m3", 8, (1000, 8192), WHOLE, 16, 8, 128, 32, pad=7, fused=True),
        # Whole prefixes are laid out contiguously again (to be handed on, or for a contiguous kernel).
        _case("read_prefix_bf16", "read", "bf16", 4, (1024, 16384), WHOLE, 16, 8, 128, 16),
        _case("read_prefix_e4m3", "read", "e4m3", 24, (333, 4096), WHOLE, 16, 16, 64, 64, pad=5),
        # One sequence, one token, a short context: the smallest step of attention.
        _case("step_small_bf16", "forward", "bf16", 1, (1024, 1024), (1, 1), 16, 4, 64, 16),
        # A serving batch, one token a sequence, grouped heads: bound by the reading of the cache.
        _case("step_bf16", "forward", "bf16", 64, (1024, 8192), (1, 1), 32, 8, 128, 16, fused=True),
        _case("step_e4m3", "forward", "e4m3", 128, (500, 16384), (1, 1), 32, 4, 128, 64),
        # Two very long sequences: the key axis has to be split over the machine and joined again.
        _case("step_long_bf16", "forward", "bf16", 2, (100001, 131072), (1, 1), 16, 2, 256, 128),
        # A few drafted tokens a sequence, checked in one pass.
        _case("draft_e4m3", "forward", "e4m3", 40, (777, 8192), (2, 8), 32, 8, 128, 32, pad=3),
        # Chunks of long prompts over what is cached of them: bound by the tensor cores.
        _case("chunk_bf16", "forward", "bf16", 4, (4096, 16384), (511, 2048), 16, 4, 128, 32, fused=True),
        _case("chunk_e4m3", "forward", "e4m3", 5, (1024, 8192), (65, 1024), 32, 8, 128, 64, pad=9),
        # Whole prompts, every head with keys of its own.
        _case("prompt_bf16", "forward", "bf16", 4, (1024, 4096), WHOLE, 16, 16, 128, 16),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["write", "read", "forward", "forward", "forward", "forward"])
        kind = rng.choice(["step", "draft", "chunk", "whole"]) if op == "forward" else rng.choice(["step", "whole"])
        hi = _log_int(rng, 16, 131072 if kind == "step" else 16384 if kind in ("draft", "chunk") else 6000)
        lo = _log_int(rng, max(1, hi // 16), hi)
        rows = {"step": (1, 1), "draft": (1, rng.randint(2, 16)), "whole": WHOLE,
                "chunk": (_log_int(rng, 1, 64), _log_int(rng, 64, 2048))}[kind]
        Hkv = rng.choice([1, 2, 4, 5, 8, 16])
        c = _case("drawn", op, rng.choice(["bf16", "e4m3"]), _log_int(rng, 1, 128 if kind == "step" else 32), (lo, hi),
                  rows, Hkv * rng.choice([1, 2, 3, 4, 8]), Hkv, rng.choice([32, 64, 128, 128, 128, 256]),
                  rng.choice([16, 16, 32, 64, 128, 256]), causal=rng.random() < 0.85, pad=rng.choice([0, 0, 3, 11]),
                  fused=rng.random() < 0.4)
        padded = c["B"] * c["Hq"] * max(_rows(c)) * c["ctx_hi"] if op == "forward" else 0
        held = c["B"] * c["ctx_hi"] * Hkv * c["d"]  # values of the cache that the plain form widens
        if _cost(c) <= most and padded <= 2 ** 31 and held <= 2 ** 31 and c["Hq"] <= 64:
            del c["name"]
            return c


def _spread(b, lo, hi, turn):
    return lo + int(round((hi - lo) * (((b + 1) * turn) % 1.0)))


def _lens(c):
    return [c["ctx_hi"] if b == 0 else _spread(b, c["ctx_lo"], c["ctx_hi"], 0.6180339887) for b in range(c["B"])]


def _rows(c):
    lens = _lens(c)
    if c["n_hi"] == 0:
        return lens
    return [min(n, c["n_hi"] if b == 0 else _spread(b, c["n_lo"], c["n_hi"], 0.7548776662)) for b, n in enumerate(lens)]


def work(case):
    c, lens, rows = case, _lens(case), _rows(case)
    row_bytes = c["d"] * 2 if c["fmt"] == "bf16" else c["d"] + 1
    T = sum(rows)
    if c["op"] != "forward":  # K and V: read once, written once
        return {"bytes": 2 * T * c["Hkv"] * (row_bytes + 2 * c["d"]), "flops": 0}
    if c["causal"]:  # row i of n sees len - n + i + 1 keys
        pairs = sum(n * (L - n) + n * (n + 1) // 2 for L, n in zip(lens, rows))
    else:
        pairs = sum(n * L for L, n in zip(lens, rows))
    kv = 2 * sum(lens) * c["Hkv"] * row_bytes
    return {"bytes": kv + T * c["Hq"] * (4 * c["d"] + 4), "flops": 4 * c["d"] * c["Hq"] * pairs}


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


def _quantise(x):
    """Codes and scale bytes of rows of bf16: scale = 2^(byte - 127), the smallest power of two that brings the row's
    largest magnitude to 448 or less (but no larger than 2^120, where codes stop at 240, which keeps every value
    finite); a row that holds an infinity or a NaN has the byte 255 (NaN) and codes 0."""
    x = x.float()
    amax = x.abs().amax(-1)
    fine = torch.isfinite(amax)
    mant, exp = torch.frexp(torch.where(fine, amax, torch.zeros_like(amax)))
    byte = torch.where(amax > 0, exp.int() - 9 + (mant > 0.875).int() + 127, torch.zeros_like(exp.int())).clamp(0, 247)
    inverse = ((254 - byte) << 23).view(torch.float32).unsqueeze(-1)
    most = torch.where(byte == 247, 240.0, 448.0).unsqueeze(-1)
    scaled = torch.where(fine.unsqueeze(-1), x, torch.zeros_like(x)) * inverse
    codes = torch.minimum(torch.maximum(scaled, -most), most).to(torch.float8_e4m3fn)
    return codes, torch.where(fine, byte, torch.full_like(byte, 255)).to(torch.uint8)


def _factor(byte):
    f = (byte.int() << 23).view(torch.float32)
    f = torch.where(byte == 0, torch.full_like(f, 2.0 ** -127), f)
    return torch.where(byte == 255, torch.full_like(f, float("nan")), f)


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    lens, rows = _lens(c), _rows(c)
    B, ps, Hkv, d = c["B"], c["page"], c["Hkv"], c["d"]
    need = [-(-n // ps) for n in lens]
    width = max(need) + 1
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device=dev)
    table = torch.full((B, width), -1, dtype=torch.int32)
    owner, at = [], 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n, dtype=torch.int32)
        owner += [max(0, min(ps, lens[b] - k * ps)) for k in range(n)]
        at += n
    table = table.to(dev)
    table = torch.where(table >= 0, order[table.clamp(min=0).long()].int(), table)
    filled = torch.zeros(pages, dtype=torch.int64, device=dev)
    filled[order[:at]] = torch.tensor(owner, device=dev)
    if c["op"] == "write":  # the new tokens' slots are empty yet
        first = torch.zeros(pages, dtype=torch.int64)
        first[:at] = torch.tensor([max(0, min(ps, lens[b] - rows[b] - k * ps)) for b in range(B) for k in range(need[b])])
        filled[order[:at]] = first[:at].to(dev)
    empty = torch.arange(ps, device=dev).view(1, ps) >= filled.view(pages, 1)
    # Keys have channels that are larger than others, as rotated and projected keys do; tokens differ in size.
    gain = torch.exp(0.5 * torch.randn(2, Hkv, 1, d, generator=g, device=dev))
    kv = []
    for j in range(2):
        x = torch.randn(pages, Hkv, ps, d, generator=g, device=dev, dtype=torch.bfloat16)
        x *= gain[j]
        x *= torch.exp(0.3 * torch.randn(pages, Hkv, ps, 1, generator=g, device=dev))
        kv.append(x)
    scales = [None, None]
    if c["fmt"] == "e4m3":
        kv, scales = zip(*[_quantise(x) for x in kv])
        hole = empty.view(pages, 1, ps).expand(pages, Hkv, ps)
        scales = [torch.where(hole, torch.full_like(s, 255), s) for s in scales]
        kv = [torch.where(hole.unsqueeze(-1), torch.full_like(x.view(torch.uint8), 127), x.view(torch.uint8)).view(x.dtype) for x in kv]
    else:
        kv = [x.masked_fill_(empty.view(pages, 1, ps, 1), float("nan")) for x in kv]
    T, Hq = sum(rows), c["Hq"]
    cu = [0]
    for n in rows:
        cu.append(cu[-1] + n)
    rows_all = T + c["pad"]
    state = {"case": dict(c), "k": kv[0], "v": kv[1], "k_scale": scales[0], "v_scale": scales[1], "table": table,
             "cu": torch.tensor(cu, dtype=torch.int32, device=dev), "lens": torch.tensor(lens, dtype=torch.int32, device=dev),
             "T": T, "max_rows": max(rows)}
    # The rows of q, k and v: contiguous, or views into the output of one fused projection.
    wide = torch.randn(rows_all, Hq + 2 * Hkv, d, generator=g, device=dev, dtype=torch.bfloat16)
    parts = [wide[:, :Hq], wide[:, Hq:Hq + Hkv], wide[:, Hq + Hkv:]]
    q, k_new, v_new = parts if c["fused"] else [x.contiguous() for x in parts]
    if c["op"] == "forward":
        state |= {"q": q, "o": torch.zeros(rows_all, Hq, d, dtype=torch.bfloat16, device=dev),
                  "lse": torch.zeros(Hq, rows_all, device=dev)}
    elif c["op"] == "write":
        state |= {"k_new": k_new, "v_new": v_new}
    else:
        state |= {"k_out": torch.zeros(rows_all, Hkv, d, dtype=torch.bfloat16, device=dev),
                  "v_out": torch.zeros(rows_all, Hkv, d, dtype=torch.bfloat16, device=dev)}
    return state


def _slots(s):
    """Page and slot of each row that stands for a token."""
    t = torch.arange(s["T"], device=s["cu"].device, dtype=torch.int32)
    b = torch.searchsorted(s["cu"][1:].contiguous(), t, right=True)
    i = t - s["cu"][b]
    pos = (s["lens"][b] - (s["cu"][b + 1] - s["cu"][b]) + i).long()
    ps = s["case"]["page"]
    return s["table"][b, pos // ps].long(), pos % ps


def _plain_write(s):
    page, slot = _slots(s)
    for name in ("k", "v"):
        x = s[name + "_new"][:s["T"]]
        if s["case"]["fmt"] == "e4m3":
            codes, byte = _quantise(x)
            s[name].view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
            s[name + "_scale"][page, :, slot] = byte
        else:
            s[name][page, :, slot] = x
    return _cache(s)


def _cache(s):
    return {k: s[k] for k in ("k", "v", "k_scale", "v_scale") if s[k] is not None}


def _plain_read(s):
    page, slot = _slots(s)
    for name in ("k", "v"):
        x = s[name].view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn) if s["case"]["fmt"] == "e4m3" else s[name][page, :, slot]
        if s["case"]["fmt"] == "e4m3":
            x = x.float() * _factor(s[name + "_scale"][page, :, slot]).unsqueeze(-1)
        s[name + "_out"][:s["T"]] = x
    return {"k": s["k_out"], "v": s["v_out"]}


def _gathered(s, name):
    """[B, Hkv, width * page, d] in 32 bits, zeros where no token is."""
    c, at = s["case"], s["table"].clamp(min=0).long()
    if c["fmt"] == "e4m3":
        x = s[name].view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * _factor(s[name + "_scale"][at]).unsqueeze(-1)
    else:
        x = s[name][at].float()
    x = x.transpose(1, 2).reshape(c["B"], c["Hkv"], -1, c["d"])
    seen = torch.arange(x.shape[2], device=x.device).view(1, -1) < s["lens"].view(-1, 1)
    return torch.where(seen.view(c["B"], 1, -1, 1), x, torch.zeros_like(x))


def _plain_forward(s):
    c = s["case"]
    B, Hkv, G, d, n = c["B"], c["Hkv"], c["Hq"] // c["Hkv"], c["d"], s["max_rows"]
    dev = s["q"].device
    k, v = _gathered(s, "k"), _gathered(s, "v")
    count = s["cu"][1:] - s["cu"][:-1]
    i = torch.arange(n, device=dev)
    row = (s["cu"][:-1].view(-1, 1) + i).clamp(max=s["q"].shape[0] - 1).long()
    q = s["q"][row].float().view(B, n, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, d)
    x = torch.matmul(q, k.transpose(2, 3))
    x *= SM_SCALE_D[d]
    j = torch.arange(k.shape[2], device=dev)
    most = (s["lens"] - count).view(-1, 1) + i if c["causal"] else (s["lens"] - 1).view(-1, 1).expand(B, n)
    most = torch.minimum(most, s["lens"].view(-1, 1) - 1)
    hidden = (j.view(1, 1, -1) > most.unsqueeze(-1)).repeat_interleave(G, 1)
    x.masked_fill_(hidden.unsqueeze(1), float("-inf"))
    top = x.amax(-1, keepdim=True)
    x -= torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = x.exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + total.log()).view(B, Hkv, n, G)
    o = o.view(B, Hkv, n, G, d)
    t = torch.arange(s["T"], device=dev, dtype=torch.int32)
    b = torch.searchsorted(s["cu"][1:].contiguous(), t, right=True)
    at = (t - s["cu"][b]).long()
    s["o"][:s["T"]] = o[b, :, at].reshape(s["T"], c["Hq"], d)
    s["lse"][:, :s["T"]] = lse[b, :, at].reshape(s["T"], c["Hq"]).t()
    return {"o": s["o"], "lse": s["lse"]}


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import tiled_attention_fwd_gb300 as fa

        if "cache" not in s:  # the handle that a user's program makes once for its cache
            s["cache"] = fa.PagedCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
            s["workspace"] = fa.paged_workspace(s["cache"], s["case"]["B"])
        if op == "write":
            fa.paged_write(s["cache"], s["k_new"], s["v_new"], s["table"], s["cu"], s["lens"])
            return _cache(s)
        if op == "read":
            k, v = fa.paged_read(s["cache"], s["table"], s["cu"], s["lens"], out=(s["k_out"], s["v_out"]))
            return {"k": k, "v": v}
        o, lse = fa.paged_forward(s["q"], s["cache"], s["table"], s["cu"], s["lens"], max_rows=s["max_rows"],
                                  causal=s["case"]["causal"], out=s["o"], lse=s["lse"], workspace=s["workspace"])
        return {"o": o, "lse": lse}
    return {"write": _plain_write, "read": _plain_read, "forward": _plain_forward}[op](s)


def _e4m3_64(x):
    """x, in 64 bits, rounded to the nearest e4m3 value (ties to the even one), for |x| <= 448."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    """From the definitions, in 64 bits, sequence by sequence and head by head."""
    s = prepare(case, seed)
    c = case
    lens, rows, ps, G = _lens(c), _rows(c), c["page"], c["Hq"] // c["Hkv"]
    table = s["table"].tolist()
    dev = s["k"].device

    def value(name, page):  # [Hkv, page, d]
        x = s[name][page].double()
        if c["fmt"] == "bf16":
            return x
        byte = s[name + "_scale"][page].double()
        two = torch.exp2(byte - 127)
        return x * torch.where(byte == 255, torch.full_like(two, float("nan")), two).unsqueeze(-1)

    start = 0
    if c["op"] == "write":
        out = {}
        for name in ("k", "v"):
            whole = s[name].double()
            start = 0
            for b, (L, n) in enumerate(zip(lens, rows)):
                pos = torch.arange(L - n, L, device=dev)
                page = s["table"][b].long()[pos // ps]
                x = s[name + "_new"][start:start + n].double()
                if c["fmt"] == "e4m3":
                    power = torch.ceil(torch.log2(x.abs().amax(-1) / 448)).clamp(-127, 120)
                    x = _e4m3_64(x / torch.exp2(power).unsqueeze(-1))
                whole[page, :, pos % ps] = x
                start += n
            out[name] = whole
        if c["fmt"] == "e4m3":
            out |= {"k_scale": None, "v_scale": None}
        return out
    if c["op"] == "read":
        out = {name: torch.zeros(s["k_out"].shape, dtype=torch.float64, device=dev) for name in ("k", "v")}
        for b, (L, n) in enumerate(zip(lens, rows)):
            for name in ("k", "v"):
                held = value(name, s["table"][b, :-(-L // ps)].long()).transpose(1, 2).reshape(-1, c["Hkv"], c["d"])
                out[name][start:start + n] = held[L - n:L]
            start += n
        return out
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device=dev)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=dev)
    for b, (L, n) in enumerate(zip(lens, rows)):
        pages = torch.tensor(table[b][:-(-L // ps)], device=dev)
        kb, vb = (value(name, pages).transpose(0, 1).reshape(c["Hkv"], -1, c["d"])[:, :L] for name in ("k", "v"))
        see = torch.arange(L, device=dev).view(1, L) <= (torch.arange(n, device=dev).view(n, 1) + (L - n))
        for h in range(c["Hq"]):
            x = s["q"][start:start + n, h].double() @ kb[h // G].t() / math.sqrt(c["d"])
            if c["causal"]:
                x = torch.where(see, x, torch.full_like(x, float("-inf")))
            lse[h, start:start + n] = torch.logsumexp(x, -1)
            o[start:start + n, h] = torch.softmax(x, -1) @ vb[h // G]
        start += n
    return {"o": o, "lse": lse}
