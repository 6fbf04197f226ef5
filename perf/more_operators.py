"""Timing cases of the second set of serving operators: rotary positions (alone,
and on the way into the 4-bit cache), the gated feed-forward product with q4tp
weights, the attention weight that cached tokens gather, and the eviction that
goes by it.

``own`` False computes an operator in its plain form (elementary torch
operations in 32 bits, angles in 64, rounded once at the end); True calls the
library.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
BLOCK = 16  # tokens per block of the cache layout


def listed():
    return [
        # One token's query and key heads: the smallest call.
        dict(name="rotary-token", op="rotary", dtype="bf16", tokens=1, heads=40, dim=128, rot=128, layout="half",
             scaling="none", start=1000, gain=1.0),
        # A long prompt's heads, interleaved pairs, far positions on frequencies stretched for them.
        dict(name="rotary-prompt", op="rotary", dtype="f16", tokens=16001, heads=40, dim=128, rot=128,
             layout="interleaved", scaling="ramp", start=100000, gain=1.2),
        # Each of 64 running sequences rotates and stores one new token.
        dict(name="store-step", op="store", dtype="bf16", tokens=64, heads=8, group=4, dim=128, rot=128, layout="half",
             scaling="base", start=3000, gain=1.0, page=64),
        # A prompt, half of the head rotated.
        dict(name="store-prompt", op="store", dtype="bf16", tokens=8001, heads=8, group=4, dim=128, rot=64,
             layout="half", scaling="linear", start=0, gain=1.0, page=64),
        # One token through the gate and up projections: the smallest product.
        dict(name="gated-token", op="gated", dtype="bf16", tokens=1, inner=14336, n=4096, act="silu", bias=False),
        # A batch of single tokens (an odd number of them), with biases and another activation.
        dict(name="gated-batch", op="gated", dtype="f16", tokens=45, inner=14336, n=4096, act="gelu_tanh", bias=True),
        # A long prompt.
        dict(name="gated-prompt", op="gated", dtype="bf16", tokens=4096, inner=14336, n=4096, act="silu", bias=False),
        # A serving batch of unequal contexts, one new token each: what its queries looked at.
        dict(name="weigh-batch", op="weigh", dtype="bf16", seqs=48, q_len=1, longest=16384, heads=8, group=8, dim=128,
             page=64),
        # The last 64 queries of one prompt, small heads, an odd length.
        dict(name="weigh-window", op="weigh", dtype="f16", seqs=1, q_len=64, longest=4001, heads=8, group=4, dim=64,
             page=16),
        # A prompt's chunk over its own cached beginning.
        dict(name="weigh-chunk", op="weigh", dtype="bf16", seqs=2, q_len=2048, longest=8192, heads=8, group=4, dim=128,
             page=64),
        # One sequence cut to a quarter in its own pages.
        dict(name="evict-one", op="evict", dtype="bf16", seqs=1, longest=4096, keep=1024, recent=64, heads=8, dim=128,
             page=64, inplace=True),
        # A batch of unequal contexts cut into fewer pages of their own.
        dict(name="evict-batch", op="evict", dtype="f16", seqs=48, longest=16384, keep=2000, recent=128, heads=8,
             dim=128, page=64, inplace=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "store", "gated", "gated", "weigh", "weigh", "evict", "evict"])
    c = dict(op=op, dtype=rng.choice(["bf16", "f16"]))
    if op == "gated":
        c.update(inner=_log_int(rng, 500, 14336), n=32 * _log_int(rng, 32, 544), bias=rng.random() < 0.5,
                 act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]))
        c["tokens"] = min(_log_int(rng, 1, 4096), (4096 * 14336 * 4096) // (c["inner"] * c["n"]))
        return c
    if op in ("rotary", "store"):
        c["dim"] = rng.choice([64, 128, 256] if op == "store" else [32, 64, 80, 96, 128, 192, 256])
        c["rot"] = 16 * rng.randint(1, c["dim"] // 16) if rng.random() < 0.5 else c["dim"]
        c.update(layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "base", "ramp"]),
                 start=rng.choice([0, 1000, 30000, 1000000]), gain=rng.choice([1.0, 1.0, 0.8, 1.2]))
        if op == "rotary":
            c["heads"] = _log_int(rng, 1, 96)
            c["tokens"] = _log_int(rng, 1, 16001 * 40 * 128 // (c["heads"] * c["dim"]))
            return c
        c.update(heads=rng.choice([1, 2, 4, 5, 8]), group=rng.choice([1, 2, 4, 5, 8, 16]), page=rng.choice([16, 32, 64, 128]))
        most = 8001 * 48 * 128 // (c["heads"] * (c["group"] + 2) * c["dim"])
        c["tokens"] = _log_int(rng, 1, min(most, 16384))
        return c
    c.update(heads=rng.choice([1, 2, 4, 5, 8]), dim=rng.choice([64, 128, 256]), page=rng.choice([16, 32, 64, 128]))
    if op == "evict":
        c["longest"] = _log_int(rng, 16, 32768)
        c["keep"] = min(_log_int(rng, 1, 8192), c["longest"])
        c["recent"] = rng.choice([0, 1, 32, 200])
        c["inplace"] = rng.random() < 0.5
        most = (48 * 16384 * 8 * 128) // (c["longest"] * c["heads"] * c["dim"])
        kept = (48 * 2000 * 8 * 128) // (c["keep"] * c["heads"] * c["dim"])
        c["seqs"] = max(1, min(_log_int(rng, 1, 64), most, kept))
        return c
    c.update(group=rng.choice([1, 2, 4, 5, 8, 16]), q_len=rng.choice([1, 1, 2, 7, 16, 32, 64, 0]))
    if c["q_len"] == 0:
        # Prompt chunks: no more scores than the largest one listed above.
        c["q_len"] = _log_int(rng, 65, 2048)
        c["longest"] = c["q_len"] + _log_int(rng, 1, 8192)
    else:
        c["longest"] = _log_int(rng, c["q_len"], 32768)
    rows = c["heads"] * c["group"] * c["q_len"] * c["longest"]
    most = (48 * 16384 * 8 * 128) // (c["longest"] * c["heads"] * c["dim"])
    c["seqs"] = max(1, min(_log_int(rng, 1, 64), most, (2 * 32 * 2048 * 8192 * 128) // max(1, rows * c["dim"])))
    return c


# ---------------------------------------------------------------- the cases' data


def _lens(case):
    """Context length of each sequence: the longest, and others spread below it."""
    ql = case.get("q_len", 1)
    r = random.Random(case["seqs"] * 1000003 + case["longest"] * 31 + ql)
    lo = max(ql, case["longest"] // 16, 1)
    return [case["longest"]] + [r.randint(lo, max(lo, case["longest"])) for _ in range(case["seqs"] - 1)]


def _frequencies(case):
    """Radians a position of each pair, in 64 bits."""
    rot, base, factor = case["rot"], 10000.0, 8.0
    if case["scaling"] == "base":
        base *= factor ** (rot / (rot - 2))
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    if case["scaling"] == "linear":
        f = [v / factor for v in f]
    if case["scaling"] == "ramp":  # stretched where fewer than 4 turns fit 8192 positions, wholly below one
        w = [min(max((8192 * v / (2 * math.pi) - 1) / 3, 0.0), 1.0) for v in f]
        f = [v * (a + (1 - a) / factor) for v, a in zip(f, w)]
    return f


def _keys(g, n, h, d, dtype):
    """Keys with channels of unequal size and offset, and plain values."""
    size = torch.exp(0.4 * torch.randn(h, d, generator=g, device="cuda"))
    off = 0.5 * torch.randn(h, d, generator=g, device="cuda")
    k = torch.randn(n, h, d, generator=g, device="cuda").mul_(size).add_(off).to(dtype)
    return k, torch.randn(n, h, d, generator=g, device="cuda").to(dtype)


def _paged(g, case, dtype):
    """A filled pool and its table for sequences of up to `longest` tokens."""
    h, d, page = case["heads"], case["dim"], case["page"]
    per = -(-case["longest"] // page)
    out_per = 0 if case.get("inplace", True) else -(-case["keep"] // page)
    pages = case["seqs"] * (per + out_per)
    order = torch.randperm(pages, generator=g, device="cuda")
    table = order[:case["seqs"] * per].view(case["seqs"], per).to(torch.int32).contiguous()
    cache = torch.zeros(pages, h, page * 5 * d // 4, dtype=torch.uint8, device="cuda")
    slots = (table.view(-1, 1).long() * page + torch.arange(page, device="cuda")).reshape(-1)
    k, v = _keys(g, slots.numel(), h, d, dtype)
    _plain_write(cache, k, v, slots, page)
    st = dict(cache=cache, table=table, lens=torch.tensor(_lens(case), dtype=torch.int32, device="cuda"), out_table=None)
    if out_per:
        st["out_table"] = order[case["seqs"] * per:].view(case["seqs"], out_per).to(torch.int32).contiguous()
    return st


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, dtype = case["op"], DT[case["dtype"]]
    st = dict(case=case)
    if op == "gated":
        # Round-to-nearest q4tp weights on the row's own ladder: the gate's rows, then the up projection's.
        t, rows, n = case["tokens"], 2 * case["inner"], case["n"]
        w = 0.015 * torch.randn(rows, n // 32, 32, generator=g, device="cuda")
        amax = w.abs().amax(2) / 7
        lo = torch.log2(amax.amin(1, keepdim=True)).half().float()
        step = ((torch.log2(amax.amax(1, keepdim=True)) - lo) / 31).clamp_min(0).half().float()
        tab = torch.exp2(lo + torch.arange(32, device="cuda") * step).contiguous()
        rung = torch.round((torch.log2(amax) - lo) / step.clamp_min(1e-6)).clamp(0, 31).long()
        q = torch.round(w / torch.gather(tab, 1, rung).unsqueeze(2)).clamp_(-8, 7).to(torch.int16).add_(8)
        nib = (q[..., 0::2] | (q[..., 1::2] << 4)).to(torch.uint8).reshape(-1)
        size = torch.exp(0.5 * torch.randn(n, generator=g, device="cuda"))
        x = torch.randn(t, n, generator=g, device="cuda").mul_(size).to(dtype)
        bias = torch.randn(rows, generator=g, device="cuda").to(dtype) if case["bias"] else None
        st.update(x=x, nib=nib, rungs=rung.to(torch.uint8).reshape(-1).contiguous(), tab=tab, bias=bias)
        return st
    h, d = case["heads"], case["dim"]
    if op in ("rotary", "store"):
        f, t = _frequencies(case), case["tokens"]
        # The library's form of the frequencies: 2^64ths of a turn a position, modulo one turn.
        turns = [(round(v / (2 * math.pi) * 2 ** 64) + 2 ** 63) % 2 ** 64 - 2 ** 63 for v in f]
        st.update(freqs=torch.tensor(f, dtype=torch.float64, device="cuda"),
                  turns=torch.tensor(turns, dtype=torch.int64, device="cuda"))
        if t <= 256:  # one token of each sequence
            st["positions"] = case["start"] + torch.randint(0, 4096, (t,), generator=g, device="cuda")
        else:
            st["positions"] = case["start"] + torch.arange(t, device="cuda")
    if op == "rotary":
        # Query and key heads in front of the values', as one projection gives them.
        qkv = torch.randn(t, h + 2, d, generator=g, device="cuda").to(dtype)
        st["x"] = qkv[:, :h]
        return st
    if op == "store":
        page, hq = case["page"], h * case["group"]
        pages = -(-t // page) + 3
        k, v = _keys(g, t, h, d, dtype)
        q = torch.randn(t, hq, d, generator=g, device="cuda").to(dtype)
        qkv = torch.cat([q, k, v], 1)
        order = torch.randperm(pages, generator=g, device="cuda")
        slots = (order.unsqueeze(1) * page + torch.arange(page, device="cuda")).reshape(-1)[:t].contiguous()
        st.update(q=qkv[:, :hq], k=qkv[:, hq:hq + h], v=qkv[:, hq + h:], slots=slots,
                  cache=torch.zeros(pages, h, page * 5 * d // 4, dtype=torch.uint8, device="cuda"))
        return st
    st.update(_paged(g, case, dtype))
    b, cap = case["seqs"], st["table"].shape[1] * case["page"]
    there = torch.arange(cap, device="cuda") < st["lens"].unsqueeze(1)
    if op == "evict":
        # What some thousand queries left: few heavy tokens, many light ones, some never looked at.
        w = torch.exp(2.5 * torch.randn(b, h, cap, generator=g, device="cuda"))
        w.mul_(torch.rand(b, h, cap, generator=g, device="cuda") > 0.1).mul_(there.unsqueeze(1))
        st["weights"] = w
        to = st["table"] if st["out_table"] is None else st["out_table"]
        at = torch.arange(case["keep"], device="cuda")
        st["slots"] = (to.long()[:, at // case["page"]] * case["page"] + at % case["page"]).reshape(-1).contiguous()
        return st
    ql, hq = case["q_len"], h * case["group"]
    st["q"] = torch.randn(b * ql, hq, d, generator=g, device="cuda").to(dtype)
    st["starts"] = torch.arange(0, b * ql + 1, ql, dtype=torch.int32, device="cuda")
    # As much as an earlier call of the same size left.
    st["weights"] = torch.rand(b, h, cap, generator=g, device="cuda").mul_(there.unsqueeze(1)).mul_(
        (2 * ql * case["group"] / st["lens"]).view(b, 1, 1))
    # What the attention of these queries returned beside its output.
    s = _scores(st)
    st["lse"] = torch.logsumexp(s, -1).permute(0, 3, 1, 2).reshape(b * ql, hq).contiguous()
    return st


# ---------------------------------------------------------------- plain forms


def _regions(cache, page, d):
    """Views of the pool: K codes, K (scale, offset), V codes, V (scale, offset),
    each [pages, heads, blocks, 16, bytes]."""
    b = cache.unflatten(2, (page // BLOCK, BLOCK * 5 * d // 4))
    c, p = BLOCK * d // 2, BLOCK * d // 8
    cut = (0, c, c + p, 2 * c + p, 2 * c + 2 * p)
    return [b[..., cut[i]:cut[i + 1]].unflatten(3, (BLOCK, -1)) for i in range(4)]


def _place(slots, page):
    return slots // page, slice(None), slots % page // BLOCK, slots % BLOCK


def _quantise(x):
    dtype = x.dtype
    g = x.float().unflatten(-1, (-1, 32))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    s = ((hi - lo) * (1.0 / 15.0)).to(dtype).float()
    z = (lo - 16 * s).to(dtype).float()
    bad = ~(torch.isfinite(s) & torch.isfinite(z))
    s, z = s.masked_fill(bad, math.nan), z.masked_fill(bad, math.nan)
    r = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    c = torch.round((g - z) * r).nan_to_num(0.0).clamp(16, 31).sub(16).to(torch.uint8).flatten(-2)
    codes = c[..., 0::2] | (c[..., 1::2] << 4)
    return codes, torch.cat([s, z], -1).to(dtype).flatten(-2).view(torch.uint8)


def _plain_write(cache, k, v, slots, page):
    kc, kp, vc, vp = _regions(cache, page, k.shape[2])
    at = _place(slots, page)
    kc[at], kp[at] = _quantise(k)
    vc[at], vp[at] = _quantise(v)


def _values(codes, params, dtype):
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().unflatten(-1, (-1, 32))
    p = params.contiguous().view(dtype).float().unflatten(-1, (-1, 2))
    return (p[..., 1:] + p[..., :1] * (16 + c)).flatten(-2).to(dtype)


def _plain_read(cache, slots, page, d, dtype):
    kc, kp, vc, vp = _regions(cache, page, d)
    at = _place(slots, page)
    return _values(kc[at], kp[at], dtype), _values(vc[at], vp[at], dtype)


def _plain_act(y, act):
    if act == "relu":
        return y.clamp_min(0)
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    if act == "silu":
        return y / (1 + torch.exp(-y))
    return y


def _plain_rotary(st, x):
    c = st["case"]
    angle = st["positions"].double().unsqueeze(1) * st["freqs"]
    cos = (torch.cos(angle).float() * c["gain"]).unsqueeze(1)
    sin = (torch.sin(angle).float() * c["gain"]).unsqueeze(1)
    r, half = c["rot"], c["rot"] // 2
    f = x.float()
    if c["layout"] == "half":
        a, b = f[..., :half], f[..., half:r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = f[..., 0:r:2], f[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, f[..., r:]], -1).to(x.dtype)


def _plain_gated(st):
    x, tab = st["x"], st["tab"]
    rows, n = tab.shape[0], x.shape[1]
    b = st["nib"].view(rows, n // 32, 16)
    c = torch.stack([b & 15, b >> 4], -1).flatten(-2).float().sub_(8)
    w = c.mul_(torch.gather(tab, 1, st["rungs"].view(rows, -1).long()).unsqueeze(2)).view(rows, n)
    y = x.float() @ w.t()
    if st["bias"] is not None:
        y = y + st["bias"].float()
    gate, up = y[:, :rows // 2], y[:, rows // 2:]
    return (_plain_act(gate, st["case"]["act"]) * up).to(x.dtype)


def _scores(st):
    """Scaled scores [seqs, heads, group, queries, places]; -inf where hidden."""
    c, q = st["case"], st["q"]
    b, ql, h, d, page = c["seqs"], c["q_len"], c["heads"], c["dim"], c["page"]
    kc, kp, _, _ = _regions(st["cache"], page, d)
    t = st["table"].long()
    k = _values(kc[t], kp[t], q.dtype)  # [seqs, pages, heads, blocks, 16, dim]
    k = k.permute(0, 2, 5, 1, 3, 4).reshape(b, h, d, -1).float()
    pos = torch.arange(k.shape[-1], device=q.device)
    last = st["lens"].long().unsqueeze(1) - ql + torch.arange(ql, device=q.device)  # the last place a query sees
    qf = q.view(b, ql, h, c["group"], d).permute(0, 2, 3, 1, 4).reshape(b, h, -1, d).float()
    s = (qf @ k).mul_(1 / math.sqrt(d)).view(b, h, c["group"], ql, -1)
    return s.masked_fill_((pos > last.unsqueeze(2)).view(b, 1, 1, ql, -1), -math.inf)


def _plain_weigh(st):
    c = st["case"]
    lse = st["lse"].view(c["seqs"], c["q_len"], c["heads"], c["group"]).permute(0, 2, 3, 1).unsqueeze(-1)
    return st["weights"].add_(torch.exp(_scores(st).sub_(lse)).sum((2, 3)))


def _plain_evict(st):
    c, w, lens = st["case"], st["weights"], st["lens"].long()
    b, h, cap = w.shape
    keep, page, d = c["keep"], c["page"], c["dim"]
    recent = min(c["recent"], keep)
    pos = torch.arange(cap, device=w.device)
    # The heaviest first, ties by place; the latest before all, places without a token after all.
    rank = torch.where((pos >= lens.view(b, 1, 1) - recent), math.inf, w)
    rank = rank.masked_fill(pos >= lens.view(b, 1, 1), -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]
    # (Short sequences keep all they have.)
    fits = torch.arange(keep, device=w.device).expand(b, h, keep)
    left = lens.view(b, 1, 1).clamp_max(keep)
    kept = torch.sort(torch.where(lens.view(b, 1, 1) > keep, order, fits), dim=-1).values
    there = fits < left
    new = torch.zeros_like(w if st["out_table"] is None else w[..., :st["out_table"].shape[1] * page])
    new[..., :keep] = torch.where(there, torch.gather(w, 2, kept), 0.0)
    to = st["table"] if st["out_table"] is None else st["out_table"]
    bi, hi = torch.arange(b, device=w.device).view(b, 1, 1), torch.arange(h, device=w.device).view(1, h, 1)
    src, dst = st["table"].long()[bi, kept // page], to.long()[bi, fits // page]
    for r in _regions(st["cache"], page, d):
        data = r[src, hi, kept % page // BLOCK, kept % BLOCK]
        at = (dst, hi, fits % page // BLOCK, fits % BLOCK)
        r[at] = torch.where(there.unsqueeze(-1), data, r[at])
    return torch.where(there, kept, -1).int(), lens.clamp_max(keep).int(), new


# ---------------------------------------------------------------- one pass


def run(st):
    c, op = st["case"], st["case"]["op"]
    if not own:
        if op == "rotary":
            return _plain_rotary(st, st["x"])
        if op == "gated":
            return _plain_gated(st)
        if op == "weigh":
            return _plain_weigh(st)
        if op == "store":
            q, k = _plain_rotary(st, st["q"]), _plain_rotary(st, st["k"])
            _plain_write(st["cache"], k, st["v"], st["slots"], c["page"])
            return (q,) + _plain_read(st["cache"], st["slots"], c["page"], c["dim"], DT[c["dtype"]])
        kept = _plain_evict(st)
        return kept + _plain_read(st["cache"], st["slots"], c["page"], c["dim"], DT[c["dtype"]])
    from gptq_post_weight_gb300 import _lib

    if op == "rotary":
        return _lib.rotary(st["x"], st["positions"], st["turns"], layout=c["layout"], gain=c["gain"])
    if op == "gated":
        return _lib.q4tp_gated(st["x"], st["nib"], st["rungs"], st["tab"], bias=st["bias"], act=c["act"])
    if op == "weigh":
        starts = None if c["q_len"] == 1 else st["starts"]
        return _lib.kv4_attention_weights(st["weights"], st["q"], st["lse"], st["cache"], st["table"], st["lens"],
                                          c["page"], q_starts=starts, max_q=c["q_len"])
    if op == "store":
        q = _lib.kv4_write_rotary(st["cache"], st["q"], st["k"], st["v"], st["slots"], c["page"], st["positions"],
                                  st["turns"], layout=c["layout"], gain=c["gain"])
        return (q,) + _lib.kv4_read(st["cache"], st["slots"], c["dim"], c["page"], DT[c["dtype"]])
    kept = _lib.kv4_evict(st["cache"], st["table"], st["lens"], st["weights"], c["keep"], c["page"],
                          recent=c["recent"], out_table=st["out_table"])
    return tuple(kept) + _lib.kv4_read(st["cache"], st["slots"], c["dim"], c["page"], DT[c["dtype"]])


def work(case):
    """Each input read once, each output written once; products counted as two operations."""
    op = case["op"]
    if op == "gated":
        t, r, n = case["tokens"], 2 * case["inner"], case["n"]
        b = r * n // 2 + r * n // 32 + 128 * r + 2 * t * n + t * r + (2 * r if case["bias"] else 0)
        return dict(bytes=b, flops=2.0 * t * r * n)
    h, d = case["heads"], case["dim"]
    if op == "rotary":
        t = case["tokens"]
        return dict(bytes=4 * t * h * d + 8 * t + 4 * case["rot"], flops=3.0 * t * h * case["rot"])
    if op == "store":
        t, hq = case["tokens"], h * case["group"]
        held = 5 * t * h * d // 4
        # rotated and written, then read back
        return dict(bytes=4 * t * hq * d + 8 * t * h * d + 2 * held + 24 * t + 4 * case["rot"],
                    flops=3.0 * t * (hq + h) * case["rot"] + 12.0 * t * h * d)
    lens = _lens(case)
    if op == "evict":
        kept = sum(min(n, case["keep"]) for n in lens) * h
        every = case["seqs"] * h * case["keep"]
        slots = 8 * case["seqs"] * case["keep"]
        cap = -(-(case["longest"] if case["inplace"] else case["keep"]) // case["page"]) * case["page"]
        # weights read, kept tokens moved, their places and weights written; then read back
        return dict(bytes=4 * sum(lens) * h + 5 * kept * d // 2 + 4 * every + 4 * case["seqs"] * h * cap + slots +
                    every * d * 5 // 4 + 4 * every * d, flops=4.0 * every * d)
    ql, hq = case["q_len"], h * case["group"]
    pairs = sum(ln - ql + i + 1 for ln in lens for i in range(ql))
    return dict(bytes=sum(lens) * h * (d * 5 // 8 + 8) + case["seqs"] * ql * hq * (2 * d + 4),
                flops=2.0 * d * hq * pairs)


# ---------------------------------------------------------------- the definitions in 64 bits


def _exact_values(flat, dim, dtype):
    """Keys or values [..., dim] of rows of code bytes followed by their parameters, in 64 bits."""
    codes = flat[..., :dim // 2].to(torch.int64)
    par = flat[..., dim // 2:].contiguous().view(dtype).double()
    out = torch.empty(*flat.shape[:-1], dim, dtype=torch.float64, device=flat.device)
    out[..., 0::2] = (codes % 16).double()
    out[..., 1::2] = (codes // 16).double()
    scale = par[..., 0::2].repeat_interleave(32, -1)
    offset = par[..., 1::2].repeat_interleave(32, -1)
    return scale * (out + 16) + offset


def _exact_sequence(cache, slots, page, dim, dtype):
    """K and V [tokens, heads, dim] of the slots; slots [tokens] or [tokens, heads]."""
    c, p = 8 * dim, 2 * dim
    s = slots.reshape(len(slots), -1).expand(-1, cache.shape[1])
    off = s % page
    raw = cache.view(cache.shape[0], cache.shape[1], page // 16, 20 * dim)
    raw = raw[s // page, torch.arange(cache.shape[1], device=cache.device), off // 16]  # [tokens, heads, block bytes]
    row = (off % 16).unsqueeze(-1)
    half, eighth = torch.arange(dim // 2, device=cache.device), torch.arange(dim // 8, device=cache.device)
    got = []
    for base in (0, c + p):
        at = torch.cat([base + row * (dim // 2) + half, base + c + row * (dim // 8) + eighth], -1)
        got.append(_exact_values(torch.gather(raw, 2, at), dim, dtype))
    return got


def _exact_round_trip(x, dtype):
    g = x.double().view(*x.shape[:-1], -1, 32)
    lo, hi = g.min(-1, keepdim=True)[0], g.max(-1, keepdim=True)[0]
    s = ((hi - lo) / 15).to(dtype).double()
    z = (lo - 16 * s).to(dtype).double()
    c = torch.round((g - z) / s).clamp(16, 31)
    return torch.where(s > 0, z + s * c, z + 16 * s).view(x.shape)


def _exact_rotary(st, x):
    c = st["case"]
    r = c["rot"]
    angle = st["positions"].double()[:, None, None] * st["freqs"]
    turn = torch.polar(torch.full_like(angle, c["gain"]), angle)
    y = x.double().clone()
    i, j = (slice(0, r // 2), slice(r // 2, r)) if c["layout"] == "half" else (slice(0, r, 2), slice(1, r, 2))
    z = torch.complex(y[..., i].contiguous(), y[..., j].contiguous()) * turn
    y[..., i], y[..., j] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    op, dtype = case["op"], DT[case["dtype"]]
    if op == "gated":
        rows, n = 2 * case["inner"], case["n"]
        out = []
        for lo in (0, rows // 2):  # the gate's rows, the up projection's
            b = st["nib"].view(rows, n // 2)[lo:lo + rows // 2]
            w = torch.empty(rows // 2, n, dtype=torch.float64, device="cuda")
            w[:, 0::2] = (b % 16).double() - 8
            w[:, 1::2] = (b // 16).double() - 8
            lane = torch.arange(lo, lo + rows // 2, device="cuda").unsqueeze(1)
            w *= st["tab"].double()[lane, st["rungs"].view(rows, -1)[lo:lo + rows // 2].long()].repeat_interleave(32, 1)
            y = st["x"].double() @ w.t()
            out.append(y + (st["bias"].double()[lo:lo + rows // 2] if case["bias"] else 0))
        y, a = out[0], case["act"]
        if a == "relu":
            y = torch.where(y > 0, y, 0.0)
        elif a == "gelu":
            y = y * torch.special.ndtr(y)
        elif a == "gelu_tanh":
            y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
        elif a == "silu":
            y = y * torch.sigmoid(y)
        return y * out[1]
    if op == "rotary":
        return _exact_rotary(st, st["x"])
    d, page, h = case["dim"], case["page"], case["heads"]
    if op == "store":
        k = _exact_rotary(st, st["k"]).to(dtype)  # the cache takes keys of its own type
        return _exact_rotary(st, st["q"]), _exact_round_trip(k, dtype), _exact_round_trip(st["v"], dtype)
    if op == "evict":
        keep, b = case["keep"], case["seqs"]
        to = st["table"] if st["out_table"] is None else st["out_table"]
        kept = torch.full((b, h, keep), -1, dtype=torch.int32, device="cuda")
        new = torch.zeros(b, h, to.shape[1] * page, dtype=torch.float64, device="cuda")
        # Places past a sequence's end keep what they held.
        k, v = _exact_sequence(st["cache"], st["slots"], page, d, dtype)
        for i, ln in enumerate(_lens(case)):
            n = min(ln, keep)
            old = max(ln - min(case["recent"], n), 0)  # up to here the weights decide
            p = torch.arange(ln, device="cuda")
            stay = (p >= old).expand(h, ln).clone()
            if n > ln - old:
                key = st["weights"][i, :, :old].double()
                least = torch.topk(key, n - (ln - old), -1).values[:, -1:]
                above = key > least
                tie = key == least
                room = n - (ln - old) - above.sum(-1, keepdim=True)
                stay[:, :old] = above | (tie & (torch.cumsum(tie, -1) <= room))
            place = stay.nonzero()[:, 1].view(h, n)
            kept[i, :, :n] = place.int()
            new[i, :, :n] = torch.gather(st["weights"][i], 1, place).double()
            slots = st["table"][i].long()[place // page] * page + place % page
            k[i * keep:i * keep + n], v[i * keep:i * keep + n] = _exact_sequence(st["cache"], slots.t(), page, d, dtype)
        return kept, st["lens"].clamp(max=keep), new, k, v
    ql, grp = case["q_len"], case["group"]
    out = st["weights"].double()
    for b, ln in enumerate(_lens(case)):
        p = torch.arange(ln, device="cuda")
        slots = st["table"][b].long()[p // page] * page + p % page
        k = _exact_sequence(st["cache"], slots, page, d, dtype)[0].to(dtype).double()
        hide = p.unsqueeze(0) > (ln - ql + torch.arange(ql, device="cuda")).unsqueeze(1)
        for head in range(h * grp):
            s = st["q"][b * ql:(b + 1) * ql, head].double() @ k[:, head // grp].t() / math.sqrt(d)
            s = s - st["lse"][b * ql:(b + 1) * ql, head].double().unsqueeze(1)
            s[hide] = -math.inf
            out[b, head // grp, :ln] += torch.exp(s).sum(0)
    return out
