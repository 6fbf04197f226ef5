"""Timing cases of the serving operators: the product with q4tp weights, the
4-bit key/value cache (written, read back) and the attention over it.

``own`` False computes an operator in its plain form (elementary torch
operations in 32 bits, rounded once at the end); True calls the library.
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
        # One token through a square projection: the smallest product, where the call itself counts.
        dict(name="linear-token-square", op="linear", dtype="bf16", tokens=1, rows=4096, n=4096, act="none",
             bias=True, residual=False),
        # One token through the down projection of the 17408-channel group, added to the residual stream.
        dict(name="linear-token-down", op="linear", dtype="bf16", tokens=1, rows=5120, n=17408, act="none",
             bias=False, residual=True),
        # A batch of single tokens (an odd number of them) through an up projection with its activation.
        dict(name="linear-batch-up", op="linear", dtype="f16", tokens=45, rows=14336, n=4096, act="gelu_tanh",
             bias=True, residual=False),
        # A long prompt through the down projection.
        dict(name="linear-prompt-down", op="linear", dtype="bf16", tokens=4096, rows=5120, n=17408, act="none",
             bias=False, residual=True),
        # Each of 64 running sequences stores one new token; the stored values come back.
        dict(name="cache-step", op="write", dtype="bf16", tokens=64, heads=8, dim=128, page=64),
        # A long prompt is stored and read back in the values the cache holds.
        dict(name="cache-prompt", op="write", dtype="f16", tokens=16001, heads=8, dim=128, page=64),
        # A short context read back, small heads, small pages.
        dict(name="read-short", op="read", dtype="f16", tokens=777, heads=8, dim=64, page=16),
        # A long context read back.
        dict(name="read-long", op="read", dtype="bf16", tokens=131072, heads=8, dim=128, page=64),
        # One sequence, one new token: the smallest attention.
        dict(name="attend-one", op="attend", dtype="bf16", seqs=1, q_len=1, longest=1000, heads=8, group=4, dim=128,
             page=64),
        # A serving batch of unequal contexts, one new token each.
        dict(name="attend-batch", op="attend", dtype="bf16", seqs=48, q_len=1, longest=16384, heads=8, group=8,
             dim=128, page=64),
        # Drafted tokens to verify: five queries a sequence, small heads, an odd longest context.
        dict(name="attend-draft", op="attend", dtype="f16", seqs=16, q_len=5, longest=4001, heads=8, group=4, dim=64,
             page=16),
        # A prompt's next chunk over its own cached beginning.
        dict(name="attend-chunk", op="attend", dtype="bf16", seqs=2, q_len=2048, longest=8192, heads=8, group=4,
             dim=128, page=64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "write", "read", "attend", "attend"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "linear":
        c = dict(op=op, dtype=dtype, rows=_log_int(rng, 1000, 14336), n=32 * _log_int(rng, 32, 544),
                 act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), bias=rng.random() < 0.5,
                 residual=rng.random() < 0.5)
        c["tokens"] = min(_log_int(rng, 1, 4096), (4096 * 5120 * 17408) // (c["rows"] * c["n"]))
        return c
    heads, dim, page = rng.choice([2, 4, 5, 8]), rng.choice([64, 128, 256]), rng.choice([16, 32, 64, 128])
    if op in ("write", "read"):
        most = (16001 if op == "write" else 131072) * 1024
        return dict(op=op, dtype=dtype, tokens=_log_int(rng, 1, most // (heads * dim)), heads=heads, dim=dim,
                    page=page)
    c = dict(op=op, dtype=dtype, heads=heads, group=rng.choice([1, 2, 4, 5, 8, 16]), dim=dim, page=page,
             q_len=rng.choice([1, 1, 1, 2, 3, 7, 16, 0]))
    if c["q_len"] == 0:
        # Prompt chunks: no more scores than the largest chunk listed above.
        c["q_len"] = _log_int(rng, 17, 2048)
        c["longest"] = c["q_len"] + _log_int(rng, 1, 8192)
        rows = heads * c["group"] * c["q_len"] * c["longest"] * dim // 128
        c["seqs"] = max(1, min(_log_int(rng, 1, 8), (2 * 32 * 2048 * 8192) // max(1, rows)))
        return c
    c["longest"] = _log_int(rng, c["q_len"], 32768)
    most = (48 * 16384 * 8 * 128) // (c["longest"] * heads * dim)
    c["seqs"] = max(1, min(_log_int(rng, 1, 64), most))
    return c


# ---------------------------------------------------------------- the cases' data


def _lens(case):
    """Context length of each sequence: the longest, and others spread below it."""
    r = random.Random(case["seqs"] * 1000003 + case["longest"] * 31 + case["q_len"])
    lo = max(case["q_len"], case["longest"] // 16, 1)
    return [case["longest"]] + [r.randint(lo, max(lo, case["longest"])) for _ in range(case["seqs"] - 1)]


def _pages(case):
    if case["op"] == "attend":
        return case["seqs"] * (-(-case["longest"] // case["page"]))
    return -(-case["tokens"] // case["page"]) + 3


def _keys(g, n, case, dtype):
    """Keys with channels of unequal size and offset, and plain values."""
    h, d = case["heads"], case["dim"]
    size = torch.exp(0.4 * torch.randn(h, d, generator=g, device="cuda"))
    off = 0.5 * torch.randn(h, d, generator=g, device="cuda")
    k = torch.randn(n, h, d, generator=g, device="cuda").mul_(size).add_(off).to(dtype)
    v = torch.randn(n, h, d, generator=g, device="cuda").to(dtype)
    return k, v


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dtype = DT[case["dtype"]]
    if case["op"] == "linear":
        t, rows, n = case["tokens"], case["rows"], case["n"]
        # Round-to-nearest q4tp weights on the row's own ladder.
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
        res = torch.randn(t, rows, generator=g, device="cuda").to(dtype) if case["residual"] else None
        return dict(case=case, x=x, nib=nib, rungs=rung.to(torch.uint8).reshape(-1).contiguous(), tab=tab, bias=bias,
                    residual=res)
    h, d, page = case["heads"], case["dim"], case["page"]
    pages = _pages(case)
    cache = torch.zeros(pages, h, page * 5 * d // 4, dtype=torch.uint8, device="cuda")
    order = torch.randperm(pages, generator=g, device="cuda")
    st = dict(case=case, cache=cache)
    if case["op"] == "attend":
        per = pages // case["seqs"]
        table = order.view(case["seqs"], per).to(torch.int32).contiguous()
        slots = (order.unsqueeze(1) * page + torch.arange(page, device="cuda")).reshape(-1)
        k, v = _keys(g, slots.numel(), case, dtype)
        _plain_write(cache, k, v, slots, page)
        lens = _lens(case)
        tq = case["seqs"] * case["q_len"]
        st.update(q=torch.randn(tq, h * case["group"], d, generator=g, device="cuda").to(dtype), table=table,
                  lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                  starts=torch.arange(0, tq + 1, case["q_len"], dtype=torch.int32, device="cuda"))
        return st
    # A prompt's tokens in the order of its pages.
    slots = (order.unsqueeze(1) * page + torch.arange(page, device="cuda")).reshape(-1)[:case["tokens"]].contiguous()
    k, v = _keys(g, case["tokens"], case, dtype)
    if case["op"] == "read":
        _plain_write(cache, k, v, slots, page)
        st.update(slots=slots)
    else:
        st.update(slots=slots, k=k, v=v)
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


def _plain_linear(st):
    x, tab = st["x"], st["tab"]
    rows, n = tab.shape[0], x.shape[1]
    b = st["nib"].view(rows, n // 32, 16)
    c = torch.stack([b & 15, b >> 4], -1).flatten(-2).float().sub_(8)
    w = c.mul_(torch.gather(tab, 1, st["rungs"].view(rows, -1).long()).unsqueeze(2)).view(rows, n)
    y = x.float() @ w.t()
    if st["bias"] is not None:
        y = y + st["bias"].float()
    y = _plain_act(y, st["case"]["act"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(x.dtype)


def _plain_attend(st):
    c, q = st["case"], st["q"]
    b, ql, h, d, page = c["seqs"], c["q_len"], c["heads"], c["dim"], c["page"]
    per = st["table"].shape[1]
    slots = (st["table"].long().unsqueeze(2) * page + torch.arange(page, device=q.device)).reshape(-1)
    k, v = _plain_read(st["cache"], slots, page, d, q.dtype)
    pos = torch.arange(per * page, device=q.device)
    lens = st["lens"].long()
    last = lens.unsqueeze(1) - ql + torch.arange(ql, device=q.device)  # the last position a query sees
    seen = pos <= last.unsqueeze(2)  # [b, ql, L]
    k = k.view(b, per * page, h, d).permute(0, 2, 3, 1).float()
    there = (pos < lens.unsqueeze(1)).view(b, -1, 1, 1)
    v = torch.where(there, v.view(b, per * page, h, d), torch.zeros((), dtype=v.dtype, device=v.device))
    v = v.permute(0, 2, 1, 3).float()
    qf = q.view(b, ql, h, c["group"], d).permute(0, 2, 3, 1, 4).reshape(b, h, -1, d).float()
    s = (qf @ k).mul_(1 / math.sqrt(d)).view(b, h, c["group"], ql, -1)
    s = s.masked_fill_(~seen.view(b, 1, 1, ql, -1), -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp_min(-1e30))
    total = p.sum(-1, keepdim=True)
    o = (p.view(b, h, -1, p.shape[-1]) @ v).view(b, h, c["group"], ql, d) / total.clamp_min(1e-30)
    return o.permute(0, 3, 1, 2, 4).reshape(b * ql, -1, d).to(q.dtype)


# ---------------------------------------------------------------- one pass


def run(st):
    c = st["case"]
    if not own:
        if c["op"] == "linear":
            return _plain_linear(st)
        if c["op"] == "attend":
            return _plain_attend(st)
        if c["op"] == "write":
            _plain_write(st["cache"], st["k"], st["v"], st["slots"], c["page"])
        return _plain_read(st["cache"], st["slots"], c["page"], c["dim"], DT[c["dtype"]])
    from gptq_post_weight_gb300 import _lib

    if c["op"] == "linear":
        return _lib.q4tp_linear(st["x"], st["nib"], st["rungs"], st["tab"], bias=st["bias"], act=c["act"],
                                residual=st["residual"])
    if c["op"] == "attend":
        starts = None if c["q_len"] == 1 else st["starts"]
        return _lib.kv4_attention(st["q"], st["cache"], st["table"], st["lens"], c["page"], q_starts=starts,
                                  max_q=c["q_len"])
    if c["op"] == "write":
        _lib.kv4_write(st["cache"], st["k"], st["v"], st["slots"], c["page"])
    return _lib.kv4_read(st["cache"], st["slots"], c["dim"], c["page"], DT[c["dtype"]])


def work(case):
    """Each input read once, each output written once; products counted as two operations."""
    if case["op"] == "linear":
        t, r, n = case["tokens"], case["rows"], case["n"]
        b = r * n // 2 + r * n // 32 + 128 * r + 2 * t * n + 2 * t * r * (2 if case["residual"] else 1)
        return dict(bytes=b + (2 * r if case["bias"] else 0), flops=2.0 * t * r * n)
    h, d = case["heads"], case["dim"]
    if case["op"] in ("write", "read"):
        held, plain, slots = case["tokens"] * h * d * 5 // 4, 4 * case["tokens"] * h * d, 8 * case["tokens"]
        if case["op"] == "read":
            return dict(bytes=held + plain + slots, flops=4.0 * case["tokens"] * h * d)
        # written, then read back
        return dict(bytes=2 * (held + plain + slots), flops=12.0 * case["tokens"] * h * d)
    lens, ql, hq = _lens(case), case["q_len"], h * case["group"]
    pairs = sum(ln - ql + i + 1 for ln in lens for i in range(ql))
    return dict(bytes=sum(lens) * h * d * 5 // 4 + 4 * case["seqs"] * ql * hq * d, flops=4.0 * d * hq * pairs)


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
    """K and V [tokens, heads, dim] of the slots."""
    c, p = 8 * dim, 2 * dim
    off = slots % page
    raw = cache.view(cache.shape[0], cache.shape[1], page // 16, 20 * dim)
    raw = raw.permute(0, 2, 1, 3)[slots // page, off // 16]  # [tokens, heads, block bytes]
    row = (off % 16).view(-1, 1, 1)
    half, quarter = torch.arange(dim // 2, device=cache.device), torch.arange(dim // 8, device=cache.device)
    got = []
    for base in (0, c + p):
        at = torch.cat([base + row * (dim // 2) + half, base + c + row * (dim // 8) + quarter], -1)
        got.append(_exact_values(torch.gather(raw, 2, at.expand(-1, raw.shape[1], -1)), dim, dtype))
    return got


def _exact_round_trip(x, dtype):
    g = x.double().view(*x.shape[:-1], -1, 32)
    lo, hi = g.min(-1, keepdim=True)[0], g.max(-1, keepdim=True)[0]
    s = ((hi - lo) / 15).to(dtype).double()
    z = (lo - 16 * s).to(dtype).double()
    c = torch.round((g - z) / s).clamp(16, 31)
    return torch.where(s > 0, z + s * c, z + 16 * s).view(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    dtype = DT[case["dtype"]]
    if case["op"] == "linear":
        rows, n = case["rows"], case["n"]
        b = st["nib"].view(rows, n // 2)
        w = torch.empty(rows, n, dtype=torch.float64, device="cuda")
        w[:, 0::2] = (b % 16).double() - 8
        w[:, 1::2] = (b // 16).double() - 8
        lane = torch.arange(rows, device="cuda").unsqueeze(1)
        w *= st["tab"].double()[lane, st["rungs"].view(rows, -1).long()].repeat_interleave(32, 1)
        y = st["x"].double() @ w.t()
        y = y + (st["bias"].double() if case["bias"] else 0)
        a = case["act"]
        if a == "relu":
            y = torch.where(y > 0, y, 0.0)
        elif a == "gelu":
            y = y * torch.special.ndtr(y)
        elif a == "gelu_tanh":
            y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
        elif a == "silu":
            y = y * torch.sigmoid(y)
        return y + (st["residual"].double() if case["residual"] else 0)
    d, page = case["dim"], case["page"]
    if case["op"] == "read":
        return tuple(_exact_sequence(st["cache"], st["slots"], page, d, dtype))
    if case["op"] == "write":
        return _exact_round_trip(st["k"], dtype), _exact_round_trip(st["v"], dtype)
    ql, h, grp = case["q_len"], case["heads"], case["group"]
    out = torch.zeros(case["seqs"] * ql, h * grp, d, dtype=torch.float64, device="cuda")
    for b, ln in enumerate(_lens(case)):
        p = torch.arange(ln, device="cuda")
        slots = st["table"][b].long()[p // page] * page + p % page
        k, v = _exact_sequence(st["cache"], slots, page, d, dtype)
        k, v = k.to(dtype).double(), v.to(dtype).double()  # the cache's values are numbers of its own type
        hide = p.unsqueeze(0) > (ln - ql + torch.arange(ql, device="cuda")).unsqueeze(1)
        for head in range(h * grp):
            s = st["q"][b * ql:(b + 1) * ql, head].double() @ k[:, head // grp].t() / math.sqrt(d)
            s[hide] = -math.inf
            out[b * ql:(b + 1) * ql, head] = torch.softmax(s, -1) @ v[:, head // grp]
    return out
