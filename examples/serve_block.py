"""One transformer block served from 4-bit weights and a 4-bit key/value cache.

The weights are quantised with calibration data (``gram_add``, then
``quantize_group`` per Hessian group), a prompt goes through the block in
chunks and single tokens follow, all through

    q4tp_linear -> kv4_write -> kv4_attention -> q4tp_linear (+ residual)

with paged storage that sequences of unequal length share.

    python examples/serve_block.py [--hidden 4096 --seqs 16 --prompt 2000 --steps 32]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gptq_post_weight_gb300 import _lib  # noqa: E402


def quantize(w, x, lam=0.01):
    """q4tp form (nibbles, rungs, tab) of w [rows, n] under the calibration
    inputs x [tokens, n]."""
    n = w.shape[1]
    h = torch.zeros(n * (n + 1) // 2, dtype=torch.float32, device=w.device)
    _lib.gram_add(h, x.float().contiguous())
    out = _lib.quantize_group(h.div_(x.shape[0]), n, w.float().contiguous(), lam, want_u=False)
    return out["nibbles"], out["rungs"], out["tab"]


class Pages:
    """Which pages of the pool each sequence has, and how many tokens."""

    def __init__(self, seqs, pages_per_seq, page_size, device):
        # Neighbouring pages of a sequence lie apart, as they do after some
        # time of serving.
        self.host = torch.arange(seqs * pages_per_seq, dtype=torch.int32).view(pages_per_seq, seqs).t().contiguous()
        self.table = self.host.to(device)
        self.lens = torch.zeros(seqs, dtype=torch.int64)
        self.page_size = page_size

    def extend(self, counts):
        """Room for counts[b] more tokens of sequence b: (slots of the new
        tokens, lengths, first query row of each sequence), on the device."""
        counts = torch.tensor(counts)
        lens = self.lens + counts
        full = (lens > self.host.shape[1] * self.page_size).nonzero().flatten().tolist()
        if full:
            raise ValueError(f"sequences {full} do not fit their pages")
        starts = F.pad(counts.cumsum(0), (1, 0))
        seq = torch.repeat_interleave(torch.arange(len(counts)), counts)
        at = torch.arange(len(seq)) - starts[seq] + self.lens[seq]
        slots = self.host[seq, at // self.page_size].long() * self.page_size + at % self.page_size
        self.lens = lens
        return (slots.to(self.table.device), lens.int().to(self.table.device), starts.int().to(self.table.device))


class Block:
    """Attention and a GELU network, each behind an RMS norm and added to the
    residual stream.  Weights are random; `calibration` [tokens, hidden] is
    what their Hessians are taken from."""

    def __init__(self, hidden, heads, kv_heads, dim, inner, calibration, seed=0):
        device, dtype = calibration.device, calibration.dtype
        g = torch.Generator(device=device).manual_seed(seed)

        def draw(rows, n):
            return torch.randn(rows, n, generator=g, device=device) * n ** -0.5

        self.heads, self.kv_heads, self.dim, self.hidden, self.dtype = heads, kv_heads, dim, hidden, dtype
        norm = self.norm(calibration)
        w = draw((heads + 2 * kv_heads) * dim, hidden)
        self.qkv = quantize(w, norm)
        # Inputs of the later groups, from the weights before quantisation.
        v = (norm.float() @ w[(heads + kv_heads) * dim:].T).view(-1, kv_heads, 1, dim)
        self.proj = quantize(draw(hidden, heads * dim), v.expand(-1, -1, heads // kv_heads, -1).reshape(len(norm), -1))
        w = draw(inner, hidden)
        self.up = quantize(w, norm)
        self.down = quantize(draw(hidden, inner), F.gelu(norm.float() @ w.T, approximate="tanh"))

    def norm(self, x):
        return F.rms_norm(x.float(), (x.shape[-1],), eps=1e-6).to(x.dtype)

    def forward(self, x, cache, pages, counts, trace=None):
        """x [tokens, hidden]: counts[b] new tokens of each sequence b, in
        order.  Returns the block's output of the same shape; a dict given as
        `trace` receives what each step read and gave."""
        t, h, kv, d = x.shape[0], self.heads, self.kv_heads, self.dim
        slots, lens, starts = pages.extend(counts)
        n1 = self.norm(x)
        qkv = _lib.q4tp_linear(n1, *self.qkv).view(t, h + 2 * kv, d)
        q, k, v = qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:]
        _lib.kv4_write(cache, k, v, slots, pages.page_size)
        one = all(c == 1 for c in counts)
        a = _lib.kv4_attention(q, cache, pages.table, lens, pages.page_size, None if one else starts,
                               max_q=1 if one else max(counts))
        y = _lib.q4tp_linear(a.view(t, h * d), *self.proj, residual=x)
        n2 = self.norm(y)
        u = _lib.q4tp_linear(n2, *self.up, act="gelu_tanh")
        out = _lib.q4tp_linear(u, *self.down, residual=y)
        if trace is not None:
            trace.update(n1=n1, q=q, k=k, v=v, attention=a, y=y, n2=n2, u=u)
        return out


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--inner", type=int, default=14336)
    ap.add_argument("--seqs", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=2000)
    ap.add_argument("--chunk", type=int, default=512)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    device, dim, page = "cuda", a.hidden // a.heads, 64
    g = torch.Generator(device=device).manual_seed(1)
    x = torch.randn(4096, a.hidden, generator=g, device=device).to(torch.bfloat16)
    block = Block(a.hidden, a.heads, a.kv_heads, dim, a.inner, x)
    per_seq = (a.prompt + a.steps + page - 1) // page
    pages = Pages(a.seqs, per_seq, page, device)
    cache = _lib.kv4_cache(a.seqs * per_seq, a.kv_heads, dim, page)

    def timed(counts):
        x = torch.randn(sum(counts), a.hidden, generator=g, device=device).to(torch.bfloat16)
        t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        t0.record()
        block.forward(x, cache, pages, counts)
        t1.record()
        t1.synchronize()
        return t0.elapsed_time(t1)

    timed([1] * a.seqs)  # loads the library's kernels
    pages.lens.zero_()
    chunks = [timed([min(a.chunk, a.prompt - at)] * a.seqs) for at in range(0, a.prompt, a.chunk)]
    steps = [timed([1] * a.seqs) for _ in range(a.steps)]
    _lib.serve_check()
    total = a.seqs * a.prompt
    print(f"prompt: {total} tokens in {len(chunks)} chunks, {sum(chunks):.2f} ms")
    print(f"tokens: {a.steps} steps of {a.seqs}, {1000 * sorted(steps)[len(steps) // 2]:.0f} us a step")
    two = 2 * 2 * a.kv_heads * dim
    print(f"cache: {cache.shape[2] // page * a.kv_heads} bytes a token, {two} in bfloat16")


if __name__ == "__main__":
    main()
