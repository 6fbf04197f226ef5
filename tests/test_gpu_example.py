"""examples/serve_block.py: the operators together, as a user runs them.

Each step of the block is compared with the 64-bit oracle on what that step
read (which the block hands out), so that the tolerances are the operators'
own.  Products round every weight to T once above 8 tokens (u / 2 of
sum |x w|), sum in f32 and round the result (u |y|, u a whole ulp); for the
attention's bound see test_gpu_kv4.py.
"""
import importlib.util
import os

import numpy as np
import pytest

from oracle import serve
from test_gpu_kv4 import tolerance

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -7  # bfloat16


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_block.py")
    spec = importlib.util.spec_from_file_location("serve_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def product(got, x, q4, act="none", residual=None):
    nib, rungs, tab = (t.cpu().numpy() for t in q4)
    want = serve.linear(x, nib, rungs, tab, None, act, residual)
    w = np.abs(serve.weights(nib, rungs, tab))
    sc = np.abs(serve.weights(np.full_like(nib, 0x99), rungs, tab))
    ax, n = np.abs(x), x.shape[1]
    err = (0.5 * U + n / 32 * 2.0 ** -23) * (ax @ w.T) + 34 * 143 * 2.0 ** -22 * (ax @ sc.T)
    assert (np.abs(host(got) - want) <= U * np.abs(want) + 1.13 * err + 2.0 ** -24).all()


def test_block_steps(lib):
    from gptq_post_weight_gb300 import _lib

    m = example()
    hidden, heads, kv, dim, inner, page, seqs = 256, 4, 2, 64, 512, 16, 3
    g = torch.Generator(device="cuda").manual_seed(3)
    draw = lambda t: torch.randn(t, hidden, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    block = m.Block(hidden, heads, kv, dim, inner, draw(1024))
    pages = m.Pages(seqs, 12, page, "cuda")
    cache = _lib.kv4_cache(seqs * 12, kv, dim, page)
    keys = [np.zeros((0, kv, dim)) for _ in range(seqs)]
    values = [np.zeros((0, kv, dim)) for _ in range(seqs)]
    # A prompt in two chunks (one sequence has nothing in the second), then
    # three single tokens, and two tokens of one sequence among single ones.
    for counts in ([97, 30, 1], [45, 0, 20], [1, 1, 1], [1, 1, 1], [1, 1, 1], [1, 2, 1]):
        x, tr = draw(sum(counts)), {}
        out = block.forward(x, cache, pages, counts, tr)
        _lib.serve_check()
        product(torch.cat([tr["q"], tr["k"], tr["v"]], 1).flatten(1), host(tr["n1"]), block.qkv)
        k, v = serve.round_trip(host(tr["k"]), "bf16"), serve.round_trip(host(tr["v"]), "bf16")
        at = 0
        for b, c in enumerate(counts):
            keys[b], values[b] = np.concatenate([keys[b], k[at:at + c]]), np.concatenate([values[b], v[at:at + c]])
            at += c
        q, lens = host(tr["q"]), [len(x) for x in keys]
        want = serve.attention(q, keys, values, lens, heads // kv, dim ** -0.5, counts)
        tol = tolerance(q, keys, values, lens, heads // kv, dim ** -0.5, counts, "bf16", want)
        assert (np.abs(host(tr["attention"]) - want) <= tol).all()
        a = host(tr["attention"]).reshape(len(q), -1)
        product(tr["y"], a, block.proj, residual=host(x))
        product(tr["u"], host(tr["n2"]), block.up, act="gelu_tanh")
        product(out, host(tr["u"]), block.down, residual=host(tr["y"]))
    assert pages.lens.tolist() == [97 + 45 + 4, 30 + 5, 25]


def test_sequences_do_not_outgrow_their_pages(lib):
    m = example()
    pages = m.Pages(2, 1, 16, "cuda")
    pages.extend([16, 3])
    with pytest.raises(ValueError, match=r"\[0\]"):
        pages.extend([1, 1])
