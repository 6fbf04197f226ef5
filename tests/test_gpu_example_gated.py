"""examples/serve_block.py with rotary positions, the gated network and a bound
on the cache: the operators together, as a user runs them.

Each step is compared with the 64-bit oracle on what that step read, the keys
and values with what the cache holds before it (see the operators' own tests for
the tolerances), and after each cut the cache with what it held before.
"""
import numpy as np
import pytest

from oracle import serve
from test_gpu_evict import score_error
from test_gpu_example import U, example, host, product
from test_gpu_kv4 import tolerance
from test_gpu_rotary import check as check_rotary

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def held(cache, pages, dim, dtype):
    """K and V [len, heads, dim] of each sequence's places."""
    from gptq_post_weight_gb300 import _lib

    out = []
    for b, n in enumerate(pages.lens.tolist()):
        at = torch.arange(n, device="cuda")
        slots = pages.table[b].long()[at // pages.page_size] * pages.page_size + at % pages.page_size
        out.append([host(x) for x in _lib.kv4_read(cache, slots, dim, pages.page_size, dtype)])
    return [k for k, _ in out], [v for _, v in out]


def gated(got, x, q4):
    nib, rungs, tab = (t.cpu().numpy() for t in q4)
    want = serve.gated(x, nib, rungs, tab)
    both = serve.linear(x, nib, rungs, tab)
    w, sc = np.abs(serve.weights(nib, rungs, tab)), np.abs(serve.weights(np.full_like(nib, 0x99), rungs, tab))
    ax, n = np.abs(x), x.shape[1]
    err = (2.0 ** -11 + n / 32 * 2.0 ** -23) * (ax @ w.T) + 34 * 143 * 2.0 ** -22 * (ax @ sc.T)
    h = both.shape[1] // 2
    g, u, eg, eu = both[:, :h], np.abs(both[:, h:]), err[:, :h], err[:, h:]
    off = 1.13 * eg * (u + eu) + np.abs(serve.activate(g, "silu")) * eu + 2.0 ** -20 * np.abs(want) + 2.0 ** -22 * np.abs(g) * u
    assert (np.abs(host(got) - want) <= off + 2.0 ** -8 * (np.abs(want) + off) + 2.0 ** -25).all()


def test_bounded_block_steps(lib):
    from gptq_post_weight_gb300 import _lib

    m = example()
    hidden, heads, kv, dim, inner, page, seqs = 256, 4, 2, 64, 384, 16, 3
    g = torch.Generator(device="cuda").manual_seed(5)
    draw = lambda t: torch.randn(t, hidden, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    block = m.GatedBlock(hidden, heads, kv, dim, inner, draw(1024),
                         frequencies=_lib.rotary_frequencies(dim, scaling="ramp", factor=4, length=64))
    pages = m.BoundedPages(seqs, 10, page, kv, budget=100, keep=75, recent=12, device="cuda")
    cache = _lib.kv4_cache(seqs * 10, kv, dim, page)
    scale, cuts = dim ** -0.5, 0
    for counts in ([97, 30, 1], [45, 0, 20], [1, 1, 1], [30, 2, 1], [1, 1, 1], [40, 60, 80], [1, 1, 1]):
        x, trace = draw(sum(counts)), {}
        before = pages.weights.double().cpu().numpy()
        out = block.forward(x, cache, pages, counts, trace)
        _lib.serve_check()
        # Positions go on where the sequence is, whatever has been evicted.
        first = pages.seen - torch.tensor(counts)
        where = np.concatenate([np.arange(n) + int(first[b]) for b, n in enumerate(counts)])
        np.testing.assert_array_equal(trace["positions"].cpu().numpy(), where)
        qkv = host(trace["qkv"])
        check_rotary(trace["q"], qkv[:, :heads], where, block.turns, "bf16", "half")
        q, ks_vs = host(trace["q"]), held(cache, pages, dim, torch.bfloat16)
        ks, vs = ks_vs
        lens = pages.lens.tolist()
        want = serve.attention(q, ks, vs, lens, heads // kv, scale, counts)
        tol = tolerance(q, ks, vs, lens, heads // kv, scale, counts, "bf16", want)
        assert (np.abs(host(trace["attention"]) - want) <= tol).all()
        lse = trace["lse"].double().cpu().numpy()
        add = serve.attention_weights(q, ks, lens, heads // kv, scale, lse, counts)
        es = score_error(q, ks, lens, heads // kv, scale, counts)
        e = max((x.max() for row in es for x in row if len(x)), default=0.0)
        w = pages.weights.double().cpu().numpy()
        for b, n in enumerate(lens):
            total = add[b] + before[b, :, :n]
            off = (e + 2.0 ** -22 * 40 + (counts[b] * 2 + 1) * 2.0 ** -24) * total  # (scores and sums below 18 each)
            assert (np.abs(w[b, :, :n] - total) <= off).all()
            assert not w[b, :, n:].any()
        product(trace["y"], host(trace["attention"]).reshape(len(x), -1), block.proj, residual=host(x))
        gated(trace["u"], host(trace["n2"]), block.up)
        product(out, host(trace["u"]), block.down, residual=host(trace["y"]))
        if (kept := pages.bound(cache)) is None:
            continue
        cuts += 1
        after_k, after_v = held(cache, pages, dim, torch.bfloat16)
        new = pages.weights.double().cpu().numpy()
        for b, n in enumerate(lens):
            for h in range(kv):
                places = serve.kept(w[b, h], n, 75, 12)
                assert kept[b, h].tolist() == places + [-1] * (75 - len(places))
                np.testing.assert_array_equal(after_k[b][:, h], ks[b][places, h])
                np.testing.assert_array_equal(after_v[b][:, h], vs[b][places, h])
                np.testing.assert_array_equal(new[b, h, :len(places)], w[b, h, places])
            assert not new[b, :, min(n, 75):].any()
    assert cuts == 3 and U == 2.0 ** -7  # at 142, 106 and 116 tokens of the first sequence


def test_example_runs(lib, monkeypatch, capsys):
    m = example()
    monkeypatch.setattr("sys.argv", ["serve_block.py", "--hidden", "256", "--heads", "4", "--kv-heads", "2", "--inner",
                                     "512", "--seqs", "3", "--prompt", "150", "--chunk", "64", "--steps", "5", "--gated",
                                     "--budget", "96"])
    m.main()
    assert "prompt: 450 tokens in 3 chunks" in capsys.readouterr().out


def test_two_streams_at_once(lib):
    # Every call twice side by side, on two streams and other data, against one
    # after the other: nothing is shared but the status word.
    from gptq_post_weight_gb300 import _lib

    heads, group, dim, page, inner, n = 2, 4, 128, 16, 700, 512
    turns = _lib.rotary_turns(_lib.rotary_frequencies(dim))
    sides = []
    for seed in (1, 2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        tokens, length = 300 + 40 * seed, 1500
        rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        sides.append(dict(
            qkv=rand(length, heads * (group + 2), dim), x=rand(tokens, n), tokens=tokens, length=length,
            nib=torch.randint(0, 256, (inner * n,), generator=g, device="cuda", dtype=torch.uint8),
            rungs=torch.randint(0, 32, (2 * inner * n // 32,), generator=g, device="cuda", dtype=torch.uint8),
            tab=torch.rand(2 * inner, 32, generator=g, device="cuda") * 0.01,
            table=torch.randperm(100, generator=g, device="cuda").int()[None]))

    def run(s):
        hq, at = heads * group, torch.arange(s["length"], device="cuda")
        cache = _lib.kv4_cache(100, heads, dim, page)
        slots = s["table"][0].long()[at // page] * page + at % page
        q = _lib.kv4_write_rotary(cache, s["qkv"][:, :hq], s["qkv"][:, hq:hq + heads], s["qkv"][:, hq + heads:], slots, page,
                                  at, turns)
        lens = torch.tensor([s["length"]], device="cuda", dtype=torch.int32)
        starts = torch.tensor([0, s["tokens"]], device="cuda", dtype=torch.int32)
        last = q[s["length"] - s["tokens"]:].contiguous()
        lse = torch.empty(s["tokens"], hq, device="cuda")
        o = _lib.kv4_attention(last, cache, s["table"], lens, page, starts, s["tokens"], lse=lse)
        w = _lib.kv4_weights(s["table"], page, heads)
        _lib.kv4_attention_weights(w, last, lse, cache, s["table"], lens, page, starts, s["tokens"])
        y = _lib.q4tp_gated(s["x"], s["nib"], s["rungs"], s["tab"])
        kept, new, left = _lib.kv4_evict(cache, s["table"], lens, w, 400, page, recent=30)
        return [q, o, lse, w, y, kept, new, left, cache, _lib.rotary(last, at[:s["tokens"]], turns, layout="interleaved")]

    alone = [run(s) for s in sides]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sides]
    together = [[], []]
    for _ in range(5):
        for k, s in enumerate(sides):
            with torch.cuda.stream(streams[k]):
                together[k].append(run(s))
    torch.cuda.synchronize()
    _lib.serve_check()
    for want, runs in zip(alone, together):
        for got in runs:
            assert all(torch.equal(a, b) for a, b in zip(want, got))
