"""The 4-bit key/value cache and its attention against the 64-bit oracle.

The codec is defined bit for bit, so written bytes and values read back are
compared exactly.  Attention, per output: the result is rounded once to T
(u |o|, u a whole ulp), a probability is rounded to T on its way into the
product (u / 2 of sum p |v| / sum p), and scores carry f32 error: with
|scale q.k| sums of D products, (D + 8) 2^-22 of scale sum |q k| goes into
each exponent, twice (numerator and sum).
"""
import numpy as np
import pytest

from oracle import serve

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def dev(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def keys(r, shape, dtype):
    return serve.round_to(r.standard_normal(shape) * np.exp(0.4 * r.standard_normal(shape[-1])) + 0.5, dtype)


def bits(x, dtype):
    """u16 patterns of numbers of the type (NaN: 0x7fff)."""
    x = np.asarray(x, dtype=np.float32)
    if dtype == "f16":
        b = x.astype(np.float16).view(np.uint16)
    else:
        b = (x.view(np.uint32) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FFF), b)


SHAPES = [(1, 1, 64, 16), (5, 3, 64, 16), (16, 2, 128, 32), (17, 5, 128, 64), (100, 8, 256, 16), (333, 2, 64, 48)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,heads,dim,page", SHAPES)
def test_write_bytes_and_read(lib, tokens, heads, dim, page, dtype):
    from gptq_post_weight_gb300 import _lib

    r = np.random.default_rng(tokens + dim)
    k, v = keys(r, (tokens, heads, dim), dtype), keys(r, (tokens, heads, dim), dtype)
    k[0, 0, :32] = 1.25  # a constant group
    k[-1, -1, 0] = 1e-7
    pages = tokens // page + 3
    slots = r.permutation(pages * page)[:tokens].astype(np.int64)
    cache = _lib.kv4_cache(pages, heads, dim, page)
    cache.fill_(0xA5)
    _lib.kv4_write(cache, dev(k, DT[dtype]), dev(v, DT[dtype]), dev(slots), page)
    # Every byte of the pool: the written rows as the oracle packs them, the
    # rest untouched.
    want = np.full((pages, heads, page // 16, 20 * dim), 0xA5, dtype=np.uint8)
    for which, x in ((0, k), (10 * dim, v)):
        c, s, z = serve.quantise(x, dtype)
        for i, slot in enumerate(slots):
            pg, blk, row = slot // page, slot % page // 16, slot % 16
            for h in range(heads):
                b = want[pg, h, blk]
                at = which + row * dim // 2
                b[at:at + dim // 2] = (c[i, h, 0::2] | (c[i, h, 1::2] << 4)).astype(np.uint8)
                at = which + 8 * dim + row * dim // 8
                b[at:at + dim // 8] = np.stack([bits(s[i, h], dtype), bits(z[i, h], dtype)], -1).reshape(-1).view(np.uint8)
    got = cache.cpu().numpy().reshape(want.shape)
    np.testing.assert_array_equal(got, want)
    kr, vr = _lib.kv4_read(cache, dev(slots), dim, page, DT[dtype])
    np.testing.assert_array_equal(host(kr), serve.round_trip(k, dtype))
    np.testing.assert_array_equal(host(vr), serve.round_trip(v, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_strided_views_and_padding_slots(lib, dtype):
    from gptq_post_weight_gb300 import _lib

    r = np.random.default_rng(5)
    tokens, heads, dim, page = 21, 2, 128, 16
    qkv = dev(keys(r, (tokens, 3 * heads, dim), dtype), DT[dtype])
    k, v = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
    slots = torch.arange(3, 3 + tokens, device="cuda")
    slots[4], slots[9], slots[20] = -1, 4 * page, 1 << 40  # outside a pool of 4 pages
    cache = _lib.kv4_cache(4, heads, dim, page)
    _lib.kv4_write(cache, k, v, slots, page)
    kr, vr = _lib.kv4_read(cache, slots, dim, page, DT[dtype])
    wk, wv = serve.round_trip(host(k), dtype), serve.round_trip(host(v), dtype)
    for i in (4, 9, 20):
        wk[i] = wv[i] = 0
    np.testing.assert_array_equal(host(kr), wk)
    np.testing.assert_array_equal(host(vr), wv)
    # Heads outermost: [heads, tokens, dim] seen as [tokens, heads, dim].
    kt = k.transpose(0, 1).contiguous().transpose(0, 1)
    again = _lib.kv4_cache(4, heads, dim, page)
    _lib.kv4_write(again, kt, v, slots, page)
    assert torch.equal(cache, again)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_non_finite_and_extreme_groups(lib, dtype):
    from gptq_post_weight_gb300 import _lib

    r = np.random.default_rng(6)
    x = keys(r, (6, 1, 128), dtype)
    x[0, 0, 5], x[1, 0, 40], x[2, 0, 70] = np.nan, np.inf, -np.inf
    big = serve.TYPES[dtype][2]
    x[3, 0, 0], x[3, 0, 1] = big, -big
    x[4, 0, 96:] = 0
    x[5, 0, :32] = serve.round_to(np.arange(32) * 1e-7, dtype)
    cache = _lib.kv4_cache(1, 1, 128, 16)
    slots = torch.arange(6, device="cuda")
    _lib.kv4_write(cache, dev(x, DT[dtype]), dev(x[::-1], DT[dtype]), slots, 16)
    k, v = _lib.kv4_read(cache, slots, 128, 16, DT[dtype])
    want = serve.round_trip(x, dtype)
    assert np.isnan(want[0, 0, :32]).all() and np.isnan(want[3, 0, :32]).all()
    np.testing.assert_array_equal(host(k), want)
    np.testing.assert_array_equal(host(v), want[::-1])


def test_large_offsets(lib):
    # A pool past 2^32 bytes: pages at its end keep their own bytes.
    from gptq_post_weight_gb300 import _lib

    heads, dim, page = 8, 128, 64
    per = heads * page * dim * 5 // 4
    pages = (1 << 32) // per + 100
    cache = _lib.kv4_cache(pages, heads, dim, page)
    r = np.random.default_rng(8)
    slots = np.array([0, 1, (pages - 1) * page, pages * page - 1, (pages // 2) * page + 7], dtype=np.int64)
    k, v = keys(r, (5, heads, dim), "bf16"), keys(r, (5, heads, dim), "bf16")
    _lib.kv4_write(cache, dev(k, torch.bfloat16), dev(v, torch.bfloat16), dev(slots), page)
    kr, vr = _lib.kv4_read(cache, dev(slots), dim, page, torch.bfloat16)
    np.testing.assert_array_equal(host(kr), serve.round_trip(k, "bf16"))
    np.testing.assert_array_equal(host(vr), serve.round_trip(v, "bf16"))
    q = keys(r, (1, heads, dim), "bf16")
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    o = _lib.kv4_attention(dev(q, torch.bfloat16), cache, table, torch.tensor([1], dtype=torch.int32, device="cuda"),
                           page)
    np.testing.assert_array_equal(host(o)[0], serve.round_trip(v[2:3], "bf16")[0])


# ---------------------------------------------------------------- attention


def context(r, lens, heads, dim, page, dtype, junk=0xFF, spare=0):
    """A pool with the sequences' keys and values in shuffled pages; every byte
    that no token wrote is junk (0xFF: NaN parameters)."""
    from gptq_post_weight_gb300 import _lib

    per = max(1, max(-(-n // page) for n in lens)) + spare
    pages = per * len(lens) + 2
    order = r.permutation(pages)
    table = order[:per * len(lens)].reshape(len(lens), per).astype(np.int32)
    cache = _lib.kv4_cache(pages, heads, dim, page)
    cache.fill_(junk)
    ks, vs = [], []
    for b, n in enumerate(lens):
        k, v = keys(r, (n, heads, dim), dtype), keys(r, (n, heads, dim), dtype)
        pos = np.arange(n)
        slots = table[b, pos // page].astype(np.int64) * page + pos % page
        if n:
            _lib.kv4_write(cache, dev(k, DT[dtype]), dev(v, DT[dtype]), dev(slots), page)
        ks.append(serve.round_trip(k, dtype) if n else k)
        vs.append(serve.round_trip(v, dtype) if n else v)
    return cache, dev(table), dev(np.array(lens, dtype=np.int32)), ks, vs


def tolerance(q, ks, vs, lens, group, scale, q_lens, dtype, want):
    u = 2.0 ** (1 - serve.TYPES[dtype][0])
    aq, dim = np.abs(q), q.shape[2]
    tol = np.zeros_like(want)
    at = 0
    for b, ln in enumerate(lens):
        nq = 1 if q_lens is None else q_lens[b]
        for i in range(nq):
            m = ln - nq + i + 1
            if m > 0:
                for h in range(q.shape[1]):
                    k, v = ks[b][:m, h // group], vs[b][:m, h // group]
                    sc = k @ q[at + i, h] * scale
                    p = np.exp(sc - sc.max())
                    p /= p.sum()
                    e = (dim + 8) * 2.0 ** -22 * scale * (np.abs(k) @ aq[at + i, h]).max()
                    tol[at + i, h] = (0.5 * u + 2 * e + 2.0 ** -20) * (p @ np.abs(v))
        at += nq
    return tol + u * np.abs(want) + 2.0 ** -24


def attend(q, cache, table, lens, page, dtype, q_lens=None, **kw):
    from gptq_post_weight_gb300 import _lib

    starts, max_q = None, 1
    if q_lens is not None:
        starts = dev(np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32))
        max_q = max(q_lens)
    o = _lib.kv4_attention(q if isinstance(q, torch.Tensor) else dev(q, DT[dtype]), cache, table, lens, page,
                           q_starts=starts, max_q=max_q, **kw)
    _lib.serve_check()
    return o


def one(lens, heads, group, dim, page, dtype, q_lens=None, seed=0, scale=None):
    r = np.random.default_rng(seed)
    cache, table, lens_d, ks, vs = context(r, lens, heads, dim, page, dtype)
    q = serve.round_to(r.standard_normal((len(lens) if q_lens is None else sum(q_lens), heads * group, dim)), dtype)
    got = host(attend(q, cache, table, lens_d, page, dtype, q_lens, scale=scale))
    sc = dim ** -0.5 if scale is None else scale
    want = serve.attention(q, ks, vs, lens, group, sc, q_lens)
    tol = tolerance(q, ks, vs, lens, group, sc, q_lens, dtype, want)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.nanmax(np.abs(got - want)[bad]), np.argwhere(bad)[:5])
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (256, 32)])
@pytest.mark.parametrize("group", [1, 4, 5, 16])
def test_single_tokens(lib, dim, page, group, dtype):
    one([1, 2, 15, 16, 17, 63, 64, 65, 200, 0, 333], 2, group, dim, page, dtype, seed=dim + group)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_groups_past_a_tile(lib, dim, dtype):
    one([40, 100], 1, 37, dim, 16, dtype, seed=3)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q_lens", [[2, 1, 5], [7, 3, 1], [16, 0, 9], [40, 33, 20]])
def test_several_queries(lib, q_lens, dim, dtype):
    # The third sequence has fewer keys than queries where q_lens allow it:
    # its first queries see nothing.
    one([50, 129, 4], 2, 4, dim, 16, dtype, q_lens, seed=4)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q_lens,lens", [([130, 65], [130, 300]), ([257], [257]), ([70, 200, 1], [1000, 200, 77])])
def test_prompt_chunks(lib, q_lens, lens, dim, dtype):
    one(lens, 2, 3, dim, 32, dtype, q_lens, seed=5)


def test_long_contexts(lib):
    one([20001, 3, 4096], 1, 8, 128, 64, "bf16", seed=6)
    one([9001], 2, 4, 128, 16, "f16", [5], seed=7)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group,q_lens,lens", [
    (2, None, [9001, 700]),      # one row block cut into scores of pieces
    (3, [4, 1], [5000, 130]),    # 12 rows
    (4, [5, 5], [3000, 2000]),   # 20 rows
    (4, [7, 8], [3000, 2000]),   # 32 rows
    (4, [9, 2], [3000, 2000]),   # 36 rows
    (4, [20], [12000]),          # 80 rows, the tiles take turns
    (4, [40], [12000]),          # one tile shared by every CTA
])
def test_cut_items(lib, group, q_lens, lens, dim, dtype):
    one(lens, 1, group, dim, 16, dtype, q_lens, seed=8)


def test_many_sequences(lib):
    r = np.random.default_rng(9)
    one([int(n) for n in r.integers(0, 40, 1500)], 1, 2, 64, 16, "bf16", seed=9)


def test_large_scores_and_scale(lib):
    one([300], 1, 2, 128, 16, "bf16", seed=10, scale=3.0)
    one([77], 1, 2, 64, 16, "f16", [9], seed=11, scale=0.0)


def test_key_of_infinite_score_or_nan_in_hidden_place_stays_hidden(lib):
    # Everything past kv_lens is 0xFF bytes (NaN parameters) in every test
    # above; here it is the tail of a page that was written with NaN.
    from gptq_post_weight_gb300 import _lib

    r = np.random.default_rng(12)
    cache, table, lens, ks, vs = context(r, [30], 1, 64, 16, "bf16", spare=1)
    nan = torch.full((10, 1, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([int(table[0, p // 16]) * 16 + p % 16 for p in range(20, 30)], device="cuda")
    _lib.kv4_write(cache, nan, nan, slots, 16)
    short = torch.tensor([20], dtype=torch.int32, device="cuda")
    q = serve.round_to(r.standard_normal((1, 4, 64)), "bf16")
    got = host(attend(q, cache, table, short, 16, "bf16"))
    want = serve.attention(q, [ks[0][:20]], [vs[0][:20]], [20], 4, 0.125)
    assert np.abs(got - want).max() < 0.02
    assert np.isnan(host(attend(q, cache, table, lens, 16, "bf16"))).all()


def test_strided_queries_given_buffers_and_stream(lib):
    from gptq_post_weight_gb300 import _lib

    r = np.random.default_rng(13)
    cache, table, lens, ks, vs = context(r, [90, 18], 2, 128, 16, "f16")
    q = serve.round_to(r.standard_normal((2, 8, 128)), "f16")
    plain = attend(q, cache, table, lens, 16, "f16")
    wide = torch.full((2, 12, 136), float("nan"), dtype=torch.float16, device="cuda")
    wide[:, 2:10, :128] = dev(q, torch.float16)
    out = torch.empty(2, 8, 128, dtype=torch.float16, device="cuda")
    ws = _lib.workspace(lib.gptq_kv4_attention_workspace_bytes(128, 4, 1), "cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = attend(wide[:, 2:10, :128], cache, table, lens, 16, "f16", out=out, ws=ws, stream=side)
    torch.cuda.synchronize()
    assert got is out and torch.equal(out, plain)


def test_same_bits_every_time(lib):
    r = np.random.default_rng(14)
    for q_lens in (None, [4, 4], [150, 90]):
        cache, table, lens, ks, vs = context(r, [3000, 777], 2, 128, 64, "bf16")
        n = 2 if q_lens is None else sum(q_lens)
        q = serve.round_to(r.standard_normal((n, 8, 128)), "bf16")
        a = attend(q, cache, table, lens, 64, "bf16", q_lens)
        for _ in range(3):
            assert torch.equal(a, attend(q, cache, table, lens, 64, "bf16", q_lens))


def test_table_entries_outside_the_pool_stay_inside(lib):
    # Documented: such an entry reads page 0; the call stays in its buffers.
    r = np.random.default_rng(15)
    cache, table, lens, ks, vs = context(r, [40], 1, 64, 16, "bf16")
    bad = table.clone()
    bad[0, 1] = 1 << 30
    bad[0, 2] = -5
    zero = table.clone()
    zero[0, 1] = zero[0, 2] = 0
    q = serve.round_to(r.standard_normal((1, 2, 64)), "bf16")
    a, b = attend(q, cache, bad, lens, 16, "bf16"), attend(q, cache, zero, lens, 16, "bf16")
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_lengths_past_the_table_count_as_its_capacity(lib):
    r = np.random.default_rng(16)
    cache, table, lens, ks, vs = context(r, [32], 1, 64, 16, "bf16")
    q = serve.round_to(r.standard_normal((1, 2, 64)), "bf16")
    a = attend(q, cache, table, lens, 16, "bf16")
    assert torch.equal(a, attend(q, cache, table, lens + 1000, 16, "bf16"))


def test_waits_run_out(lib):
    from gptq_post_weight_gb300 import _lib

    r = np.random.default_rng(17)
    cache, table, lens, ks, vs = context(r, [500], 2, 128, 16, "bf16")
    for q_lens in (None, [3], [200]):
        q = serve.round_to(r.standard_normal((1 if q_lens is None else q_lens[0], 4, 128)), "bf16")
        want = attend(q, cache, table, lens, 16, "bf16", q_lens)
        try:
            _lib.test_set_wait(1_000_000, no_loads=True)
            with pytest.raises(_lib.GptqError) as ei:
                attend(q, cache, table, lens, 16, "bf16", q_lens)
            assert ei.value.code == 6
        finally:
            _lib.test_set_wait()
        assert torch.equal(want, attend(q, cache, table, lens, 16, "bf16", q_lens))


def test_nothing_to_do(lib):
    from gptq_post_weight_gb300 import _lib

    cache = _lib.kv4_cache(2, 2, 64, 16)
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    s = torch.empty(0, dtype=torch.int64, device="cuda")
    _lib.kv4_write(cache, e, e, s, 16)
    k, v = _lib.kv4_read(cache, s, 64, 16, torch.bfloat16)
    assert k.shape == v.shape == (0, 2, 64) and not cache.any()
    o = _lib.kv4_attention(e, cache, torch.empty(0, 1, dtype=torch.int32, device="cuda"),
                           torch.empty(0, dtype=torch.int32, device="cuda"), 16)
    assert o.shape == (0, 2, 64)


def test_buffers_belong_to_the_call_s_stream(lib):
    # What a call on a given stream allocates is that stream's memory: given
    # back, it goes to that stream's next allocation, never to one of the
    # current stream's, which would not wait for the call.
    from gptq_post_weight_gb300 import _lib

    r = np.random.default_rng(17)
    cache, table, lens, ks, vs = context(r, [9000, 40], 2, 128, 16, "bf16")
    q = dev(serve.round_to(r.standard_normal((2, 8, 128)), "bf16"), torch.bfloat16)
    slots = torch.arange(3, device="cuda")
    x = torch.ones(3, 64, dtype=torch.bfloat16, device="cuda")
    nib, rungs = torch.zeros(64 * 32, dtype=torch.uint8, device="cuda"), torch.zeros(64 * 2, dtype=torch.uint8, device="cuda")
    tab = torch.ones(64, 32, device="cuda")
    side = torch.cuda.Stream()
    calls = [lambda: _lib.kv4_attention(q, cache, table, lens, 16, stream=side),
             lambda: _lib.kv4_read(cache, slots, 128, 16, torch.bfloat16, stream=side)[1],
             lambda: _lib.q4tp_linear(x, nib, rungs, tab, stream=side)]
    torch.cuda.synchronize()
    for call in calls:
        y = call()
        at, shape = y.data_ptr(), y.shape
        del y
        mine = [torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
        assert at not in [t.data_ptr() for t in mine]
        with torch.cuda.stream(side):
            theirs = [torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
        assert at in [t.data_ptr() for t in theirs]
        side.synchronize()
    # The workspace of cut items, too: the same bits as on the current stream.
    a, b = _lib.kv4_attention(q, cache, table, lens, 16), calls[0]()
    torch.cuda.synchronize()
    assert torch.equal(a, b)
