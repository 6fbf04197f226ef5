"""Uses of the serving operators beside the sizes of test_gpu_linear.py and
test_gpu_kv4.py, whose tolerances these tests use."""
import numpy as np
import pytest

from oracle import serve
import test_gpu_kv4 as kv

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q_lens,lens", [([3, 0, 1], [70, 5, 1]), ([1, 1, 2], [17, 0, 300]), ([40, 2, 9], [50, 33, 4]),
                                         ([300, 1, 140], [700, 64, 140])])
def test_one_query_head_with_several_queries(lib, q_lens, lens, dim, dtype):
    kv.one(lens, 1, 1, dim, 16, dtype, q_lens, seed=20)


@pytest.mark.parametrize("seqs", [0, 2])
def test_no_queries_with_starts(lib, seqs):
    from gptq_post_weight_gb300 import _lib

    cache = _lib.kv4_cache(2, 2, 64, 16)
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    o = _lib.kv4_attention(q, cache, torch.zeros(seqs, 1, **i32), torch.ones(seqs, **i32), 16,
                           q_starts=torch.zeros(seqs + 1, **i32), max_q=3)
    assert o.shape == (0, 4, 64)


@pytest.mark.parametrize("heads,group", [(1, 1), (2, 4)])
def test_one_token_of_any_token_stride(lib, heads, group):
    r = np.random.default_rng(21)
    cache, table, lens, ks, vs = kv.context(r, [40], heads, 64, 16, "bf16")
    q = serve.round_to(r.standard_normal((1, heads * group, 64)), "bf16")
    plain = kv.attend(q, cache, table, lens, 16, "bf16")
    wide = torch.zeros(heads * group * 64 + 3, dtype=torch.bfloat16, device="cuda")
    wide[:-3] = kv.dev(q, torch.bfloat16).flatten()
    odd = torch.as_strided(wide, (1, heads * group, 64), (heads * group * 64 + 3, 64, 1))
    assert torch.equal(plain, kv.attend(odd, cache, table, lens, 16, "bf16"))
    assert torch.equal(plain, kv.attend(odd, cache, table, lens, 16, "bf16", [1]))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_slot_given_twice_mixes_its_tokens_and_leaves_the_others(lib, dtype):
    # What the header says of it: each word is one of the tokens', the other
    # slots hold what they should.
    from gptq_post_weight_gb300 import _lib

    r = np.random.default_rng(22)
    tokens, heads, dim, page = 300, 2, 128, 16
    k, v = kv.keys(r, (tokens, heads, dim), dtype), kv.keys(r, (tokens, heads, dim), dtype)
    slots = r.permutation(400)[:tokens].astype(np.int64)
    pairs = [(0, 1), (5, 299), (40, 200)]
    for i, j in pairs:
        slots[j] = slots[i]
    last = [b for _, b in pairs]
    first = [a for a, _ in pairs]

    def written(keep):
        cache = _lib.kv4_cache(25, heads, dim, page)
        _lib.kv4_write(cache, kv.dev(k[keep], kv.DT[dtype]), kv.dev(v[keep], kv.DT[dtype]), kv.dev(slots[keep]), page)
        return cache.view(torch.int32)

    everyone = np.arange(tokens)
    both = written(everyone)
    one, two = written(np.setdiff1d(everyone, last)), written(np.setdiff1d(everyone, first))
    assert (one != two).any()
    assert ((both == one) | (both == two)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("group,max_q,lens,q_lens,extra", [
    (2, 1, [30, 40], [1, 1], [0, 3]),        # clusters; two sequences have rows past max_q
    (2, 3, [30, 40, 9], [3, 0, 2], [0, 0, 0]),
    (4, 5, [300, 7000, 12], [5, 4, 5], [2, 0, 1]),  # shares and a join
    (4, 60, [100, 3000, 70], [60, 0, 31], [0, 0, 0]),  # tcgen05, the tiles in turns
    (4, 150, [200, 900], [150, 7], [70, 0]),   # tcgen05
    (2, 2, [20] * 1100, [2, 1] * 550, [0, 1] * 550),  # more sequences than one launch takes
])
def test_rows_that_no_sequence_has_are_zero(lib, group, max_q, lens, q_lens, extra, dtype):
    # Rows before the first sequence's, after the last one's and past max_q of
    # their own: zeros in `out`, and the others as without them.
    r = np.random.default_rng(23)
    heads, dim, page, before, after = 2, 64, 16, 3, 70
    counts = [n if e == 0 else max_q + e for n, e in zip(q_lens, extra)]
    q_lens = [min(c, max_q) for c in counts]
    cache, table, lens_d, ks, vs = kv.context(r, lens, heads, dim, page, dtype)
    starts = before + np.concatenate([[0], np.cumsum(counts)])
    tq = int(starts[-1]) + after
    q = serve.round_to(r.standard_normal((tq, heads * group, dim)), dtype)
    out = torch.full((tq, heads * group, dim), float("nan"), dtype=kv.DT[dtype], device="cuda")
    from gptq_post_weight_gb300 import _lib

    got = kv.host(_lib.kv4_attention(kv.dev(q, kv.DT[dtype]), cache, table, lens_d, page,
                                     q_starts=kv.dev(starts.astype(np.int32)), max_q=max_q, out=out))
    _lib.serve_check()
    seen = np.concatenate([np.arange(s, s + n) for s, n in zip(starts, q_lens)])
    rest = np.setdiff1d(np.arange(tq), seen)
    assert not got[rest].any()  # (a NaN counts as any)
    want = serve.attention(q[seen], ks, vs, lens, group, dim ** -0.5, q_lens)
    tol = kv.tolerance(q[seen], ks, vs, lens, group, dim ** -0.5, q_lens, dtype, want)
    assert (np.abs(got[seen] - want) <= tol).all()


def test_no_sequences_leave_every_row_zero(lib):
    from gptq_post_weight_gb300 import _lib

    cache = _lib.kv4_cache(2, 2, 64, 16)
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.ones(5, 4, 64, dtype=torch.float16, device="cuda")
    out = torch.full_like(q, float("nan"))
    _lib.kv4_attention(q, cache, torch.zeros(0, 1, **i32), torch.zeros(0, **i32), 16,
                       q_starts=torch.zeros(1, **i32), max_q=3, out=out)
    assert not out.any()


def product_of(p, dtype, x):
    """(result, what it has to be, how far off a finite one may be)."""
    import test_gpu_linear as lin

    q = dict(p, x=x)
    with np.errstate(invalid="ignore"):
        want = serve.linear(x, p["nib"], p["rungs"], p["tab"])
        # Past T's range a result is an infinity.
        want = np.where(np.abs(want) > serve.TYPES[dtype][2], np.copysign(np.inf, want), want)
    w = np.abs(serve.weights(p["nib"], p["rungs"], p["tab"]))
    sc = np.abs(serve.weights(np.full_like(p["nib"], 0x99), p["rungs"], p["tab"]))
    ax = np.where(np.isfinite(x), np.abs(x), 0)
    u = 2.0 ** (1 - serve.TYPES[dtype][0])
    # As in test_gpu_linear.py; plain sums in f32 instead of a group's at a time
    # are n 2^-23 of sum |x w|.
    err = 34 * 143 * 2.0 ** -22 * (ax @ sc.T) + x.shape[1] * 2.0 ** -23 * (ax @ w.T)
    if len(x) > 8:
        err = err + 0.5 * u * (ax @ w.T)
    tol = np.where(np.isfinite(want), u * np.abs(want) + err + 2.0 ** -24, 0)
    return lin.run(q, dtype, "none").float().cpu().numpy().astype(np.float64), want, tol


def same_numbers(got, want, tol):
    with np.errstate(invalid="ignore"):
        near = np.abs(got - want) <= tol
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    assert (near | np.isnan(want) | (got == want)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens", [1, 2, 3, 4, 6, 8, 12, 40, 300])
def test_infinite_activations(lib, tokens, dtype):
    # A row has an infinity in columns of every sign of code, one of a zero
    # code gives NaN, opposite ones give NaN; the other rows do not notice.
    import test_gpu_linear as lin

    rows, n = 300, 2080
    p = lin.problem(tokens, rows, n, dtype, 41)
    r = np.random.default_rng(42)
    x = p["x"].copy()
    x[0, 7] = np.inf
    if tokens > 2:
        x[1, [40, 2079]] = -np.inf, np.inf
        x[2, 1000] = np.nan
    got, want, tol = product_of(p, dtype, x)
    assert np.isinf(want[0]).any() and np.isnan(want[0]).any()
    same_numbers(got, want, tol)
    plain = lin.run(p, dtype, "none").float().cpu().numpy()
    clean = np.isfinite(x).all(1)
    np.testing.assert_array_equal(got[clean], plain[clean])


@pytest.mark.parametrize("tokens", [1, 2, 4, 8])
def test_activations_near_the_end_of_bf16(lib, tokens):
    # 2^112 and more times an offset of 136 would leave f32's range.
    import test_gpu_linear as lin

    p = lin.problem(tokens, 70, 544, "bf16", 43)
    p["tab"] = (p["tab"] / 64).astype(np.float32)
    x = p["x"].copy()
    x[0, ::50] = serve.round_to(np.float64(3e38) * np.sign(x[0, ::50]), "bf16")
    if tokens > 1:
        x[1] = serve.round_to(x[1] * 2.0 ** 111, "bf16")
    got, want, tol = product_of(p, "bf16", x)
    assert np.isfinite(want).all()
    same_numbers(got, want, tol)


@pytest.mark.parametrize("tokens", [1, 5, 33])
@pytest.mark.parametrize("how", ["debias", "act order"])
def test_product_with_weights_of_the_other_quantizers(lib, how, tokens):
    # What debias leaves of the ladder, and act order's scales put back into one
    # (it returns a scale a group, and every scale is its rung's entry).
    import synth
    import test_gpu_linear as lin
    from gptq_post_weight_gb300 import _lib

    cfg = synth.config("tiny")
    hp, w = (t.cuda() for t in synth.make_problem(cfg, "cpu"))
    if how == "debias":
        q = _lib.quantize_group(hp, cfg.n, w, cfg.lam)
        before = q["tab"].clone()
        _lib.debias(4, w, hp, q["nibbles"], q["rungs"], q["tab"], q["lost"], q["scales"])
        tab = q["tab"]
        assert (tab != before).any()
        at = q["rungs"].view(len(w), -1).long()
        assert torch.equal(torch.gather(tab, 1, at).flatten(), q["scales"].flatten())
    else:
        q = _lib.quantize_group_act_order(hp, cfg.n, w, cfg.lam)
        at = q["rungs"].view(len(w), -1).long()
        tab = torch.zeros(len(w), 32, device="cuda").scatter_(1, at, q["scales"].view(len(w), -1))
    r = np.random.default_rng(51)
    p = dict(x=serve.round_to(r.standard_normal((tokens, cfg.n)), "bf16"), bias=None, residual=None,
             nib=q["nibbles"].cpu().numpy(), rungs=q["rungs"].cpu().numpy(), tab=tab.cpu().numpy())
    lin.check(lin.run(p, "bf16", "none"), p, "bf16", "none")
    # The oracle's weights are the quantizer's: close to what it was given.
    wq = serve.weights(p["nib"], p["rungs"], p["tab"])
    alive = torch.diagonal(full(hp, cfg.n)).cpu().numpy() > 0
    w0 = w.cpu().numpy()[:, alive]
    assert np.linalg.norm(wq[:, alive] - w0) < 0.3 * np.linalg.norm(w0)


def full(hp, n):
    h = torch.zeros(n, n, device=hp.device)
    i = torch.triu_indices(n, n, device=hp.device)
    h[i[0], i[1]] = hp
    return h


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group,nq,ln", [(1, 5, 40), (4, 6, 300), (4, 20, 200), (2, 150, 400)])
def test_keys_that_are_no_numbers_reach_only_queries_that_see_them(lib, group, nq, ln, dim, dtype):
    # Keys of NaN and of infinities (which the cache holds as NaN) a few places
    # before the end: the queries before them are as ever, the others NaN.
    from gptq_post_weight_gb300 import _lib

    r = np.random.default_rng(61)
    heads, page = 2, 16
    cache, table, lens, ks, vs = kv.context(r, [ln], heads, dim, page, dtype)
    bad = [ln - 3, ln - 2]
    k = kv.keys(r, (2, heads, dim), dtype)
    k[0, :, 5], k[1, :, dim - 1] = np.nan, -np.inf
    slots = torch.tensor([int(table[0, p // page]) * page + p % page for p in bad], device="cuda")
    _lib.kv4_write(cache, kv.dev(k, kv.DT[dtype]), kv.dev(vs[0][bad], kv.DT[dtype]), slots, page)
    v = vs[0].copy()
    v[bad] = serve.round_trip(vs[0][bad], dtype)
    q = serve.round_to(r.standard_normal((nq, heads * group, dim)), dtype)
    got = kv.host(kv.attend(q, cache, table, lens, page, dtype, [nq]))
    n = nq - 3  # queries before the first of them
    want = serve.attention(q[:n], [ks[0][:ln - 3]], [v[:ln - 3]], [ln - 3], group, dim ** -0.5, [n])
    tol = kv.tolerance(q[:n], [ks[0][:ln - 3]], [v[:ln - 3]], [ln - 3], group, dim ** -0.5, [n], dtype, want)
    assert (np.abs(got[:n] - want) <= tol).all()
    assert np.isnan(got[n:]).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group,nq", [(2, 20), (1, 150), (1, 300)])
def test_prompt_chunks_of_many_sequences_that_see_nothing(lib, group, nq, dim):
    # Tiles without steps one after the other, which the roles of a CTA pass at
    # their own speed, before and between tiles with steps.
    from gptq_post_weight_gb300 import _lib

    r = np.random.default_rng(24)
    heads, page, seqs = 8, 16, 400
    lens = [0] * seqs
    lens[seqs // 2], lens[-1] = 90, 33
    cache, table, _, kk, vv = kv.context(r, [90, 33], heads, dim, page, "bf16")
    wide = torch.zeros(seqs, table.shape[1], dtype=torch.int32, device="cuda")
    wide[seqs // 2], wide[-1] = table[0], table[1]
    q = serve.round_to(r.standard_normal((2 * nq, heads * group, dim)), "bf16")
    qd = torch.ones(seqs * nq, heads * group, dim, dtype=torch.bfloat16, device="cuda")
    qd.view(seqs, nq, -1)[[seqs // 2, seqs - 1]] = kv.dev(q, torch.bfloat16).view(2, nq, -1)
    starts = torch.arange(0, seqs * nq + 1, nq, dtype=torch.int32, device="cuda")
    out = torch.full_like(qd, float("nan"))
    _lib.kv4_attention(qd, cache, wide, torch.tensor(lens, dtype=torch.int32, device="cuda"), page, q_starts=starts,
                       max_q=nq, out=out)
    _lib.serve_check()
    got = kv.host(out).reshape(seqs, nq, heads * group, dim)
    assert not np.delete(got, [seqs // 2, seqs - 1], 0).any()
    want = serve.attention(q, kk, vv, [90, 33], group, dim ** -0.5, [nq, nq])
    tol = kv.tolerance(q, kk, vv, [90, 33], group, dim ** -0.5, [nq, nq], "bf16", want)
    assert (np.abs(got[[seqs // 2, seqs - 1]].reshape(want.shape) - want) <= tol).all()


def spoil(r, cache, table, ks, vs, lens, page, dtype, places):
    """Writes a NaN or an infinity into one group of a value at each (sequence,
    token) of `places`; the oracle's copy of the values follows."""
    from gptq_post_weight_gb300 import _lib

    heads, dim = vs[0].shape[1:]
    slots, k, v = [], [], []
    for i, (b, p) in enumerate(places):
        x = vs[b][p].copy()
        x[np.isnan(x)] = 1.0
        x[r.integers(heads), r.integers(dim)] = [np.nan, np.inf, -np.inf][i % 3]
        slots.append(int(table[b, p // page]) * page + p % page)
        k.append(ks[b][p])
        v.append(x)
    k, v = np.stack(k), np.stack(v)
    _lib.kv4_write(cache, kv.dev(k, kv.DT[dtype]), kv.dev(v, kv.DT[dtype]), torch.tensor(slots, device="cuda"), page)
    k, v = serve.round_trip(k, dtype), serve.round_trip(v, dtype)
    for (b, p), kk, x in zip(places, k, v):
        ks[b][p], vs[b][p] = kk, x


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,group,q_lens,lens", [
    (1, 1, [6], [40]),                                  # clusters
    (2, 2, [4, 1], [70, 33]),                           # clusters, two sequences
    (2, 4, [5, 3, 1, 2] * 5, [300, 40, 7, 129] * 5),    # shares, several items each
    (1, 4, [8], [9000]),                                # an item cut into pieces
    (2, 4, [20, 9, 1] * 4, [200, 60, 30] * 4),          # tcgen05, the tiles in turns
    (1, 2, [60], [12000]),                              # the same, cut
    (2, 2, [150, 3, 128] * 3, [400, 20, 128] * 3),      # tcgen05
    (1, 4, [130], [9000]),                              # the same, cut
])
def test_values_that_are_no_numbers_reach_only_queries_that_see_them(lib, heads, group, q_lens, lens, dim, dtype):
    # Values spoiled at places that the last queries of every other sequence see
    # and its first ones do not, at one that all see, and at its very last.
    r = np.random.default_rng(62)
    page = 16
    cache, table, lens_d, ks, vs = kv.context(r, lens, heads, dim, page, dtype)
    places = []
    for b in range(0, len(lens), 2):
        first = lens[b] - q_lens[b]  # the first token that not every query sees
        some = {lens[b] - 1, first + int(r.integers(q_lens[b])), first + int(r.integers(q_lens[b]))}
        if b % 4 == 2 and first > 0:
            some.add(int(r.integers(first)))
        places += [(b, p) for p in sorted(some)]
    spoil(r, cache, table.cpu(), ks, vs, lens, page, dtype, places)
    q = serve.round_to(r.standard_normal((sum(q_lens), heads * group, dim)), dtype)
    got = kv.host(kv.attend(q, cache, table, lens_d, page, dtype, q_lens))
    with np.errstate(invalid="ignore"):
        want = serve.attention(q, ks, vs, lens, group, dim ** -0.5, q_lens)
    clean = [np.where(np.isnan(v), 0, v) for v in vs]
    tol = kv.tolerance(q, ks, clean, lens, group, dim ** -0.5, q_lens, dtype, np.nan_to_num(want))
    assert np.isnan(want).any() and np.isfinite(want).any()
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    assert (np.abs(got - want) <= tol)[np.isfinite(want)].all()


@pytest.mark.parametrize("page", [48, 80, 4096])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q_lens,lens", [(None, [47, 48, 49, 500, 1]), ([3, 1, 5], [50, 161, 300]),
                                         ([40, 9], [400, 97]), ([200, 1, 70], [700, 33, 81])])
def test_pages_that_are_no_power_of_two_or_large(lib, q_lens, lens, dim, page):
    kv.one(lens, 2, 2, dim, page, "bf16", q_lens, seed=71)


@pytest.mark.parametrize("nq", [1, 4, 30, 150])
def test_queries_in_strided_and_transposed_layouts(lib, nq):
    # A slice of a wider projection, and heads outermost.
    r = np.random.default_rng(72)
    cache, table, lens, ks, vs = kv.context(r, [400, 160], 2, 128, 32, "f16")
    q = kv.dev(serve.round_to(r.standard_normal((2 * nq, 8, 128)), "f16"), torch.float16)
    plain = kv.attend(q, cache, table, lens, 32, "f16", [nq, nq])
    wide = torch.full((2 * nq, 13, 136), float("nan"), dtype=torch.float16, device="cuda")
    wide[:, 3:11, :128] = q
    for view in (wide[:, 3:11, :128], q.transpose(0, 1).contiguous().transpose(0, 1)):
        assert torch.equal(plain, kv.attend(view, cache, table, lens, 32, "f16", [nq, nq]))


@pytest.mark.parametrize("dim,seqs,nq,ln", [(64, 2, 2048, 8000), (128, 2, 2048, 8192), (256, 2, 500, 4000), (64, 24, 30, 9000),
                                            (128, 24, 30, 9000), (128, 16, 5, 4001), (64, 48, 1, 9000)])
def test_same_bits_over_many_launches(lib, dim, seqs, nq, ln):
    # Enough work for every SM and enough launches to meet a rare order of
    # copies, decoding and products.
    from gptq_post_weight_gb300 import _lib

    g = torch.Generator(device="cuda").manual_seed(81)
    heads, group, page = 8, 4, 64
    per = -(-ln // page)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    cache = _lib.kv4_cache(seqs * per, heads, dim, page)
    table = torch.randperm(seqs * per, generator=g, device="cuda").to(torch.int32).view(seqs, per)
    for b in range(seqs):
        slots = (table[b].long().unsqueeze(1) * page + torch.arange(page, device="cuda")).flatten()
        _lib.kv4_write(cache, draw(per * page, heads, dim), draw(per * page, heads, dim), slots, page)
    lens = torch.randint(nq, ln + 1, (seqs,), generator=g, device="cuda", dtype=torch.int32)
    lens[0] = ln
    starts = torch.arange(0, seqs * nq + 1, nq, dtype=torch.int32, device="cuda")
    q = draw(seqs * nq, heads * group, dim)
    first = _lib.kv4_attention(q, cache, table, lens, page, q_starts=starts, max_q=nq)
    same = torch.ones((), dtype=torch.bool, device="cuda")
    for _ in range(80):
        same &= (_lib.kv4_attention(q, cache, table, lens, page, q_starts=starts, max_q=nq) == first).all()
    _lib.serve_check()
    assert same


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,rows,n", [(1, 5120, 17408), (2, 5120, 17408), (4, 4096, 14336), (8, 5120, 17408),
                                           (45, 14336, 4096), (300, 4096, 4096), (1500, 4099, 1056)])
def test_same_bits_of_the_product_over_many_launches(lib, tokens, rows, n, dtype):
    import test_gpu_linear as lin
    from gptq_post_weight_gb300 import _lib

    g = torch.Generator(device="cuda").manual_seed(82)
    x = torch.randn(tokens, n, generator=g, device="cuda").to(lin.DT[dtype])
    nib = torch.randint(0, 256, (rows * n // 2,), generator=g, device="cuda", dtype=torch.uint8)
    rungs = torch.randint(0, 32, (rows * n // 32,), generator=g, device="cuda", dtype=torch.uint8)
    tab = torch.rand(rows, 32, generator=g, device="cuda") * 0.01
    first = _lib.q4tp_linear(x, nib, rungs, tab)
    same = torch.ones((), dtype=torch.bool, device="cuda")
    for _ in range(300):
        same &= (_lib.q4tp_linear(x, nib, rungs, tab) == first).all()
    _lib.serve_check()
    assert same
