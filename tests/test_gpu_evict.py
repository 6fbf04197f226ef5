"""The attention's logarithms of sums, the weights that cached tokens gather and
the eviction that goes by them, against the 64-bit oracle.

A score is off by at most e = (D + 8) 2^-22 scale sum |q k| (f32 sums of D
products).  lse: e, the sum's own roundings (n 2^-24 at worst), and its
logarithm's (2^-22 of |lse| + 4).  A weight exp(s - lse), lse given: relative e,
2^-22 of |s| + |lse| + 4 for the exponent's f32 arithmetic and the exponential;
the rows' sum rounds once a row (2^-24 of the sum).  Places, lengths and moved
bytes are exact.
"""
import numpy as np
import pytest

from oracle import serve
from test_gpu_kv4 import DT, context, dev, keys

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def starts_of(q_lens):
    if q_lens is None:
        return None, 1
    return dev(np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)), max(q_lens)


def score_error(q, ks, lens, group, scale, q_lens):
    """[rows, heads] largest e of a row's scores, and one array of e and |s| a row and head."""
    q, at, out = np.abs(np.asarray(q)), 0, []
    for b, ln in enumerate(lens):
        nq = 1 if q_lens is None else q_lens[b]
        for i in range(nq):
            m = max(ln - nq + i + 1, 0)
            out.append([(q.shape[2] + 8) * 2.0 ** -22 * abs(scale) * (np.abs(ks[b][:m, h // group]) @ q[at + i, h])
                        for h in range(q.shape[1])])
        at += nq
    return out


def one(lens, heads, group, dim, page, dtype, q_lens=None, seed=0, scale=None):
    """lse and weights of a call; returns what the attention was given and gave."""
    from gptq_post_weight_gb300 import _lib

    r = np.random.default_rng(seed)
    cache, table, lens_d, ks, vs = context(r, lens, heads, dim, page, dtype)
    hq, tokens = heads * group, len(lens) if q_lens is None else sum(q_lens)
    q = serve.round_to(r.standard_normal((tokens, hq, dim)), dtype)
    qd = dev(q, DT[dtype])
    starts, max_q = starts_of(q_lens)
    sc = dim ** -0.5 if scale is None else scale
    plain = _lib.kv4_attention(qd, cache, table, lens_d, page, starts, max_q, scale=scale)
    lse = torch.full((tokens, hq), 7.0, device="cuda")
    out = _lib.kv4_attention(qd, cache, table, lens_d, page, starts, max_q, scale=scale, lse=lse)
    assert torch.equal(plain, out)  # the outputs' bits do not depend on it
    want = serve.log_sums(q, ks, lens, group, sc, q_lens)
    es = score_error(q, ks, lens, group, sc, q_lens)
    e = np.array([[x.max() if len(x) else 0.0 for x in row] for row in es]).reshape(tokens, hq)
    got = lse.double().cpu().numpy()
    none = np.isneginf(want)
    np.testing.assert_array_equal(np.isneginf(got), none)
    tol = e + max(lens) * 2.0 ** -24 + 2.0 ** -22 * (np.abs(np.where(none, 0, want)) + 4)
    assert (np.abs(np.where(none, 0, got) - np.where(none, 0, want)) <= tol).all()

    cap = table.shape[1] * page
    before = r.uniform(0, 2, (len(lens), heads, cap)).astype(np.float32)
    weights = dev(before)
    assert _lib.kv4_attention_weights(weights, qd, lse, cache, table, lens_d, page, starts, max_q, scale=scale) is weights
    _lib.serve_check()
    add = serve.attention_weights(q, ks, lens, group, sc, np.where(none, 0, got), q_lens)
    w, at = weights.double().cpu().numpy(), 0
    for b, ln in enumerate(lens):
        nq = 1 if q_lens is None else q_lens[b]
        off = np.zeros((heads, ln))
        for i in range(nq):
            m = ln - nq + i + 1
            for h in range(hq):
                if m > 0:
                    s = ks[b][:m, h // group] @ q[at + i, h] * sc
                    p = np.exp(s - got[at + i, h])
                    off[h // group, :m] += p * (es[at + i][h] + 2.0 ** -22 * (np.abs(s) + abs(got[at + i, h]) + 4))
        at += nq
        total = add[b] + before[b, :, :ln]
        off += (nq * group + 1) * 2.0 ** -24 * total
        bad = ~(np.abs(w[b, :, :ln] - total) <= off)
        assert not bad.any(), (np.abs(w[b, :, :ln] - total)[bad].max(), off[bad].min(), np.argwhere(bad)[:5])
        np.testing.assert_array_equal(w[b, :, ln:], before[b, :, ln:])  # places past the end stay
    return qd, lse, cache, table, lens_d, starts, max_q


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (256, 32)])
@pytest.mark.parametrize("group", [1, 4, 5, 16])
def test_single_tokens(lib, dim, page, group, dtype):
    one([1, 2, 15, 16, 17, 63, 127, 128, 129, 0, 333], 2, group, dim, page, dtype, seed=dim + group)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q_lens,group", [([2, 1, 5], 4), ([7, 3, 1], 4), ([16, 0, 9], 4), ([40, 33, 20], 4),
                                          ([9, 2, 3], 37)])
def test_several_queries(lib, q_lens, group, dim, dtype):
    # The third sequence has fewer keys than queries where q_lens allow it: its
    # first queries see nothing.
    one([50, 129, 4], 2, group, dim, 16, dtype, q_lens, seed=4)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q_lens,lens", [([130, 65], [130, 300]), ([257], [257]), ([70, 200, 1], [1000, 200, 77])])
def test_prompt_chunks(lib, q_lens, lens, dim, dtype):
    one(lens, 2, 3, dim, 48, dtype, q_lens, seed=5)


@pytest.mark.parametrize("lens,heads,group,dim,page,dtype,q_lens", [
    ([20001, 3, 4096], 1, 8, 128, 64, "bf16", None), ([9001], 2, 4, 128, 16, "f16", [5]),
    ([9001, 700], 1, 2, 64, 16, "bf16", None), ([5000, 130], 1, 3, 256, 16, "f16", [4, 1]),
    ([3000, 2000], 1, 4, 128, 16, "bf16", [7, 8]), ([12000], 1, 4, 64, 16, "bf16", [20]),
    ([5000], 1, 4, 128, 16, "f16", [40]), ([150001], 1, 2, 64, 64, "f16", None), ([70000], 1, 16, 64, 64, "bf16", [9])])
def test_long_contexts(lib, lens, heads, group, dim, page, dtype, q_lens):
    one(lens, heads, group, dim, page, dtype, q_lens, seed=6)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_in_parts(lib, dim):
    # Few steps of keys and many query rows: the rows of a step are cut, and steps
    # that only the last rows see have fewer tiles of rows than parts.
    size = lib.gptq_kv4_attention_weights_workspace_bytes
    for lens, group, q_lens in (([900], 4, [600]), ([700, 300, 1500], 16, [80, 300, 70]), ([300], 300, None)):
        max_q = 1 if q_lens is None else max(q_lens)
        assert size(dim, 1, group, max_q, len(lens), -(-max(lens) // 16) * 16) > 0 or q_lens is None
        one(lens, 1, group, dim, 16, "bf16", q_lens, seed=19)


def test_given_workspace(lib):
    from gptq_post_weight_gb300 import _lib

    qd, lse, cache, table, lens, starts, max_q = one([900], 1, 4, 64, 16, "f16", [600], seed=21)
    want, got = _lib.kv4_weights(table, 16, 1), _lib.kv4_weights(table, 16, 1)
    _lib.kv4_attention_weights(want, qd, lse, cache, table, lens, 16, starts, max_q)
    ws = _lib.workspace(lib.gptq_kv4_attention_weights_workspace_bytes(64, 1, 4, max_q, 1, table.shape[1] * 16), "cuda")
    ws.fill_(0xFF)
    _lib.kv4_attention_weights(got, qd, lse, cache, table, lens, 16, starts, max_q, ws=ws)
    assert torch.equal(got, want)


def test_waits_of_the_weights_run_out(lib):
    from gptq_post_weight_gb300 import _lib

    for q_lens in (None, [3], [200]):
        qd, lse, cache, table, lens, starts, max_q = one([500], 2, 2, 128, 16, "bf16", q_lens, seed=22)
        want = _lib.kv4_weights(table, 16, 2)
        _lib.kv4_attention_weights(want, qd, lse, cache, table, lens, 16, starts, max_q)
        try:
            _lib.test_set_wait(1_000_000, no_loads=True)
            _lib.kv4_attention_weights(_lib.kv4_weights(table, 16, 2), qd, lse, cache, table, lens, 16, starts, max_q)
            with pytest.raises(_lib.GptqError) as ei:
                _lib.serve_check()
            assert ei.value.code == 6
        finally:
            _lib.test_set_wait()
        got = _lib.kv4_weights(table, 16, 2)
        _lib.kv4_attention_weights(got, qd, lse, cache, table, lens, 16, starts, max_q)
        _lib.serve_check()
        assert torch.equal(got, want)


def test_many_sequences(lib):
    r = np.random.default_rng(9)
    one([int(n) for n in r.integers(0, 40, 1500)], 1, 2, 64, 16, "bf16", seed=9)


def test_many_sequences_of_many_rows(lib):
    # More sequences than a launch takes, tiles of many rows (the longest has 160)
    # and parts of them; some sequences have no queries, some no keys.
    r = np.random.default_rng(10)
    q_lens = [int(n) for n in r.integers(0, 4, 700)]
    q_lens[3] = q_lens[600] = 10
    one([int(n) for n in r.integers(0, 30, 700)], 1, 16, 64, 16, "bf16", q_lens, seed=10)


def test_scales(lib):
    one([300], 1, 2, 128, 16, "bf16", seed=10, scale=3.0)
    one([77], 1, 2, 64, 16, "f16", [9], seed=11, scale=0.0)
    one([200], 1, 2, 64, 16, "bf16", [50], seed=12, scale=-0.2)
    one([90], 2, 2, 64, 16, "bf16", None, seed=13, scale=-0.2)


def test_a_row_s_weights_add_to_one(lib):
    from gptq_post_weight_gb300 import _lib

    for q_lens in (None, [6, 90]):
        r = np.random.default_rng(3)
        cache, table, lens, ks, vs = context(r, [1000, 3000], 2, 128, 64, "bf16")
        tokens = 2 if q_lens is None else sum(q_lens)
        q = dev(serve.round_to(r.standard_normal((tokens, 8, 128)), "bf16"), torch.bfloat16)
        starts, max_q = starts_of(q_lens)
        lse = torch.empty(tokens, 8, device="cuda")
        _lib.kv4_attention(q, cache, table, lens, 64, starts, max_q, lse=lse)
        w = _lib.kv4_weights(table, 64, 2)
        _lib.kv4_attention_weights(w, q, lse, cache, table, lens, 64, starts, max_q)
        n = np.array([1, 1] if q_lens is None else q_lens) * 4.0
        np.testing.assert_allclose(w.sum(-1).cpu().numpy(), np.stack([n, n], 1), rtol=1e-4)
        again = _lib.kv4_weights(table, 64, 2)
        _lib.kv4_attention_weights(again, q, lse, cache, table, lens, 64, starts, max_q)
        assert torch.equal(w, again)  # a fixed order


def test_keys_without_numbers_reach_their_own_place_only(lib):
    from gptq_post_weight_gb300 import _lib

    for q_lens in ([3], [60]):
        r = np.random.default_rng(12)
        cache, table, lens, ks, vs = context(r, [300], 1, 64, 16, "bf16")
        q = dev(serve.round_to(r.standard_normal((q_lens[0], 4, 64)), "bf16"), torch.bfloat16)
        starts, max_q = starts_of(q_lens)
        lse = torch.empty(q_lens[0], 4, device="cuda")
        _lib.kv4_attention(q, cache, table, lens, 16, starts, max_q, lse=lse)
        clean = _lib.kv4_weights(table, 16, 1)
        _lib.kv4_attention_weights(clean, q, lse, cache, table, lens, 16, starts, max_q)
        nan = torch.full((1, 1, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
        at = 100
        slot = torch.tensor([int(table[0, at // 16]) * 16 + at % 16], device="cuda")
        _lib.kv4_write(cache, nan, nan, slot, 16)
        w = _lib.kv4_weights(table, 16, 1)
        _lib.kv4_attention_weights(w, q, lse, cache, table, lens, 16, starts, max_q)
        assert torch.isnan(w[0, 0, at])
        w[0, 0, at] = clean[0, 0, at]
        assert torch.equal(w, clean)


def test_rows_of_no_sequence_and_tables_past_the_pool(lib):
    from gptq_post_weight_gb300 import _lib

    r = np.random.default_rng(14)
    cache, table, lens, ks, vs = context(r, [40, 90], 2, 64, 16, "bf16")
    q = dev(serve.round_to(r.standard_normal((20, 4, 64)), "bf16"), torch.bfloat16)
    starts = dev(np.array([3, 8, 15], dtype=np.int32))
    for max_q in (7, 4, 40):  # rows 0-2 and 15-19, and what passes max_q, are nobody's
        lse = torch.zeros(20, 4, device="cuda")
        out = _lib.kv4_attention(q, cache, table, lens, 16, starts, max_q, lse=lse)
        nobody = [0, 1, 2, 15, 16, 17, 18, 19] + ([7, 12, 13, 14] if max_q == 4 else [])
        mine = [i for i in range(20) if i not in nobody]
        assert torch.isneginf(lse[nobody]).all() and torch.isfinite(lse[mine]).all()
        assert not out[nobody].any()
        w = _lib.kv4_weights(table, 16, 2)
        _lib.kv4_attention_weights(w, q, lse, cache, table, lens, 16, starts, max_q)
        n = [min(5, max_q) * 2.0, min(7, max_q) * 2.0]
        np.testing.assert_allclose(w.sum(-1).cpu().numpy(), [[n[0]] * 2, [n[1]] * 2], rtol=1e-4)
    bad, zero = table.clone(), table.clone()
    bad[0, 1], bad[1, 2] = 1 << 30, -5
    zero[0, 1] = zero[1, 2] = 0
    one_each = q[:2]
    lse = torch.zeros(2, 4, device="cuda")
    got, want = _lib.kv4_weights(table, 16, 2), _lib.kv4_weights(table, 16, 2)
    _lib.kv4_attention_weights(got, one_each, lse, cache, bad, lens, 16)
    _lib.kv4_attention_weights(want, one_each, lse, cache, zero, lens, 16)
    assert torch.equal(got.view(torch.int32), want.view(torch.int32))
    # Lengths past the table count as its capacity.
    full = torch.full_like(lens, table.shape[1] * 16)
    got, want = _lib.kv4_weights(table, 16, 2), _lib.kv4_weights(table, 16, 2)
    _lib.kv4_attention_weights(got, one_each, lse, cache, table, full + 1000, 16)
    _lib.kv4_attention_weights(want, one_each, lse, cache, table, full, 16)
    assert torch.equal(got.view(torch.int32), want.view(torch.int32))


def test_no_sequences_and_no_queries(lib):
    from gptq_post_weight_gb300 import _lib

    cache = _lib.kv4_cache(2, 2, 64, 16)
    q = torch.ones(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    none, table = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, 1, dtype=torch.int32, device="cuda")
    starts = torch.zeros(1, dtype=torch.int32, device="cuda")
    lse = torch.zeros(3, 4, device="cuda")
    out = _lib.kv4_attention(q, cache, table, none, 16, starts, 1, lse=lse)
    assert not out.any() and torch.isneginf(lse).all()
    _lib.kv4_attention_weights(torch.empty(0, 2, 16, device="cuda"), q, lse, cache, table, none, 16, starts, 1)
    kept, lens, w = _lib.kv4_evict(cache, table, none, torch.empty(0, 2, 16, device="cuda"), 4, 16)
    assert kept.shape == (0, 2, 4) and lens.shape == (0,) and w.shape == (0, 2, 16)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    one_len = torch.ones(1, dtype=torch.int32, device="cuda")
    w = torch.ones(1, 2, 16, device="cuda")
    _lib.kv4_attention_weights(w, q[:0], lse[:0], cache, table, one_len, 16, torch.zeros(2, dtype=torch.int32, device="cuda"), 1)
    assert (w == 1).all()


def test_strided_queries_stream_capture(lib):
    from gptq_post_weight_gb300 import _lib

    for q_lens in (None, [40, 3]):
        qd, lse, cache, table, lens, starts, max_q = one([300, 18], 2, 4, 128, 16, "f16", q_lens, seed=13)
        want = _lib.kv4_weights(table, 16, 2)
        _lib.kv4_attention_weights(want, qd, lse, cache, table, lens, 16, starts, max_q)
        wide = torch.full((qd.shape[0], 12, 136), float("nan"), dtype=torch.float16, device="cuda")
        wide[:, 2:10, :128] = qd
        got = _lib.kv4_weights(table, 16, 2)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        _lib.kv4_attention_weights(got, wide[:, 2:10, :128], lse, cache, table, lens, 16, starts, max_q, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _lib.kv4_attention(qd, cache, table, lens, 16, starts, max_q, lse=lse)
            _lib.kv4_attention_weights(got, qd, lse, cache, table, lens, 16, starts, max_q)
        got.zero_()
        g.replay()
        assert torch.equal(got, want)


# ---------------------------------------------------------------- eviction


def heavy(r, shape):
    """Weights as attention leaves them, with zeros and ties."""
    w = np.exp(2.5 * r.standard_normal(shape)).astype(np.float32)
    w[r.uniform(size=shape) < 0.2] = 0
    return np.where(r.uniform(size=shape) < 0.3, np.round(w * 2) / 2, w).astype(np.float32)


def evict(lens, heads, dim, page, keep, recent, other, seed=0, weights=None, out_pages=None):
    from gptq_post_weight_gb300 import _lib

    r = np.random.default_rng(seed)
    per = max(max(-(-n // page) for n in lens), -(-keep // page) if not other else 1, 1)
    to = (out_pages or -(-keep // page)) if other else 0
    pages = len(lens) * (per + to) + 2
    order = r.permutation(pages).astype(np.int32)
    table = order[:len(lens) * per].reshape(len(lens), per)
    out = order[len(lens) * per:len(lens) * (per + to)].reshape(len(lens), to) if other else None
    raw = r.integers(0, 256, (pages, heads, page // 16, 20 * dim), dtype=np.uint8)
    w = heavy(r, (len(lens), heads, per * page)) if weights is None else weights(r, (len(lens), heads, per * page))
    cache = dev(raw.reshape(pages, heads, -1))
    wd = dev(w)
    kept, lens_out, w_out = _lib.kv4_evict(cache, dev(table), dev(np.array(lens, dtype=np.int32)), wd, keep, page,
                                           recent=recent, out_table=None if out is None else dev(out))
    dst = table if out is None else out
    want, want_w = raw.copy(), np.zeros((len(lens), heads, dst.shape[1] * page), dtype=np.float32)
    want_kept = np.full((len(lens), heads, keep), -1, dtype=np.int32)
    pieces = [(0, dim // 2), (8 * dim, dim // 8), (10 * dim, dim // 2), (18 * dim, dim // 8)]
    for b, n in enumerate(lens):
        for h in range(heads):
            places = serve.kept(w[b, h], n, keep, recent)
            want_kept[b, h, :len(places)] = places
            want_w[b, h, :len(places)] = w[b, h, places]
            for i, t in enumerate(places):
                for at, size in pieces:
                    want[dst[b, i // page], h, i % page // 16, at + i % 16 * size:at + (i % 16 + 1) * size] = \
                        raw[table[b, t // page], h, t % page // 16, at + t % 16 * size:at + (t % 16 + 1) * size]
    np.testing.assert_array_equal(kept.cpu().numpy(), want_kept)
    np.testing.assert_array_equal(lens_out.cpu().numpy(), np.minimum(lens, keep))
    np.testing.assert_array_equal(w_out.cpu().numpy(), want_w)
    assert torch.equal(wd.view(torch.int32), dev(w).view(torch.int32))  # (bits: a NaN equals itself)
    np.testing.assert_array_equal(cache.cpu().numpy().reshape(raw.shape), want)  # every byte of the pool
    return kept


@pytest.mark.parametrize("other", [False, True])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 48), (256, 32)])
@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 5), (16, 4), (33, 0), (50, 50), (64, 7)])
def test_evict(lib, keep, recent, dim, page, other):
    evict([0, 1, 15, 16, 17, 33, 64, 65, 200, 64], 2, dim, page, keep, recent, other, seed=dim + keep)


@pytest.mark.parametrize("other", [False, True])
@pytest.mark.parametrize("lens,heads,dim,keep,recent", [
    ([5000], 3, 128, 1000, 64), ([3001, 2500], 1, 64, 2400, 0), ([1030, 1024, 1023], 2, 256, 1023, 31),
    ([20000], 1, 64, 700, 1), ([4100], 1, 128, 4099, 10), ([2500], 9, 64, 2000, 1999),
    ([45000, 100], 1, 64, 3000, 16)])  # (the last: more places than the selection keeps in shared memory)
def test_evict_long(lib, lens, heads, dim, keep, recent, other):
    evict(lens, heads, dim, 16, keep, recent, other, seed=keep)


@pytest.mark.parametrize("other", [False, True])
def test_many_heads(lib, other):
    """More heads than start at once, of unequal lengths; weights of either sign, zeros of either, NaN."""
    def weights(r, shape):
        w = heavy(r, shape) * np.where(r.uniform(size=shape) < 0.3, -1, 1).astype(np.float32)
        return np.where(r.uniform(size=shape) < 0.02, np.float32(np.nan), w)

    lens = [0, 1, 99, 100, 101, 513, 1500, 1040] + [int(n) for n in np.random.default_rng(4).integers(0, 700, 70)]
    evict(lens, 8, 64, 16, 100, 7, other, seed=3, weights=weights)


def test_ties_nan_and_signs(lib):
    evict([700], 2, 64, 16, 100, 10, False, weights=lambda r, s: np.zeros(s, np.float32))
    evict([700], 2, 64, 16, 100, 10, True, weights=lambda r, s: np.full(s, 3.5, np.float32))

    def odd(r, s):
        v = np.array([np.nan, -np.nan, np.inf, -np.inf, 0.0, -0.0, 1.0, -1.0, 1e-42, -1e-42, 3e38], np.float32)
        return v[r.integers(0, len(v), s)]

    evict([900, 40], 2, 64, 16, 300, 0, False, seed=1, weights=lambda r, s: np.where(np.isnan(odd(r, s)), -2.0, odd(r, s)).astype(np.float32))
    from gptq_post_weight_gb300 import _lib

    w = odd(np.random.default_rng(5), (1, 1, 512))
    cache = _lib.kv4_cache(32, 1, 64, 16)
    table = torch.arange(32, dtype=torch.int32, device="cuda").view(1, 32)
    for keep in (5, 100, 400, 500):
        kept, _, _ = _lib.kv4_evict(cache, table, torch.tensor([512], dtype=torch.int32, device="cuda"), dev(w), keep, 16)
        assert kept[0, 0].tolist() == serve.kept(w[0, 0], 512, keep, 0)


def test_roomy_outputs_and_same_result_again(lib):
    a = evict([300, 20], 2, 128, 16, 100, 8, True, seed=3, out_pages=11)
    b = evict([300, 20], 2, 128, 16, 100, 8, True, seed=3, out_pages=11)
    assert torch.equal(a, b)


def test_shared_pages_only_lose(lib):
    # Two sequences that share a prefix's pages are cut into pages of their own.
    from gptq_post_weight_gb300 import _lib

    r = np.random.default_rng(8)
    raw = r.integers(0, 256, (20, 2, 16 * 80), dtype=np.uint8)
    cache = dev(raw)
    table = dev(np.array([[0, 1, 2, 3], [0, 1, 2, 4]], dtype=np.int32))
    out = dev(np.array([[10, 11], [12, 13]], dtype=np.int32))
    lens = dev(np.array([64, 60], dtype=np.int32))
    w = dev(heavy(r, (2, 2, 64)))
    kept, _, _ = _lib.kv4_evict(cache, table, lens, w, 20, 16, recent=4, out_table=out)
    got = cache.cpu().numpy()
    np.testing.assert_array_equal(got[:10], raw[:10])
    blocks, was = got.reshape(20, 2, 16 * 80), raw.reshape(20, 2, 16 * 80)
    for b in range(2):
        for h in range(2):
            for i, t in enumerate(kept[b, h].tolist()):
                d, s = blocks[int(out[b, i // 16]), h], was[int(table[b, t // 16]), h]
                np.testing.assert_array_equal(d[i % 16 * 32:i % 16 * 32 + 32], s[t % 16 * 32:t % 16 * 32 + 32])


def test_pages_outside_the_pool_take_nothing(lib):
    from gptq_post_weight_gb300 import _lib

    r = np.random.default_rng(9)
    raw = r.integers(0, 256, (9, 1, 16 * 80), dtype=np.uint8)
    cache = dev(raw)
    table = dev(np.array([[2, 3, 4]], dtype=np.int32))
    out = dev(np.array([[1 << 30, 6], ], dtype=np.int32))
    w = dev(heavy(r, (1, 1, 48)))
    _lib.kv4_evict(cache, table, dev(np.array([48], dtype=np.int32)), w, 30, 16, out_table=out)
    got = cache.cpu().numpy()
    np.testing.assert_array_equal(got[[0, 1, 2, 3, 4, 5, 7, 8]], raw[[0, 1, 2, 3, 4, 5, 7, 8]])
    assert (got[6] != raw[6]).any()


def test_evict_stream_and_capture(lib):
    from gptq_post_weight_gb300 import _lib

    r = np.random.default_rng(10)
    raw = dev(r.integers(0, 256, (16, 2, 16 * 160), dtype=np.uint8))
    table = dev(r.permutation(16).astype(np.int32).reshape(2, 8))
    lens = dev(np.array([128, 100], dtype=np.int32))
    w = dev(heavy(r, (2, 2, 128)))
    cache = raw.clone()
    want = _lib.kv4_evict(cache, table, lens, w, 40, 16, recent=3)
    side = torch.cuda.Stream()
    again = raw.clone()
    side.wait_stream(torch.cuda.current_stream())
    got = _lib.kv4_evict(again, table, lens, w, 40, 16, recent=3, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(again, cache) and all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = _lib.kv4_evict(again, table, lens, w, 40, 16, recent=3)
    again.copy_(raw)
    g.replay()
    assert torch.equal(again, cache) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_past_32_bits(lib):
    # A pool past 2^32 bytes: tokens come from its end and go there.
    from gptq_post_weight_gb300 import _lib

    heads, dim, page = 8, 128, 64
    per = heads * page * dim * 5 // 4
    pages = (1 << 32) // per + 100
    cache = torch.zeros(pages, heads, page * dim * 5 // 4, dtype=torch.uint8, device="cuda")
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device="cuda")
    r = np.random.default_rng(11)
    for p in table[0].tolist():
        cache[p] = dev(r.integers(0, 256, tuple(cache.shape[1:]), dtype=np.uint8))
    small = cache[table[0].long()].clone()
    w = dev(heavy(r, (1, heads, 3 * page)))
    lens = torch.tensor([190], dtype=torch.int32, device="cuda")
    kept, _, _ = _lib.kv4_evict(cache, table, lens, w, 100, page, recent=10)
    kept2, _, _ = _lib.kv4_evict(small, torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda"), lens, w, 100, page,
                                 recent=10)
    assert torch.equal(kept, kept2) and torch.equal(cache[table[0].long()], small)
    k = keys(r, (1, 8, dim), "bf16")
    q, lse = dev(k, torch.bfloat16), torch.zeros(1, 8, device="cuda")
    a, b = _lib.kv4_weights(table, page, heads), _lib.kv4_weights(table, page, heads)
    _lib.kv4_attention_weights(a, q, lse, cache, table, lens, page)
    _lib.kv4_attention_weights(b, q, lse, small, torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda"), lens, page)
    assert torch.equal(a.view(torch.int32), b.view(torch.int32))
