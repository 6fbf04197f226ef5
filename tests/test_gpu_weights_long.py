"""The weights of cached tokens where a context's length times the query heads of
a key head passes 32 bits.

Tolerance: as in test_gpu_evict.py, with lse given in f32: a weight
exp(scale q k - lse) is off by e = (D + 8) 2^-22 scale sum |q k| and 2^-22 of
|s| + |lse| + 4, relative; the sum over R rows rounds once a row, 2^-24 of it.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("length,queries", [(2_199_991, 1), (2_100_003, 2)])
def test_length_times_group_past_32_bits(lib, length, queries):
    from gptq_post_weight_gb300 import _lib

    dim, page, group = 64, 64, 1024
    assert length * group > 2 ** 31
    g = torch.Generator(device="cuda")
    g.manual_seed(length)
    per = -(-length // page)
    table = torch.randperm(per, generator=g, device="cuda").to(torch.int32).view(1, per)
    cache = _lib.kv4_cache(per, 1, dim, page)
    q = torch.randn(queries, group, dim, generator=g, device="cuda").bfloat16()
    pos = torch.arange(length, device="cuda")
    slots = table[0].long()[pos // page] * page + pos % page
    keys = torch.empty(length, dim, dtype=torch.bfloat16, device="cuda")
    for a in range(0, length, 1 << 20):
        s = slots[a:a + (1 << 20)].contiguous()
        k = torch.randn(len(s), 1, dim, generator=g, device="cuda").bfloat16()
        _lib.kv4_write(cache, k, k, s, page)
        keys[a:a + len(s)] = _lib.kv4_read(cache, s, dim, page, torch.bfloat16)[0][:, 0]
    lens = torch.tensor([length], dtype=torch.int32, device="cuda")
    starts, scale = torch.tensor([0, queries], dtype=torch.int32, device="cuda"), dim ** -0.5
    rows = q.double().view(-1, dim)
    # The last key that a row sees is its own query's.
    last = (length - queries + torch.arange(queries, device="cuda")).repeat_interleave(group).unsqueeze(1)
    lse = torch.full((queries * group,), -torch.inf, dtype=torch.float64, device="cuda")
    for a in range(0, length, 50_000):
        k = keys[a:a + 50_000].double()
        s = (rows @ k.t() * scale).masked_fill(pos[a:a + len(k)] > last, -torch.inf)
        lse = torch.logaddexp(lse, torch.logsumexp(s, -1))
    lse = lse.float().view(queries, group)

    weights = torch.ones(1, 1, per * page, device="cuda")
    _lib.kv4_attention_weights(weights, q, lse, cache, table, lens, page, starts, queries)
    _lib.serve_check()
    assert (weights[0, 0, length:] == 1).all()
    off = lse.double().view(-1, 1)
    for a in range(0, length, 50_000):
        k = keys[a:a + 50_000].double()
        s = (rows @ k.t() * scale).masked_fill(pos[a:a + len(k)] > last, -torch.inf)
        p = torch.exp(s - off)
        e = (dim + 8) * 2.0 ** -22 * scale * (rows.abs() @ k.abs().t()) + 2.0 ** -22 * (s.abs() + off.abs() + 4)
        want = 1 + p.sum(0)
        tol = torch.where(p > 0, p * e, 0.0).sum(0) + (queries * group + 1) * 2.0 ** -24 * want
        got = weights[0, 0, a:a + len(k)].double()
        assert ((got - want).abs() <= tol).all(), ((got - want).abs() - tol).max()
