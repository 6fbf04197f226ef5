"""The weights of cached tokens where a cached key has no numbers and lse is what the
attention over that cache returned, and what eviction does with them."""
import numpy as np
import pytest

from oracle import serve
from test_gpu_evict import starts_of
from test_gpu_kv4 import context, dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_lens", [None, [3, 2], [60, 7]])
def test_key_without_numbers_in_the_whole_sequence_of_calls(lib, q_lens):
    from gptq_post_weight_gb300 import _lib

    r = np.random.default_rng(51)
    lens, heads, dim, page = [300, 90], 2, 64, 16
    cache, table, lens_d, ks, vs = context(r, lens, heads, dim, page, "bf16")
    tokens = 2 if q_lens is None else sum(q_lens)
    q = dev(serve.round_to(r.standard_normal((tokens, 4 * heads, dim)), "bf16"), torch.bfloat16)
    starts, max_q = starts_of(q_lens)

    def calls():
        lse = torch.empty(tokens, 4 * heads, device="cuda")
        _lib.kv4_attention(q, cache, table, lens_d, page, starts, max_q, lse=lse)
        w = _lib.kv4_weights(table, page, heads)
        _lib.kv4_attention_weights(w, q, lse, cache, table, lens_d, page, starts, max_q)
        return lse, w

    clean_lse, clean = calls()
    at = 100
    slot = torch.tensor([int(table[0, at // page]) * page + at % page], device="cuda")
    k, v = _lib.kv4_read(cache, slot, dim, page, torch.bfloat16)
    k[0, 1, 7] = float("nan")
    _lib.kv4_write(cache, k, v, slot, page)
    lse, w = calls()
    rows = 1 if q_lens is None else q_lens[0]
    sees = torch.zeros(tokens, 4 * heads, dtype=torch.bool, device="cuda")
    sees[:rows, 4:] = True  # all of the first sequence's queries come after the key
    assert torch.isnan(lse[sees]).all() and torch.equal(lse[~sees], clean_lse[~sees])
    assert torch.isnan(w[0, 1, :lens[0]]).all() and not w[0, 1, lens[0]:].any()
    w[0, 1] = clean[0, 1]
    assert torch.equal(w, clean)

    w[0, 1, :lens[0]] = float("nan")
    kept, _, _ = _lib.kv4_evict(cache, table, lens_d, w, 40, page, recent=8)
    assert kept[0, 1].tolist() == list(range(32)) + list(range(292, 300))
    assert kept[0, 0].tolist() == serve.kept(clean[0, 0].cpu().numpy(), 300, 40, 8)
