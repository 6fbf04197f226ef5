"""gptq_kv4_evict with tables wider than any sequence: what a narrow table gives
(test_gpu_evict.py has that against the oracle), bit for bit, whichever way the
selection keeps a head's weights and however many heads there are.
"""
import numpy as np
import pytest

from test_gpu_evict import dev, heavy

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("other", [False, True])
@pytest.mark.parametrize("seqs", [3, 40])
@pytest.mark.parametrize("places", [17008, 41504])
def test_table_wider_than_the_sequences(lib, places, seqs, other):
    from gptq_post_weight_gb300 import _lib

    heads, dim, page, keep, recent = 8, 64, 16, 90, 5
    r = np.random.default_rng(places + seqs)
    lens = r.integers(0, 700, seqs).astype(np.int32)
    lens[0] = 700
    per, to = -(-700 // page), -(-keep // page)
    pages = seqs * (per + to)
    order = r.permutation(pages).astype(np.int32)
    narrow = order[:seqs * per].reshape(seqs, per)
    wide = np.zeros((seqs, places // page), dtype=np.int32)
    wide[:, :per] = narrow
    out = dev(order[seqs * per:].reshape(seqs, to)) if other else None
    w = np.full((seqs, heads, places), 1e30, dtype=np.float32)  # past the end: nobody's
    w[..., :per * page] = heavy(r, (seqs, heads, per * page))
    raw = dev(r.integers(0, 256, (pages, heads, page * dim * 5 // 4), dtype=np.uint8))
    got = []
    for table in (narrow, wide):
        cache = raw.clone()
        kept, n, left = _lib.kv4_evict(cache, dev(table), dev(lens), dev(np.ascontiguousarray(w[..., :table.shape[1] * page])),
                                       keep, page, recent=recent, out_table=out)
        got.append((cache, kept, n, left))
    a, b = got
    assert all(torch.equal(x, y) for x, y in zip(a[:3], b[:3]))
    assert torch.equal(a[3], b[3][..., :a[3].shape[2]]) and not b[3][..., a[3].shape[2]:].any()
    assert not torch.equal(a[0], raw)
