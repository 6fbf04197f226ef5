"""The calls for rotary positions, the gated product, attention weights and
eviction refuse what they cannot use before anything is launched (CPU only),
and hand the library what they were given."""
import ctypes
import math

import pytest

from test_serve_binding import Gpu, Stream, gpu, rec, weights  # noqa: F401
from test_serve_checks import b16, blib, refused, u8  # noqa: F401

torch = pytest.importorskip("torch")


def i64(*v):
    return torch.tensor(v, dtype=torch.int64)


def test_frequencies(blib):  # noqa: F811
    f = blib.rotary_frequencies(64)
    assert len(f) == 32 and f[0] == 1.0 and f[-1] == 10000.0 ** (-62 / 64)
    lin = blib.rotary_frequencies(64, scaling="linear", factor=4)
    assert lin == [v / 4 for v in f]
    base = blib.rotary_frequencies(64, scaling="base", factor=4)
    assert base[0] == 1.0 and abs(base[-1] * 4 / f[-1] - 1) < 1e-12
    ramp = blib.rotary_frequencies(64, scaling="ramp", factor=4, length=1000, low=1, high=4)
    for v, w in zip(f, ramp):
        turns = 1000 * v / (2 * math.pi)
        part = min(max((turns - 1) / 3, 0), 1)
        assert abs(w - (part * v + (1 - part) * v / 4)) <= 1e-15
    assert ramp[0] == 1.0 and ramp[-1] == f[-1] / 4
    refused(blib.rotary_frequencies, 63, match="rot must be")
    refused(blib.rotary_frequencies, 0, match="rot must be")
    refused(blib.rotary_frequencies, 64, scaling="other", match="scaling must be one of")
    refused(blib.rotary_frequencies, 2, scaling="base", match="rot of 4")
    refused(blib.rotary_frequencies, 64, factor=0.0, match="must be positive")
    refused(blib.rotary_frequencies, 64, scaling="ramp", low=4, high=4, match="high above low")


def test_turns(blib):  # noqa: F811
    t = blib.rotary_turns([1.0, math.pi, -math.pi / 2, 2 * math.pi, 0.0], device="cpu")
    assert t.dtype == torch.int64
    v = [x / 2 ** 64 for x in t.tolist()]
    assert abs(v[0] - 1 / (2 * math.pi)) < 1e-15 and v[1] == -0.5 and v[2] == -0.25 and v[3] == 0 and v[4] == 0
    refused(blib.rotary_turns, [], device="cpu", match="finite numbers")
    refused(blib.rotary_turns, [1.0, float("inf")], device="cpu", match="finite numbers")


def test_rotary(blib):  # noqa: F811
    f, x, p, t = blib.rotary, b16(3, 4, 64), i64(1, 2, 3), torch.zeros(16, dtype=torch.int64)
    refused(f, x.float(), p, t, match="x must be torch.bfloat16")
    refused(f, x[0], p, t, match="3-D")
    refused(f, b16(3, 4, 72), p, t, match="multiple of 16 channels")
    refused(f, b16(3, 4, 1040), p, t, match="at most 1024")
    refused(f, b16(3, 0, 64), p, t, match="multiple of 16 channels")
    refused(f, b16(3, 4, 128)[..., ::2], p, t, match="contiguous in its last")
    refused(f, b16(3, 4, 68)[..., :64], p, t, match="multiple of 8 elements")
    refused(f, x, p[:2], t, match="positions must have 3")
    refused(f, x, p.int(), t, match="positions must be torch.int64")
    refused(f, x, p, t[:15], match="turns must have a multiple of 8")
    refused(f, x, p, torch.zeros(40, dtype=torch.int64), match="up to 32")
    refused(f, x, p, t.double(), match="turns must be torch.int64")
    refused(f, x, p, t, layout="pairs", match="layout must be one of")
    refused(f, x, p, t, gain=float("nan"), match="gain must be finite")
    refused(f, x, p, t, out=b16(3, 4, 32), match="out must have shape")
    refused(f, x, p, t, out=b16(1, 4, 64).expand(3, 4, 64), match="do not overlap")
    refused(f, x, p, t, out=torch.as_strided(b16(1000), (3, 4, 64), (64, 64, 1)), match="do not overlap")
    flat = b16(2000)
    refused(f, torch.as_strided(flat, (3, 4, 64), (256, 64, 1)), p, t, out=torch.as_strided(flat, (3, 4, 64), (512, 64, 1)),
            match="the input with other strides")
    # In place, the rows may not overlap either.
    rows = b16(1, 4, 64).expand(3, 4, 64)
    refused(f, rows, p, t, out=rows, match="out must have rows that do not overlap")
    refused(f, x.clone().requires_grad_(), p, t, match="requires a gradient")
    refused(f, x, p, t, match="CUDA tensors")


def test_write_rotary(blib):  # noqa: F811
    f, cache = blib.kv4_write_rotary, u8(4, 2, 16 * 64 * 5 // 4)
    q, k, s, p, t = b16(5, 8, 64), b16(5, 2, 64), torch.zeros(5, dtype=torch.int64), i64(0, 1, 2, 3, 4), torch.zeros(32, dtype=torch.int64)
    refused(f, cache, q, k.float(), k, s, 16, p, t, match="k must be")
    refused(f, cache, q, k, b16(5, 2, 128), s, 16, p, t, match="v must have shape")
    refused(f, cache, q, b16(5, 3, 64), b16(5, 3, 64), s, 16, p, t, match="3 heads, the cache 2")
    refused(f, cache, q.half(), k, k, s, 16, p, t, match="q must be torch.bfloat16")
    refused(f, cache, None, k, k, s, 16, p, t, match="q must be a torch tensor")
    refused(f, cache, b16(4, 8, 64), k, k, s, 16, p, t, match=r"q must be \[5, heads, 64\]")
    refused(f, cache, b16(5, 0, 64), k, k, s, 16, p, t, match=r"q must be \[5, heads, 64\]")
    refused(f, cache, q, k, k, s[:4], 16, p, t, match="slots must have 5")
    refused(f, cache, q, k, k, s, 16, p[:4], t, match="positions must have 5")
    refused(f, cache, q, k, k, s, 16, p, t[:4], match="turns must have")
    refused(f, cache, q, k, k, s, 16, p, t, out=b16(5, 8, 32), match="out must have shape")
    refused(f, cache, q, k, k.clone().requires_grad_(), s, 16, p, t, match="v requires a gradient")
    refused(f, cache, q, k, k, s, 16, p, t, match="CUDA tensors")


def test_gated(blib):  # noqa: F811
    t, rows, n = 3, 6, 64
    x, nib, rungs, tab = b16(t, n), u8(rows * n // 2), u8(rows * 2), torch.zeros(rows, 32)
    f = blib.q4tp_gated
    refused(f, x.float(), nib, rungs, tab, match="x must be torch.bfloat16")
    refused(f, x, nib[:-1], rungs, tab, match="nibbles must have 192")
    refused(f, x, nib, rungs, tab, bias=b16(3), match="bias must have 6")
    refused(f, x, nib, rungs, tab, act="swish", match="act must be one of")
    refused(f, x, nib, rungs, tab, match="CUDA tensors")
    odd = (u8(5 * n // 2), u8(10), torch.zeros(5, 32))
    refused(f, x, *odd, match="as many of the up projection")
    refused(f, x, nib, rungs, tab, out=b16(t, 6), match="out must have shape")
    refused(f, x, nib, rungs, tab, ws=torch.zeros(4), match="ws must be")
    refused(f, x, nib, rungs, tab, out=b16(3, t).t(), match="dense rows")
    refused(f, x.clone().requires_grad_(), nib, rungs, tab, match="requires a gradient")


def test_attention_weights_and_lse(blib):  # noqa: F811
    cache = u8(4, 2, 16 * 64 * 5 // 4)
    q, table, lens = b16(3, 4, 64), torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    lse, w = torch.zeros(3, 4), torch.zeros(3, 2, 32)
    refused(blib.kv4_attention, q, cache, table, lens, 16, lse=torch.zeros(3, 3), match="lse must have 12")
    refused(blib.kv4_attention, q, cache, table, lens, 16, lse=lse.double(), match="lse must be torch.float32")
    f = blib.kv4_attention_weights
    refused(f, w, q.float(), lse, cache, table, lens, 16, match="q must be")
    refused(f, w, q, lse[:2], cache, table, lens, 16, match="lse must have 12")
    refused(f, w, q, None, cache, table, lens, 16, match="lse must be a torch tensor")
    refused(f, w, q, lse, cache, table[:2], lens[:2], 16, match="one query a sequence")
    refused(f, w, q, lse, cache, table, lens, 16, ws=torch.zeros(4), match="ws must be")
    refused(f, w[:, :1], q, lse, cache, table, lens, 16, match="weights must be")
    refused(f, w.double(), q, lse, cache, table, lens, 16, match="weights must be torch.float32")
    refused(f, w, q.clone().requires_grad_(), lse, cache, table, lens, 16, match="q requires a gradient")
    refused(f, w.clone().requires_grad_(), q, lse, cache, table, lens, 16, match="weights requires a gradient")
    refused(f, w, q, lse, cache, table, lens, 16, match="CUDA tensors")
    assert blib.kv4_weights(table, 16, 2).shape == (3, 2, 32)


def test_evict(blib):  # noqa: F811
    cache = u8(9, 2, 16 * 64 * 5 // 4)
    table, lens, w = torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32), torch.zeros(3, 2, 32)
    f = blib.kv4_evict
    refused(f, cache.int(), table, lens, w, 4, 16, match="cache must be")
    refused(f, cache, table, lens, w, 4, 24, match="cache must be a pool|page_size must be|dim must be")
    refused(f, cache, table, lens, w, 4, 0, match="cache must be a pool")
    refused(f, cache, table.long(), lens, w, 4, 16, match="table must be torch.int32")
    refused(f, cache, table, lens[:2], w, 4, 16, match="kv_lens must have 3")
    refused(f, cache, table, lens, w[:, :, :16], 4, 16, match="weights must be")
    refused(f, cache, table, lens, w.half(), 4, 16, match="weights must be torch.float32")
    refused(f, cache, table, lens, w, 0, 16, match="keep must be 1 to 32")
    refused(f, cache, table, lens, w, 33, 16, match="keep must be 1 to 32")
    refused(f, cache, table, lens, w, 4, 16, recent=-1, match="recent must not be negative")
    out = torch.zeros(3, 1, dtype=torch.int32)
    refused(f, cache, table, lens, w, 17, 16, out_table=out, match="keep must be 1 to 16")
    refused(f, cache, table, lens, w, 4, 16, out_table=table, match="out_table is table")
    refused(f, cache, table, lens, w, 4, 16, out_table=out[:2], match="out_table must be")
    refused(f, cache, table, lens, w, 4, 16, out_table=out.long(), match="out_table must be torch.int32")
    refused(f, cache, table, lens, w.clone().requires_grad_(), 4, 16, match="requires a gradient")
    refused(f, cache, table, lens, w, 4, 16, match="CUDA tensors")


def test_c_entries(blib):  # noqa: F811
    lib = blib.load()
    P = ctypes.c_void_p
    ok, mis = P(1 << 20), P((1 << 20) + 4)

    def rotary(dt=0, x=ok, xt=256, xh=64, t=3, h=4, d=64, rot=64, lay=0, p=ok, gain=1.0, y=P(1 << 21), yt=256):
        return lib.gptq_rotary(dt, x, xt, xh, t, h, d, rot, lay, p, ok, gain, y, yt, 64, None)

    assert rotary(t=-1) == 2 and rotary(h=0) == 2 and rotary(h=70000) == 2 and rotary(d=72) == 2 and rotary(d=2048) == 2
    assert rotary(rot=0) == 2 and rotary(rot=24) == 2 and rotary(rot=80) == 2 and rotary(lay=2) == 2
    assert rotary(xt=12) == 2 and rotary(yt=-8) == 2 and rotary(y=ok, yt=512) == 2
    assert rotary(dt=2) == 1 and rotary(gain=float("inf")) == 1 and rotary(x=mis) == 1 and rotary(p=None) == 1
    assert rotary(t=0, x=None) == 0

    def write(dt=0, cache=ok, d=64, page=16, q=ok, hq=4, k=ok, slots=ok, t=5, rot=64, lay=0, p=ok, y=P(1 << 21), yt=256):
        return lib.gptq_kv4_write_rotary(dt, cache, 4, 2, d, page, q, 256, 64, hq, k, ok, 128, 64, 128, 64, slots, t, rot,
                                         lay, p, ok, 1.0, y, yt, 64, None)

    assert write(d=96) == 2 and write(page=24) == 2 and write(hq=0) == 2 and write(rot=8) == 2 and write(lay=-1) == 2
    assert write(t=1 << 21) == 2 and write(yt=4) == 2 and write(y=ok, yt=512) == 2
    assert write(dt=5) == 1 and write(cache=None) == 1 and write(q=mis) == 1 and write(k=None) == 1
    assert write(slots=None) == 1 and write(p=None) == 1 and write(t=0, q=None) == 0

    def gated(dt=0, x=ok, ldx=64, t=3, nib=ok, inner=6, n=64, act=4, bias=None, y=ok, ldy=6, ws=None, wn=0):
        return lib.gptq_q4tp_gated(dt, x, ldx, t, nib, ok, ok, inner, n, bias, act, y, ldy, ws, wn, None, None)

    need = lib.gptq_q4tp_gated_workspace_bytes(0, 9, 64)
    assert need >= 9 * (64 * 2 + 4) and gated(t=9) == 3 and gated(t=9, ws=ok, wn=need - 1) == 3 and gated(t=9, ws=mis, wn=need) == 1
    assert lib.gptq_q4tp_gated_workspace_bytes(0, 8, 64) == 0 and lib.gptq_q4tp_gated_workspace_bytes(1, 100, 64) == 0
    assert lib.gptq_q4tp_gated_workspace_bytes(2, 100, 64) == 0 and lib.gptq_q4tp_gated_workspace_bytes(0, -1, 64) == 0

    assert gated(n=48, ldx=48) == 2 and gated(t=-1) == 2 and gated(inner=0) == 2 and gated(inner=(1 << 23) + 1) == 2
    assert gated(ldx=32) == 2 and gated(ldx=68) == 2 and gated(ldy=5) == 2
    assert gated(dt=2) == 1 and gated(act=5) == 1 and gated(x=None) == 1 and gated(nib=mis) == 1 and gated(bias=mis) == 1
    assert gated(t=0, x=None, y=None) == 0

    def weigh(dt=0, q=ok, qt=256, tq=3, lse=ok, group=2, stride=2, lens=ok, starts=None, seqs=3, max_q=1, scale=1.0, w=ok, ws=None,
              wn=0):
        return lib.gptq_kv4_attention_weights(dt, q, qt, 64, tq, lse, ok, 4, 2, group, 64, 16, ok, stride, lens, starts,
                                              seqs, max_q, scale, w, ws, wn, None, None)

    size = lib.gptq_kv4_attention_weights_workspace_bytes
    need = size(64, 2, 2, 5000, 3, 32)
    assert need > 0 and need % (3 * 2 * 32 * 4) == 0
    assert weigh(starts=ok, max_q=5000) == 3 and weigh(starts=ok, max_q=5000, ws=ok, wn=need - 1) == 3
    assert weigh(starts=ok, max_q=5000, ws=mis, wn=need) == 1
    assert size(64, 2, 2, 16, 3, 32) == 0 and size(96, 2, 2, 5000, 3, 32) == 0 and size(64, 2, 2, 5000, 0, 32) == 0
    assert size(64, 8, 4, 2048, 400, 1 << 15) == 0  # enough steps for every SM
    assert size(64, 1024, 1024, 1 << 20, 1 << 20, 1 << 30) == 0

    assert weigh(group=0) == 2 and weigh(stride=0) == 2 and weigh(tq=4) == 2 and weigh(max_q=2) == 2 and weigh(qt=4) == 2
    assert weigh(dt=3) == 1 and weigh(scale=float("nan")) == 1 and weigh(q=mis) == 1 and weigh(lse=None) == 1
    assert weigh(w=None) == 1 and weigh(lens=None) == 1 and weigh(tq=0, starts=ok) == 0 and weigh(seqs=0, starts=ok) == 0

    def evict(cache=ok, pages=4, heads=2, d=64, page=16, stride=2, out=None, out_stride=0, lens=ok, seqs=3, w=ok, keep=8,
              recent=0, kept=ok):
        return lib.gptq_kv4_evict(cache, pages, heads, d, page, ok, stride, out, out_stride, lens, seqs, w, keep, recent,
                                  kept, ok, ok, None)

    assert evict(d=32) == 2 and evict(page=8) == 2 and evict(stride=0) == 2 and evict(keep=0) == 2 and evict(keep=33) == 2
    other = P(1 << 22)
    assert evict(recent=-1) == 2 and evict(out=other) == 2 and evict(out=other, out_stride=1, keep=17) == 2
    assert evict(seqs=1 << 20, heads=1000) == 2
    assert evict(out=ok, out_stride=2) == 1  # table itself
    assert evict(cache=None) == 1 and evict(lens=None) == 1 and evict(w=None) == 1 and evict(kept=None) == 1
    assert evict(seqs=0, cache=None) == 0


def more_calls():
    """One good call of each wrapper; what it allocates comes from the host."""
    from gptq_post_weight_gb300 import _lib

    def g16(*shape):
        return gpu(torch.zeros(*shape, dtype=torch.bfloat16))

    cache = gpu(torch.zeros(4, 2, 16 * 64 * 5 // 4, dtype=torch.uint8))
    q, k, s = g16(3, 4, 64), g16(3, 2, 64), gpu(torch.zeros(3, dtype=torch.int64))
    turns, table = gpu(torch.zeros(32, dtype=torch.int64)), gpu(torch.zeros(3, 1, dtype=torch.int32))
    lens, w = gpu(torch.ones(3, dtype=torch.int32)), gpu(torch.zeros(3, 2, 16))
    lse = gpu(torch.zeros(3, 4))
    return {
        "x": lambda: _lib.rotary(q, s, turns, out=q, stream=Stream),
        "k": lambda: _lib.kv4_write_rotary(cache, q, k, k, s, 16, s, turns, out=q, stream=Stream),
        "tab": lambda: _lib.q4tp_gated(g16(3, 64), *weights(6, 64), out=g16(3, 3), stream=Stream),
        "q": lambda: _lib.kv4_attention_weights(w, q, lse, cache, table, lens, 16, stream=Stream),
        "lse": lambda: _lib.kv4_attention(q, cache, table, lens, 16, out=g16(3, 4, 64), lse=lse, stream=Stream),
    }


def test_calls_are_made_on_the_current_device_only(rec, monkeypatch):  # noqa: F811
    from gptq_post_weight_gb300 import _lib

    names = []
    for call in more_calls().values():
        call()
        names.append(rec.calls[-1][0])
    assert names == ["gptq_rotary", "gptq_kv4_write_rotary", "gptq_q4tp_gated", "gptq_kv4_attention_weights",
                     "gptq_kv4_attention_lse"]
    done = len(rec.calls)
    monkeypatch.setitem(_lib._serve, "current", lambda: 1)
    for call in more_calls().values():
        with pytest.raises(ValueError, match="the current device is cuda:1"):
            call()
    assert len([c for c in rec.calls[done:] if not c[0].endswith("_bytes")]) == 0


def test_strides_that_one_element_does_not_use(rec):  # noqa: F811
    from gptq_post_weight_gb300 import _lib

    turns, p = gpu(torch.zeros(32, dtype=torch.int64)), gpu(torch.zeros(1, dtype=torch.int64))
    x = torch.as_strided(gpu(torch.zeros(999, dtype=torch.bfloat16)), (1, 1, 64), (67, 3, 1))
    _lib.rotary(x, p, turns, out=x, stream=Stream)
    _, a = rec.calls[-1]
    assert a[2] % 8 == 0 and a[3] % 8 == 0 and a[13] % 8 == 0 and a[14] % 8 == 0


def test_overlapping_rows_are_not_turned_in_place(rec):  # noqa: F811
    from gptq_post_weight_gb300 import _lib

    turns, p = gpu(torch.zeros(32, dtype=torch.int64)), gpu(torch.zeros(3, dtype=torch.int64))
    rows = gpu(torch.zeros(1, 4, 64, dtype=torch.bfloat16)).expand(3, 4, 64)
    with pytest.raises(ValueError, match="do not overlap"):
        _lib.rotary(rows, p, turns, out=rows, stream=Stream)
    cache, k = gpu(torch.zeros(4, 2, 16 * 64 * 5 // 4, dtype=torch.uint8)), gpu(torch.zeros(3, 2, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="do not overlap"):
        _lib.kv4_write_rotary(cache, rows, k, k, p, 16, p, turns, out=rows, stream=Stream)
    assert not rec.calls
