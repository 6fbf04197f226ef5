"""The serving calls refuse what they cannot use before anything is launched
(CPU only): the binding with a ValueError naming the argument, the C entries
with their status."""
import ctypes
import os

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def blib():
    from gptq_post_weight_gb300 import _lib, build

    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    _lib.load()
    return _lib


def refused(fn, *args, match, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*args, **kw)


def b16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def test_linear(blib):
    t, rows, n = 3, 6, 64
    x, nib, rungs, tab = b16(t, n), u8(rows * n // 2), u8(rows * 2), torch.zeros(rows, 32)
    f = blib.q4tp_linear
    refused(f, x.float(), nib, rungs, tab, match="x must be torch.bfloat16 or torch.float16")
    refused(f, b16(t, 48), nib, rungs, tab, match="multiple of 32 columns")
    refused(f, b16(t * n), nib, rungs, tab, match="2-D")
    refused(f, b16(t, 2 * n)[:, ::2], nib, rungs, tab, match="contiguous in its last dimension")
    refused(f, b16(t, n + 4)[:, :n], nib, rungs, tab, match="multiple of 8 elements")
    refused(f, x, nib[:-1], rungs, tab, match="nibbles must have 192")
    refused(f, x, nib, rungs[:-1], tab, match="rungs must have 12")
    refused(f, x, nib, rungs, tab.view(-1), match="tab must be")
    refused(f, x, nib, rungs, tab, bias=b16(rows + 1), match="bias must have 6")
    refused(f, x, nib, rungs, tab, bias=torch.zeros(rows), match="bias must be torch.bfloat16")
    refused(f, x, nib, rungs, tab, act="swish", match="act must be one of")
    refused(f, x, nib, rungs, tab, residual=b16(t, rows - 1), match="residual must have shape")
    refused(f, x, nib, rungs, tab, residual=b16(1, rows).expand(t, rows), match="do not overlap")
    refused(f, x, nib, rungs, tab, out=b16(rows, t).t(), match="dense rows")
    refused(f, x, nib, rungs, tab, out=torch.zeros(t, rows), match="out must be")
    refused(f, x, nib, rungs, tab, match="CUDA tensors")


def test_cache(blib):
    cache = u8(4, 2, 16 * 64 * 5 // 4)
    k, slots = b16(5, 2, 64), torch.zeros(5, dtype=torch.int64)
    f = blib.kv4_write
    refused(f, cache, k.float(), k, slots, 16, match="k must be")
    refused(f, cache, k, k.half(), slots, 16, match="v must be torch.bfloat16")
    refused(f, cache, k, b16(5, 2, 128), slots, 16, match="v must have shape")
    refused(f, cache, b16(5, 3, 64), b16(5, 3, 64), slots, 16, match="3 heads, the cache 2")
    refused(f, cache, k, k, slots[:-1], 16, match="slots must have 5")
    refused(f, cache, k, k, slots.int(), 16, match="slots must be torch.int64")
    refused(f, cache, k, k, slots, 32, match="cache must be")
    refused(f, cache, k, k, slots, 24, match="page_size must be")
    refused(f, cache, b16(5, 2, 96), b16(5, 2, 96), slots, 16, match="dim must be 64, 128 or 256")
    refused(f, cache, b16(5, 2, 68)[..., :64], k, slots, 16, match="multiple of 8")
    refused(f, cache, k, k, slots, 16, match="CUDA tensors")
    refused(blib.kv4_read, cache, slots, 64, 16, torch.float32, match="dtype must be")
    refused(blib.kv4_read, cache, slots.int(), 64, 16, torch.float16, match="slots must be")
    refused(blib.kv4_read, cache, slots, 128, 16, torch.float16, match="cache must be")
    refused(blib.kv4_cache, 4, 2, 80, 16, "cpu", match="dim must be")
    refused(blib.kv4_cache, 4, 2, 64, 8, "cpu", match="page_size must be")


def test_attention(blib):
    cache = u8(4, 2, 16 * 64 * 5 // 4)
    q, table, lens = b16(3, 4, 64), torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    starts = torch.arange(4, dtype=torch.int32)
    f = blib.kv4_attention
    refused(f, q.float(), cache, table, lens, 16, match="q must be")
    refused(f, b16(3, 5, 64), cache, table, lens, 16, match="not a multiple of the cache's 2")
    refused(f, q, cache, table.long(), lens, 16, match="table must be torch.int32")
    refused(f, q, cache, table[:, :0], lens, 16, match="table must be 2-D")
    refused(f, q, cache, table, lens[:2], 16, match="kv_lens must have 3")
    refused(f, q, cache, table[:2], lens[:2], 16, match="one query a sequence")
    refused(f, q, cache, table, lens, 16, max_q=2, match="one query a sequence")
    refused(f, q, cache, table, lens, 16, q_starts=starts[:3], match="q_starts must have 4")
    refused(f, q, cache, table, lens, 16, q_starts=starts, max_q=0, match="max_q must be positive")
    refused(f, q, cache, table, lens, 16, out=b16(3, 4, 32), match="out must have")
    refused(f, q, cache, table, lens, 16, ws=torch.zeros(4), match="ws must be")
    refused(f, q, cache, table, lens, 32, match="cache must be")


def test_c_entries(blib):
    lib = blib.load()
    P = ctypes.c_void_p
    ok, mis, big = P(1 << 20), P((1 << 20) + 4), 1 << 40

    def linear(dt=0, x=ok, ldx=64, t=3, nib=ok, rows=6, n=64, act=0, res=None, ldr=0, y=ok, ldy=6):
        return lib.gptq_q4tp_linear(dt, x, ldx, t, nib, ok, ok, rows, n, None, act, res, ldr, y, ldy, None, None)

    assert linear(n=48, ldx=48) == 2 and linear(t=-1) == 2 and linear(rows=0) == 2 and linear(t=(1 << 20) + 1) == 2
    assert linear(ldx=32) == 2 and linear(ldx=68) == 2 and linear(ldy=5) == 2 and linear(res=ok, ldr=5) == 2
    assert linear(dt=2) == 1 and linear(act=5) == 1 and linear(act=-1) == 1
    assert linear(x=None) == 1 and linear(nib=mis) == 1 and linear(y=mis) == 1
    assert linear(t=0, x=None, y=None) == 0

    def write(dt=0, cache=ok, pages=4, heads=2, dim=64, page=16, k=ok, kt=128, slots=ok, t=5):
        return lib.gptq_kv4_write(dt, cache, pages, heads, dim, page, k, ok, kt, 64, 128, 64, slots, t, None)

    assert write(pages=0) == 2 and write(heads=0) == 2 and write(dim=96) == 2 and write(page=24) == 2
    assert write(page=8192) == 2 and write(t=-1) == 2 and write(kt=12) == 2 and write(kt=-8) == 2
    assert write(dt=7) == 1 and write(cache=None) == 1 and write(k=mis) == 1 and write(slots=None) == 1
    assert write(t=0, k=None) == 0
    assert lib.gptq_kv4_read(0, ok, 4, 2, 64, 16, ok, 5, mis, ok, None) == 1
    assert lib.gptq_kv4_read(0, ok, 4, 2, 32, 16, ok, 5, ok, ok, None) == 2

    def attend(dt=0, q=ok, qt=256, tq=3, group=2, stride=2, lens=ok, starts=None, seqs=3, max_q=1, scale=1.0, ws=big):
        return lib.gptq_kv4_attention(dt, q, qt, 64, tq, ok, 4, 2, group, 64, 16, ok, stride, lens, starts, seqs, max_q,
                                      scale, ok, ok, ws, None, None)

    assert attend(group=0) == 2 and attend(stride=0) == 2 and attend(tq=4) == 2 and attend(max_q=2) == 2
    assert attend(qt=4) == 2 and attend(seqs=-1) == 2 and attend(starts=ok, max_q=0) == 2
    assert attend(dt=3) == 1 and attend(scale=float("nan")) == 1 and attend(q=mis) == 1 and attend(lens=None) == 1
    assert attend(ws=16, stride=1000) == 3 and attend(ws=0, starts=ok, max_q=100) == 3
    assert attend(tq=0, starts=ok) == 0
    assert lib.gptq_kv4_attention_workspace_bytes(96, 4, 1) == 0
    assert lib.gptq_kv4_attention_workspace_bytes(64, 0, 1) == 0
    # What one call needs: nothing for few rows over a short table, never more
    # than the bound that does not know the call.
    assert lib.gptq_kv4_attention_call_bytes(96, 8, 4, 1, 1, 1, 1024) == 0
    for dim in (64, 128, 256):
        for group, max_q in ((1, 1), (8, 1), (16, 1), (4, 5), (4, 8), (8, 9), (4, 512)):
            bound = lib.gptq_kv4_attention_workspace_bytes(dim, group, max_q)
            for heads, seqs, length in ((1, 1, 16), (8, 1, 8192), (8, 64, 1024), (1024, 5000, 1 << 30)):
                need = lib.gptq_kv4_attention_call_bytes(dim, heads, group, max_q, seqs, max_q == 1, length)
                assert need <= bound
                assert (need == 0) == (group * max_q <= 8 and seqs * heads <= 8)
