"""gptq_rotary and gptq_kv4_write_rotary against the 64-bit oracle.

Tolerance, per output y = x0 c - x1 s (or its mate), from the definition: the
angle is a whole number of 2^-32 turns rounded to f32 (at most pi 2^-25), sine
and cosine are good to two f32 steps (2^-23) and three products and sums round
once each (2^-24 of at most |x0| + |x1|): 4e-7 < 2^-21 of gain (|x0| + |x1|)
together.  The result rounds to T: half a step, 2^-8 (bf16) or 2^-11 (f16) of
it, or half of f16's smallest number.
"""
import numpy as np
import pytest

from oracle import serve

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def dev(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def bits(t):
    return t.contiguous().view(torch.int16)


def problem(tokens, heads, dim, rot, dtype, seed, start=0, scaling="none"):
    from gptq_post_weight_gb300 import _lib

    r = np.random.default_rng(seed)
    x = serve.round_to(r.standard_normal((tokens, heads, dim)), dtype)
    positions = start + r.permutation(3 * tokens)[:tokens].astype(np.int64)
    turns = _lib.rotary_turns(_lib.rotary_frequencies(rot, scaling=scaling, factor=4.0))
    return x, positions, turns


def check(got, x, positions, turns, dtype, layout, gain=1.0):
    t = turns.cpu().numpy()
    n = len(t)
    want = serve.rotary(x, serve.angles(positions, t), layout, gain)
    mag = np.abs(x).copy()
    i, j = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    mag[..., i] = mag[..., j] = np.abs(x[..., i]) + np.abs(x[..., j])
    err = 2.0 ** -21 * abs(gain) * mag
    err[..., 2 * n:] = 0
    tol = err + HALF[dtype] * (np.abs(want) + err) + 2.0 ** -25
    got = host(got)
    assert got.shape == want.shape
    assert (np.abs(got - want) <= tol).all(), np.abs(got - want).max()
    np.testing.assert_array_equal(got[..., 2 * n:], x[..., 2 * n:])


SHAPES = [(1, 1, 16, 16), (1, 40, 128, 128), (3, 5, 64, 64), (7, 3, 80, 48), (33, 2, 96, 32), (130, 9, 256, 256),
          (257, 4, 128, 64), (1000, 3, 192, 112), (5, 2, 1024, 1024)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,heads,dim,rot", SHAPES)
def test_matches_oracle(lib, tokens, heads, dim, rot, layout, dtype):
    from gptq_post_weight_gb300 import _lib

    x, positions, turns = problem(tokens, heads, dim, rot, dtype, tokens + dim)
    y = _lib.rotary(dev(x, DT[dtype]), dev(positions), turns, layout=layout)
    check(y, x, positions, turns, dtype, layout)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("scaling", ["none", "linear", "base", "ramp"])
def test_far_positions_scaling_and_gain(lib, scaling, layout):
    from gptq_post_weight_gb300 import _lib

    x, positions, turns = problem(40, 2, 128, 128, "f16", 3, start=5_000_000, scaling=scaling)
    # Any 64-bit position, negative ones among them: the product is modulo one turn.
    positions[:6] = [0, -1, -7_000_001, 2 ** 40 + 3, 2 ** 62, -2 ** 63]
    y = _lib.rotary(dev(x, torch.float16), dev(positions), turns, layout=layout, gain=1.25)
    check(y, x, positions, turns, "f16", layout, 1.25)
    y = _lib.rotary(dev(x, torch.float16), dev(positions), turns, layout=layout, gain=-0.5)
    check(y, x, positions, turns, "f16", layout, -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_strided_in_place_and_stream(lib, layout, dtype):
    from gptq_post_weight_gb300 import _lib

    x, positions, turns = problem(70, 6, 128, 96, dtype, 5)
    plain = _lib.rotary(dev(x, DT[dtype]), dev(positions), turns, layout=layout)
    wide = torch.full((70, 9, 136), float("nan"), dtype=DT[dtype], device="cuda")
    view = wide[:, 2:8, :128]
    view.copy_(dev(x, DT[dtype]))
    before = wide.clone()
    assert torch.equal(_lib.rotary(view, dev(positions), turns, layout=layout), plain)
    assert torch.equal(bits(wide), bits(before))
    # Into another tensor, heads outermost; rows around it stay.
    out = torch.zeros(6, 72, 128, dtype=DT[dtype], device="cuda").transpose(0, 1)[1:71]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _lib.rotary(view, dev(positions), turns, layout=layout, out=out, stream=side)
    torch.cuda.synchronize()
    assert got is out and torch.equal(out, plain) and not out._base[:, [0, 71]].any()
    assert _lib.rotary(view, dev(positions), turns, layout=layout, out=view) is view
    assert torch.equal(view, plain)
    before[:, 2:8, :128] = plain
    assert torch.equal(bits(wide), bits(before))


def test_not_a_number_stays_in_its_pair(lib):
    from gptq_post_weight_gb300 import _lib

    x, positions, turns = problem(4, 2, 64, 32, "bf16", 6)
    clean = _lib.rotary(dev(x, torch.bfloat16), dev(positions), turns)
    x[1, 0, 3], x[2, 1, 40], x[3, 1, 63] = np.nan, np.inf, np.nan
    y = _lib.rotary(dev(x, torch.bfloat16), dev(positions), turns)
    bad = ~np.isfinite(host(y))
    where = np.zeros_like(bad)
    where[1, 0, 3] = where[1, 0, 19] = where[2, 1, 40] = where[3, 1, 63] = True
    np.testing.assert_array_equal(bad, where)
    assert torch.equal(y[torch.from_numpy(~where).cuda()], clean[torch.from_numpy(~where).cuda()])


def test_no_tokens(lib):
    from gptq_post_weight_gb300 import _lib

    _, _, turns = problem(1, 1, 64, 64, "bf16", 0)
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    x = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert _lib.rotary(x, none, turns).shape == (0, 2, 64)
    cache = _lib.kv4_cache(1, 2, 64, 16)
    assert _lib.kv4_write_rotary(cache, x, x, x, none, 16, none, turns).shape == (0, 2, 64) and not cache.any()


def test_largest_call(lib):
    # More than 2^31 elements: rows at both ends against a small call's.
    from gptq_post_weight_gb300 import _lib

    tokens, heads, dim = (1 << 20), 17, 128
    _, _, turns = problem(1, 1, dim, dim, "bf16", 0)
    x = torch.randn(64, heads, dim, device="cuda").to(torch.bfloat16).repeat(tokens // 64, 1, 1)
    positions = torch.arange(tokens, device="cuda")
    y = _lib.rotary(x, positions, turns, layout="interleaved")
    for rows in (slice(0, 64), slice(tokens // 2, tokens // 2 + 64), slice(tokens - 64, tokens)):
        assert torch.equal(y[rows], _lib.rotary(x[rows], positions[rows].contiguous(), turns, layout="interleaved"))


# ---------------------------------------------------------------- into the cache


def store(tokens, heads, group, dim, rot, page, layout, dtype, seed, gain=1.0, in_place=False):
    """kv4_write_rotary on strided views, and rotary with kv4_write beside it."""
    from gptq_post_weight_gb300 import _lib

    r = np.random.default_rng(seed)
    hq = heads * group
    x, positions, turns = problem(tokens, hq + 2 * heads, dim, rot, dtype, seed)
    x[..., hq:, :] *= np.exp(0.4 * r.standard_normal(dim))
    qkv = dev(serve.round_to(x, dtype), DT[dtype])
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + heads], qkv[:, hq + heads:]
    pages = tokens // page + 2
    slots = dev(r.permutation(pages * page)[:tokens].astype(np.int64))
    if tokens > 4:
        slots[3], slots[4] = -1, pages * page  # outside the pool
    p = dev(positions)
    want_q = _lib.rotary(q, p, turns, layout=layout, gain=gain)
    want = _lib.kv4_cache(pages, heads, dim, page).fill_(0xA5)
    _lib.kv4_write(want, _lib.rotary(k, p, turns, layout=layout, gain=gain), v, slots, page)
    cache = _lib.kv4_cache(pages, heads, dim, page).fill_(0xA5)
    before = qkv.clone()
    got = _lib.kv4_write_rotary(cache, q, k, v, slots, page, p, turns, layout=layout, gain=gain,
                                out=q if in_place else None)
    assert torch.equal(got, want_q) and torch.equal(cache, want)
    if in_place:
        before[:, :hq] = want_q
        assert got is q
    assert torch.equal(qkv, before)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,heads,group,dim,rot,page", [
    (1, 1, 1, 64, 64, 16), (1, 8, 4, 128, 128, 64), (5, 2, 5, 64, 16, 16), (17, 3, 2, 128, 96, 32),
    (64, 8, 4, 128, 128, 64), (33, 1, 8, 256, 256, 16), (300, 2, 3, 256, 112, 48), (2000, 4, 4, 128, 64, 16)])
def test_write_has_the_bits_of_both_calls(lib, tokens, heads, group, dim, rot, page, layout, dtype):
    store(tokens, heads, group, dim, rot, page, layout, dtype, tokens + rot, gain=1.0 if tokens < 50 else 0.9,
          in_place=tokens % 2 == 1)


def test_write_of_a_long_prompt(lib):
    store(20011, 8, 4, 128, 128, 64, "half", "bf16", 9)


def test_captured_and_replayed(lib):
    from gptq_post_weight_gb300 import _lib

    x, positions, turns = problem(6, 8, 64, 64, "bf16", 12)
    qkv, p = dev(x, torch.bfloat16), dev(positions)
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    slots = torch.arange(6, device="cuda")
    cache = _lib.kv4_cache(2, 2, 64, 16)
    first = _lib.kv4_write_rotary(cache, q, k, v, slots, 16, p, turns)  # loads the kernels
    first_cache = cache.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = _lib.kv4_write_rotary(cache, q, k, v, slots, 16, p, turns)
        z = _lib.rotary(q, p, turns)
    cache.zero_()
    g.replay()
    assert torch.equal(y, first) and torch.equal(z, first) and torch.equal(cache, first_cache)
    p.add_(100)
    g.replay()
    assert torch.equal(y, _lib.rotary(q, p, turns)) and not torch.equal(y, first)
