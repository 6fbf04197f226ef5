"""Pins of the serving oracle: its rounding against numpy's own f16, the
codec's error bound, exact cases and what it does with NaN and infinity, the
block layout against a byte-by-byte packer, and the attention against a
direct sum."""
import math

import numpy as np
import pytest

from oracle import serve


def test_round_to_is_numpy_f16():
    r = np.random.default_rng(1)
    x = np.concatenate([r.standard_normal(4000) * 10.0 ** r.integers(-9, 6, 4000), [0.0, 65519.9, 65520.0, -65520.0,
                        2.0 ** -25, 2.0 ** -24, np.inf, np.nan]])
    with np.errstate(over="ignore"):
        want = x.astype(np.float16).astype(np.float64)
    np.testing.assert_array_equal(serve.round_to(x, "f16"), want)


def test_round_to_bf16_is_the_top_half_of_f32():
    r = np.random.default_rng(2)
    x = r.standard_normal(4000).astype(np.float32)
    b = x.view(np.uint32).astype(np.uint64)
    want = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16).astype(np.uint32).view(np.float32)
    np.testing.assert_array_equal(serve.round_to(x, "bf16"), want)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_round_trip_error(dtype):
    # Half a step, plus what rounding s (15 half-ulps at the top code) and the
    # value itself can add.
    r = np.random.default_rng(3)
    x = serve.round_to(r.standard_normal((50, 3, 128)) * 3 + 1, dtype)
    c, s, z = serve.quantise(x, dtype)
    assert c.min() == 0 and c.max() == 15
    u = 2.0 ** -serve.TYPES[dtype][0]
    back = serve.values(c, s, z, dtype)
    step = np.repeat(s.astype(np.float64), 32, -1)
    off = np.repeat(np.abs(z.astype(np.float64)), 32, -1)
    assert np.all(np.abs(back - x) <= step * (0.5 + 15 * u) + u * (off + np.abs(x)) + 1e-6 * np.abs(x))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_constant_and_two_level_groups_are_exact(dtype):
    x = np.full((2, 64), 1.5)
    np.testing.assert_array_equal(serve.round_trip(x, dtype), x)
    y = np.zeros((1, 32))
    y[0, ::2] = 15.0  # s = 1, z = -16
    np.testing.assert_array_equal(serve.round_trip(y, dtype), y)
    np.testing.assert_array_equal(serve.round_trip(np.arange(32).reshape(1, 32) // 2 * 1.0, dtype),
                                  np.arange(32).reshape(1, 32) // 2)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_non_finite_groups_are_nan_and_others_are_not(bad):
    x = np.random.default_rng(4).standard_normal((2, 64))
    x = serve.round_to(x, "bf16")
    x[1, 40] = bad
    y = serve.round_trip(x, "bf16")
    assert np.isnan(y[1, 32:]).all() and np.isfinite(y[0]).all() and np.isfinite(y[1, :32]).all()


def test_f16_range():
    x = np.zeros((1, 32))
    x[0, 0], x[0, 1] = 20000, -20000
    assert np.isfinite(serve.round_trip(x, "f16")).all()
    x[0, 0], x[0, 1] = 60000, -60000
    assert np.isnan(serve.round_trip(x, "f16")).all()


def test_weights_and_linear():
    rows, n = 3, 64
    r = np.random.default_rng(5)
    nib = r.integers(0, 256, rows * n // 2, dtype=np.uint8)
    rungs = np.array([0, 31, 5, 7, 40, 2], dtype=np.uint8)
    tab = np.exp2(r.standard_normal((rows, 32)))
    w = serve.weights(nib, rungs, tab)
    for i in range(rows):
        for c in range(n):
            b = int(nib[i * n // 2 + c // 2])
            q = (b >> 4 if c % 2 else b & 15) - 8
            g = rungs[i * 2 + c // 32]
            assert w[i, c] == q * (tab[i, g] if g < 32 else 0.0)
    x = r.standard_normal((2, n))
    y = serve.linear(x, nib, rungs, tab, bias=[1, 2, 3], act="relu", residual=np.ones((2, rows)))
    np.testing.assert_allclose(y, np.maximum(x @ w.T + [1, 2, 3], 0) + 1)


def test_activations():
    assert serve.activate(0.0, "gelu") == 0 and serve.activate(-1.0, "relu") == 0
    assert math.isclose(float(serve.activate(1.0, "gelu")), 0.8413447460685429, rel_tol=1e-12)
    assert math.isclose(float(serve.activate(1.0, "silu")), 1 / (1 + math.exp(-1)), rel_tol=1e-12)
    assert abs(float(serve.activate(1.0, "gelu_tanh")) - 0.8411919906082768) < 1e-12


def test_pack_block():
    d = 64
    r = np.random.default_rng(6)
    kc, vc = r.integers(0, 16, (16, d)), r.integers(0, 16, (16, d))
    kp, vp = r.integers(0, 65536, (16, 2, 2)), r.integers(0, 65536, (16, 2, 2))
    b = serve.pack_block(kc, vc, kp, vp)
    assert b.size == 20 * d
    for t in range(16):
        for j in range(d):
            assert (b[t * d // 2 + j // 2] >> (4 * (j % 2))) & 15 == kc[t, j]
            assert (b[10 * d + t * d // 2 + j // 2] >> (4 * (j % 2))) & 15 == vc[t, j]
        for g in range(2):
            for e in range(2):
                at = 8 * d + ((t * 2 + g) * 2 + e) * 2
                assert int(b[at]) + 256 * int(b[at + 1]) == kp[t, g, e]


def test_attention_is_causal_and_empty_rows_are_zero():
    r = np.random.default_rng(7)
    d, lens, q_lens = 4, [3, 1, 0], [2, 3, 1]
    q = r.standard_normal((6, 2, d))
    k = [r.standard_normal((n, 1, d)) for n in lens]
    v = [r.standard_normal((n, 1, d)) for n in lens]
    o = serve.attention(q, k, v, lens, 2, 0.5, q_lens)
    e = np.exp(0.5 * k[0][:2, 0] @ q[0, 1])
    np.testing.assert_allclose(o[0, 1], e @ v[0][:2, 0] / e.sum())
    assert not o[2].any() and not o[3].any() and not o[5].any()  # before the first key; an empty sequence
    np.testing.assert_allclose(o[4, 0], v[1][0, 0])
