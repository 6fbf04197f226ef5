"""Pins of the oracle's rotary positions, gated product, attention weights and
choice of what stays: against complex numbers, plain sums and small cases by
hand."""
import math

import numpy as np
import pytest

from oracle import serve


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_is_a_product_of_complex_numbers(layout):
    r = np.random.default_rng(1)
    x, angle = r.standard_normal((5, 2, 32)), r.uniform(-9, 9, (5, 12))
    y = serve.rotary(x, angle, layout, 1.5)
    i, j = (slice(0, 12), slice(12, 24)) if layout == "half" else (slice(0, 24, 2), slice(1, 24, 2))
    z = (x[..., i] + 1j * x[..., j]) * 1.5 * np.exp(1j * angle)[:, None]
    np.testing.assert_allclose(y[..., i], z.real, atol=1e-14)
    np.testing.assert_allclose(y[..., j], z.imag, atol=1e-14)
    np.testing.assert_array_equal(y[..., 24:], x[..., 24:])
    # Scores depend on the distance alone.
    f = angle[0]
    a, b = (serve.rotary(x[:1], (p * f)[None], layout)[0, 0, :24] for p in (7, 3))
    c, d = (serve.rotary(x[:1], (p * f)[None], layout)[0, 0, :24] for p in (104, 100))
    assert abs(a @ b - c @ d) < 1e-12


def test_angles_are_modulo_one_turn():
    t = [2 ** 62, -(2 ** 62), 1]  # a quarter, minus a quarter, 2^-64 of a turn
    a = serve.angles([0, 1, 2, 5, -1, 2 ** 62], t)
    np.testing.assert_allclose(a[:, 0], np.array([0, 0.5, 1, 0.5, 1.5, 0]) * math.pi)
    np.testing.assert_allclose(a[:, 1], np.array([0, 1.5, 1, 1.5, 0.5, 0]) * math.pi)
    assert a[5, 2] == math.pi / 2


def test_gated():
    r = np.random.default_rng(2)
    x, nib = r.standard_normal((3, 32)), r.integers(0, 256, 6 * 16, dtype=np.uint8)
    rungs, tab, bias = r.integers(0, 32, 6, dtype=np.uint8), r.uniform(0.1, 1, (6, 32)), r.standard_normal(6)
    y = x @ serve.weights(nib, rungs, tab).T + bias
    np.testing.assert_allclose(serve.gated(x, nib, rungs, tab, bias), y[:, :3] / (1 + np.exp(-y[:, :3])) * y[:, 3:])


def test_weights_add_to_the_rows_and_give_the_attention():
    r = np.random.default_rng(3)
    lens, q_lens = [5, 2], [3, 4]
    ks, vs = ([r.standard_normal((n, 2, 8)) for n in lens] for _ in range(2))
    q = r.standard_normal((7, 4, 8))
    lse = serve.log_sums(q, ks, lens, 2, 0.3, q_lens)
    assert np.isneginf(lse[3:5]).all() and np.isfinite(lse[[0, 1, 2, 5, 6]]).all()
    w = serve.attention_weights(q, ks, lens, 2, 0.3, np.where(np.isneginf(lse), 0, lse), q_lens)
    np.testing.assert_allclose(w[0].sum(1), 6)
    np.testing.assert_allclose(w[1].sum(1), 4)
    # One query alone: its weights times the values are its output.
    one = serve.attention_weights(q[:1, :1], [ks[0][:, :1]], [5], 1, 0.3, serve.log_sums(q[:1, :1], [ks[0][:, :1]], [5], 1, 0.3))
    o = serve.attention(q[:1, :1], [ks[0][:, :1]], [vs[0][:, :1]], [5], 1, 0.3)
    np.testing.assert_allclose(one[0][0] @ vs[0][:, 0], o[0, 0])


def test_kept():
    w = [3.0, 1.0, 3.0, np.nan, 0.0, 9.0]
    assert serve.kept(w, 6, 6, 0) == [0, 1, 2, 3, 4, 5]
    assert serve.kept(w, 6, 2, 0) == [0, 5]
    assert serve.kept(w, 6, 3, 1) == [0, 2, 5]
    assert serve.kept(w, 6, 2, 1) == [0, 5]
    assert serve.kept(w, 6, 4, 9) == [2, 3, 4, 5]
    assert serve.kept(w, 5, 4, 0) == [0, 1, 2, 4]  # a NaN goes first
    assert serve.kept([np.nan] * 4, 4, 2, 0) == [0, 1]
    assert serve.kept([0.0, -0.0, 1.0], 3, 2, 0) == [0, 2]
    assert serve.kept([], 0, 2, 1) == []
