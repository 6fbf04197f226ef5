"""gptq_q4tp_gated against the 64-bit oracle.

Tolerance, per output act(g) * u: the two sums are off by eg and eu as a plain
product's are (test_gpu_linear.py: f32 sums of 32 products of x and a code, the
groups' sums, above 8 tokens half a step of f16, in either type, for every weight), so the product
by 1.13 eg (|u| + eu) + |act(g)| eu with the activations' largest slope; an
activation and the product in f32 add 2^-20 of the result and, where 1 + erf
or a large exponential cancels, 2^-22 |g| |u|; and the result rounds to T by
half a step, 2^-8 (bf16) or 2^-11 (f16) of it.
"""
import numpy as np
import pytest

import test_gpu_linear as lin
from oracle import serve

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def run(p, dtype, act, **kw):
    from gptq_post_weight_gb300 import _lib

    y = _lib.q4tp_gated(lin.dev(p["x"], lin.DT[dtype]), lin.dev(p["nib"]), lin.dev(p["rungs"]), lin.dev(p["tab"]),
                        bias=lin.dev(p["bias"], lin.DT[dtype]), act=act, **kw)
    _lib.serve_check()
    return y


def check(y, p, dtype, act):
    tokens, n = p["x"].shape
    want = serve.gated(p["x"], p["nib"], p["rungs"], p["tab"], p["bias"], act)
    both = serve.linear(p["x"], p["nib"], p["rungs"], p["tab"], p["bias"])
    w = serve.weights(p["nib"], p["rungs"], p["tab"])
    sc = serve.weights(np.full_like(p["nib"], 0x99), p["rungs"], p["tab"])
    ax = np.abs(p["x"])
    mag = ax @ np.abs(w).T
    err = 34 * 143 * 2.0 ** -22 * (ax @ np.abs(sc).T) + (n / 32) * 2.0 ** -23 * mag
    if tokens > 8:
        err = err + HALF["f16"] * mag
    if p["bias"] is not None:
        err = err + 2.0 ** -23 * np.abs(p["bias"])
    half = both.shape[1] // 2
    g, u, eg, eu = both[:, :half], np.abs(both[:, half:]), err[:, :half], err[:, half:]
    off = (1.13 * eg * (u + eu) + np.abs(serve.activate(g, act)) * eu + 2.0 ** -20 * np.abs(want) +
           2.0 ** -22 * np.abs(g) * u)
    tol = off + HALF[dtype] * (np.abs(want) + off) + 2.0 ** -25
    got = y.float().cpu().numpy().astype(np.float64)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.abs(got - want)[bad].max(), tol[bad].min(), np.argwhere(bad)[:5])


def problem(tokens, inner, n, dtype, seed, bias=False):
    p = lin.problem(tokens, 2 * inner, n, dtype, seed, bias)
    # Row scales far apart in neighbouring sixteens: another row's would show.
    p["tab"] = np.ldexp(p["tab"], (np.arange(2 * inner) // 16 % 5 - 2)[:, None]).astype(np.float32)
    return p


SHAPES = [(1, 1, 32), (1, 8, 64), (1, 150, 1024), (2, 65, 96), (3, 64, 256), (5, 129, 2080), (8, 72, 544),
          (9, 32, 288), (16, 100, 1056), (33, 63, 96), (45, 250, 4096), (64, 64, 320), (100, 131, 32),
          (128, 500, 608), (129, 65, 1024), (300, 391, 2080), (513, 128, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,inner,n", SHAPES)
def test_matches_oracle(lib, tokens, inner, n, dtype):
    p = problem(tokens, inner, n, dtype, tokens + inner + n)
    check(run(p, dtype, "silu"), p, dtype, "silu")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,inner", [(1, 71), (4, 72), (12, 71), (70, 136), (300, 71)])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_activations_and_bias(lib, tokens, inner, act, dtype):
    p = problem(tokens, inner, 480, dtype, 7, bias=True)
    check(run(p, dtype, act), p, dtype, act)


@pytest.mark.parametrize("tokens,inner,n", [(1, 2048, 17408), (2, 7168, 4096), (7, 4096, 14336), (40, 512, 17408),
                                            (6, 20, 65536)])
def test_long_and_many_rows(lib, tokens, inner, n):
    p = problem(tokens, inner, n, "bf16", 11)
    check(run(p, "bf16", "silu"), p, "bf16", "silu")


# One round of the pairs of SMs; two, the last tile three outputs and nothing
# for its second CTA; six, so that the row scales' turns come round.
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,inner,n", [(1000, 1500, 800), (1500, 2051, 1056), (2000, 6505, 544)])
def test_pairs_of_sms(lib, tokens, inner, n, dtype):
    import test_gpu_linear_many as many

    p = problem(tokens, inner, n, dtype, tokens, bias=True)
    y, ran = many.kernels_of(lambda: run(p, dtype, "gelu_tanh"))
    assert ran == ({"q4_linear_many": 1, "q4_scale_x": 1} if dtype == "bf16" else {"q4_linear_many": 1})
    check(y, p, dtype, "gelu_tanh")


@pytest.mark.parametrize("tokens", [1, 4, 90, 1500])
def test_strides_out_stream_and_same_bits(lib, tokens):
    from gptq_post_weight_gb300 import _lib

    inner, n = (203, 352) if tokens < 1000 else (2051, 1056)
    p = problem(tokens, inner, n, "bf16", 13, bias=True)
    plain = run(p, "bf16", "silu")
    wide = torch.full((tokens, n + 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + n] = lin.dev(p["x"], torch.bfloat16)
    out = torch.zeros(tokens, inner + 5, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = _lib.q4tp_gated(wide[:, 8:8 + n], lin.dev(p["nib"]), lin.dev(p["rungs"]), lin.dev(p["tab"]),
                        bias=lin.dev(p["bias"], torch.bfloat16), out=out[:, :inner], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, plain) and not out[:, inner:].any()
    assert torch.equal(run(p, "bf16", "silu"), plain)


def test_agrees_with_two_plain_products(lib):
    # The same sums as gptq_q4tp_linear's, so that without an activation and
    # with an up projection of ones the gate comes back as that call gives it.
    from gptq_post_weight_gb300 import _lib

    for tokens in (1, 2, 6, 50):
        p = lin.problem(tokens, 96, 256, "bf16", 3)
        r = np.random.default_rng(4)
        nib = np.concatenate([p["nib"], r.integers(0, 256, p["nib"].size, dtype=np.uint8)])
        rungs = np.concatenate([p["rungs"], p["rungs"]])
        tab = np.concatenate([p["tab"], np.zeros_like(p["tab"])])  # the up projection: 0 x + 1
        bias = torch.cat([torch.zeros(96), torch.ones(96)]).to("cuda", torch.bfloat16)
        x = lin.dev(p["x"], torch.bfloat16)
        y = _lib.q4tp_gated(x, lin.dev(nib), lin.dev(rungs), lin.dev(tab), bias=bias, act="none")
        z = _lib.q4tp_linear(x, lin.dev(p["nib"]), lin.dev(p["rungs"]), lin.dev(p["tab"]))
        assert (y.float() - z.float()).abs().max() <= 2.0 ** -8 * z.float().abs().max()


@pytest.mark.parametrize("tokens", [1, 5, 40])
def test_infinite_activation(lib, tokens):
    p = problem(tokens, 40, 128, "bf16", 17)
    p["x"][0, 5] = np.inf
    p["nib"][:] |= 0x11  # no code is 8: no weight 0
    y = run(p, "bf16", "none").float().cpu().numpy()
    want = serve.gated(p["x"], p["nib"], p["rungs"], p["tab"], None, "none")
    assert np.isinf(want[0]).all()
    np.testing.assert_array_equal(y[0], want[0].astype(np.float32))
    assert np.isfinite(y[1:]).all()


def test_no_tokens_zero_rows_and_large_rungs(lib):
    from gptq_post_weight_gb300 import _lib

    p = problem(20, 100, 96, "f16", 19)
    p["tab"][[0, 99, 100, 150]] = 0
    p["rungs"][::7] = 250  # counts as scale 0
    y = run(p, "f16", "silu")
    check(y, p, "f16", "silu")
    assert not y[:, [0, 50, 99]].any()
    e = torch.empty(0, 96, dtype=torch.float16, device="cuda")
    assert _lib.q4tp_gated(e, lin.dev(p["nib"]), lin.dev(p["rungs"]), lin.dev(p["tab"])).shape == (0, 100)


@pytest.mark.parametrize("tokens", [1, 8, 100, 1500])
def test_waits_run_out(lib, tokens):
    from gptq_post_weight_gb300 import _lib

    inner, n = (128, 608) if tokens < 1000 else (2051, 1056)
    p = problem(tokens, inner, n, "bf16", 23)
    want = run(p, "bf16", "silu")
    try:
        _lib.test_set_wait(1_000_000, no_loads=True)
        with pytest.raises(_lib.GptqError) as ei:
            run(p, "bf16", "silu")
        assert ei.value.code == 6
    finally:
        _lib.test_set_wait()
    assert torch.equal(run(p, "bf16", "silu"), want)


def test_captured_and_replayed(lib):
    from gptq_post_weight_gb300 import _lib

    p = problem(3, 64, 256, "bf16", 29)
    x, nib, rungs, tab = lin.dev(p["x"], torch.bfloat16), lin.dev(p["nib"]), lin.dev(p["rungs"]), lin.dev(p["tab"])
    first = _lib.q4tp_gated(x, nib, rungs, tab)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = _lib.q4tp_gated(x, nib, rungs, tab)
    g.replay()
    assert torch.equal(y, first)
    x.mul_(2)
    g.replay()
    assert torch.equal(y, _lib.q4tp_gated(x, nib, rungs, tab)) and not torch.equal(y, first)


@pytest.mark.parametrize("tokens", [12, 1500])
def test_tokens_of_any_size(lib, tokens):
    # Above 8 tokens bf16 rows are f16 numbers times a power of two each: rows from
    # 2^-120 to 2^100, elements 2^30 apart in one row, a row of zeros.  (No
    # activation, and gate and up projection alike in size, so that the results
    # of the small rows are what bf16 holds of their squares: those past its ends
    # are left out.)
    inner, n = (70, 256) if tokens < 1000 else (2051, 256)
    p = problem(tokens, inner, n, "bf16", 31)
    size = np.array([0, 20, 40, 60, -20, -40, -60, 100, -120, 3, -3, 0])[np.arange(tokens) % 12]
    p["x"] = np.ldexp(p["x"], size[:, None])
    p["x"][3, ::2] = serve.round_to(np.ldexp(p["x"][3, ::2], -30), "bf16")
    p["x"][11] = 0
    y = run(p, "bf16", "none")
    fits = (np.abs(size) <= 60)
    p["x"] = p["x"][fits]
    check(y[torch.from_numpy(fits).cuda()], p, "bf16", "none")
    assert not y[11].any()
    assert torch.isinf(y[7]).any() and torch.isfinite(y[8]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,inner,n", [(20, 40, 128), (20, 41, 608), (1500, 2051, 1056)])
def test_infinite_and_nan_rows_above_eight_tokens(lib, tokens, inner, n, dtype):
    # Columns of both halves of a box; scales that are powers of two, so that the
    # weights' rounding leaves nothing, among others.
    p = problem(tokens, inner, n, dtype, 18)
    p["tab"][::2] = np.exp2(np.round(np.log2(p["tab"][::2])))
    p["x"][4, 5], p["x"][7, 9], p["x"][11, 100] = -np.inf, np.nan, np.inf
    if n > 300:
        p["x"][13, 200] = np.inf
    p["nib"][:] |= 0x11  # no code is 8: no weight 0
    y = run(p, dtype, "none").float().cpu().numpy()
    some = slice(0, 20)
    want = serve.gated(p["x"][some], p["nib"], p["rungs"], p["tab"], None, "none")
    rows = [4, 11] + ([13] if n > 300 else [])
    assert np.isinf(want[rows]).all()
    np.testing.assert_array_equal(y[rows], want[rows].astype(np.float32))
    assert np.isnan(y[7]).all() and np.isfinite(np.delete(y, rows + [7], 0)).all()


def test_given_workspace(lib):
    from gptq_post_weight_gb300 import _lib

    p = problem(30, 50, 160, "bf16", 20)
    want = run(p, "bf16", "silu")
    ws = _lib.workspace(lib.gptq_q4tp_gated_workspace_bytes(0, 30, 160), "cuda")
    assert torch.equal(run(p, "bf16", "silu", ws=ws), want)
