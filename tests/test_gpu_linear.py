"""gptq_q4tp_linear against the 64-bit oracle.

Tolerance, per output: one rounding to T of the result (u |y|, u = 2^-8 or
2^-11 taken as a whole ulp), plus the product's own error times the
activation's largest slope (1.13): every weight rounded once to T (u / 2 of
sum |x w|, only above 8 tokens) and f32 sums.  For these, a group's 32
products of x and a code of at most 143 (bf16: 128 + 15; the f16 codes are
smaller) are added with at most 2^-22 of error each to their running total,
so 34 * 143 * 2^-22 of s sum |x|, and the n / 32 groups add 2^-23 of
sum |x w| each.
"""
import numpy as np
import pytest

from oracle import serve

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def problem(tokens, rows, n, dtype, seed, bias=False, residual=False):
    r = np.random.default_rng(seed)
    p = dict(
        x=serve.round_to(r.standard_normal((tokens, n)) * np.exp(0.5 * r.standard_normal(n)), dtype),
        nib=r.integers(0, 256, rows * n // 2, dtype=np.uint8),
        rungs=r.integers(0, 32, rows * n // 32, dtype=np.uint8),
        tab=np.exp2(-9 + r.standard_normal((rows, 1)) + np.arange(32) * r.uniform(0, 0.1, (rows, 1))).astype(np.float32),
        bias=serve.round_to(r.standard_normal(rows), dtype) if bias else None,
        residual=serve.round_to(r.standard_normal((tokens, rows)), dtype) if residual else None)
    return p


def dev(a, dtype=None):
    return None if a is None else torch.from_numpy(np.asarray(a)).to("cuda", dtype)


def run(p, dtype, act, **kw):
    from gptq_post_weight_gb300 import _lib

    y = _lib.q4tp_linear(dev(p["x"], DT[dtype]), dev(p["nib"]), dev(p["rungs"]), dev(p["tab"]),
                         bias=dev(p["bias"], DT[dtype]), act=act, residual=dev(p["residual"], DT[dtype]), **kw)
    _lib.serve_check()
    return y


def check(y, p, dtype, act):
    tokens, n = p["x"].shape
    want = serve.linear(p["x"], p["nib"], p["rungs"], p["tab"], p["bias"], act, p["residual"])
    w = serve.weights(p["nib"], p["rungs"], p["tab"])
    full = np.full_like(p["nib"], 0x99)  # every code 1: the scales alone
    sc = serve.weights(full, p["rungs"], p["tab"])
    ax = np.abs(p["x"])
    mag = ax @ np.abs(w).T
    u = 2.0 ** (1 - serve.TYPES[dtype][0])
    err = 34 * 143 * 2.0 ** -22 * (ax @ np.abs(sc).T) + (n / 32) * 2.0 ** -23 * mag
    if tokens > 8:
        err = err + 0.5 * u * mag
    if p["bias"] is not None:
        err = err + 2.0 ** -23 * np.abs(p["bias"])
    tol = u * np.abs(want) + 1.13 * err + 2.0 ** -24
    got = y.float().cpu().numpy().astype(np.float64)
    assert got.shape == want.shape
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.abs(got - want)[bad].max(), tol[bad].min(), np.argwhere(bad)[:5])


SHAPES = [(1, 1, 32), (1, 16, 64), (1, 300, 1024), (2, 129, 96), (3, 128, 256), (5, 257, 2080), (8, 130, 544),
          (9, 64, 288), (16, 200, 1056), (17, 200, 1056), (33, 129, 96), (45, 500, 4096), (64, 128, 320),
          (100, 257, 32), (128, 1000, 608), (129, 130, 1024), (255, 384, 672), (300, 777, 2080), (513, 256, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,rows,n", SHAPES)
def test_matches_oracle(lib, tokens, rows, n, dtype):
    p = problem(tokens, rows, n, dtype, tokens + rows + n)
    check(run(p, dtype, "none"), p, dtype, "none")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens", [1, 12, 70, 300])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_epilogue(lib, tokens, act, dtype):
    for bias, residual in ((True, False), (False, True), (True, True)):
        p = problem(tokens, 141, 480, dtype, 7, bias, residual)
        check(run(p, dtype, act), p, dtype, act)


@pytest.mark.parametrize("tokens,rows,n", [(1, 5120, 17408), (7, 4096, 14336), (40, 1024, 17408), (200, 700, 17408)])
def test_long_rows(lib, tokens, rows, n):
    p = problem(tokens, rows, n, "bf16", 11, residual=True)
    check(run(p, "bf16", "none"), p, "bf16", "none")


@pytest.mark.parametrize("tokens", [1, 6, 50, 140])
def test_widest_row(lib, tokens):
    p = problem(tokens, 40, 65536, "f16", 12)
    p["x"] = p["x"] / 64
    check(run(p, "f16", "none"), p, "f16", "none")


@pytest.mark.parametrize("tokens", [4, 90, 260])
def test_strided_rows_in_place_residual_and_out(lib, tokens):
    from gptq_post_weight_gb300 import _lib

    rows, n = 203, 352
    p = problem(tokens, rows, n, "bf16", 13, bias=True, residual=True)
    wide = torch.full((tokens, n + 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + n] = dev(p["x"], torch.bfloat16)
    out = torch.zeros(tokens, rows + 9, dtype=torch.bfloat16, device="cuda")
    out[:, :rows] = dev(p["residual"], torch.bfloat16)
    y = out[:, :rows]
    got = _lib.q4tp_linear(wide[:, 8:8 + n], dev(p["nib"]), dev(p["rungs"]), dev(p["tab"]),
                           bias=dev(p["bias"], torch.bfloat16), act="silu", residual=y, out=y)
    assert got is y and not out[:, rows:].any()
    check(y, p, "bf16", "silu")


@pytest.mark.parametrize("tokens", [1, 30, 150])
def test_zero_rows_large_rungs_and_non_finite_x(lib, tokens):
    p = problem(tokens, 70, 128, "f16", 14)
    p["tab"][3] = 0
    p["rungs"][4 * 5 + 1] = 200  # counts as scale 0
    y = run(p, "f16", "none")
    check(y, p, "f16", "none")
    assert not y[:, 3].any()
    x = dev(p["x"], torch.float16)
    x[0, 7] = float("nan")
    from gptq_post_weight_gb300 import _lib

    z = _lib.q4tp_linear(x, dev(p["nib"]), dev(p["rungs"]), dev(p["tab"]))
    assert z[0, 8:].isnan().all()
    if tokens > 1:
        assert torch.equal(z[1:], y[1:])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens", [2, 20, 200])
@pytest.mark.parametrize("scale", [2.0 ** -40, 2.0 ** 12])
def test_scales_far_from_one(lib, tokens, dtype, scale):
    # f16 weights are rounded relative to the row's largest rung, so their
    # own range does not matter.
    p = problem(tokens, 40, 160, dtype, 15)
    p["tab"] = (p["tab"] * np.float32(scale)).astype(np.float32)
    y = run(p, dtype, "none").float().cpu().numpy().astype(np.float64)
    want = serve.linear(p["x"], p["nib"], p["rungs"], p["tab"])
    if scale < 1 and dtype == "f16":
        want = serve.round_to(want, dtype)
        assert np.abs(y - want).max() <= 2.0 ** -24
    else:
        check(torch.from_numpy(y), p, dtype, "none")


def test_same_bits_every_time_and_on_another_stream(lib):
    for tokens in (3, 60, 180):
        p = problem(tokens, 640, 2048, "bf16", 16)
        a = run(p, "bf16", "none")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        b = run(p, "bf16", "none", stream=side)
        torch.cuda.synchronize()
        assert torch.equal(a, b)


def test_no_tokens(lib):
    p = problem(0, 20, 64, "bf16", 17)
    assert run(p, "bf16", "none").shape == (0, 20)


@pytest.mark.parametrize("tokens", [2, 60, 300])
def test_waits_run_out(lib, tokens):
    from gptq_post_weight_gb300 import _lib

    p = problem(tokens, 300, 1024, "bf16", 18)
    try:
        _lib.test_set_wait(1_000_000, no_loads=True)
        with pytest.raises(_lib.GptqError) as ei:
            run(p, "bf16", "none")
        assert ei.value.code == 6
    finally:
        _lib.test_set_wait()
    check(run(p, "bf16", "none"), p, "bf16", "none")


def test_on_quantized_weights(lib):
    # The operator on what quantize_group returns, against x times the
    # dequantised weights; the ladder as gptq_debias rewrites it stays in form.
    import synth
    from gptq_post_weight_gb300 import _lib

    cfg = synth.config("tiny")
    hp, w = synth.make_problem(cfg, "cpu")
    q = _lib.quantize_group(hp.cuda(), cfg.n, w.cuda(), cfg.lam)
    r = np.random.default_rng(19)
    for tokens in (1, 33):
        p = dict(x=serve.round_to(r.standard_normal((tokens, cfg.n)), "bf16"), bias=None, residual=None,
                 nib=q["nibbles"].cpu().numpy(), rungs=q["rungs"].cpu().numpy(), tab=q["tab"].cpu().numpy())
        check(run(p, "bf16", "none"), p, "bf16", "none")
