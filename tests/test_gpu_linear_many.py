"""gptq_q4tp_linear at the sizes that its rule sends to the kernel of SM pairs
(k_q4_many): tiles in one and in several rounds, ragged rows and tokens, its
epilogue and its bounded waits.  Which kernel ran is asked of the launch
accounting.  Tolerances: see test_gpu_linear.py."""
import numpy as np
import pytest

import test_gpu_linear as lin

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def kernels_of(call):
    from gptq_post_weight_gb300 import _lib

    _lib.profile_start(100)
    y = call()
    return y, {k: n for k, (_, n) in _lib.profile_stop().items() if n}


# One round of the pairs; two, the second nearly empty, the last row tile three
# rows and nothing for its second CTA; six, so that the row scales' turns come round.
SHAPES = [(1000, 3000, 800), (1500, 4099, 1056), (2000, 13001, 544)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,rows,n", SHAPES)
def test_matches_oracle(lib, tokens, rows, n, dtype):
    p = lin.problem(tokens, rows, n, dtype, tokens)
    # Row scales far apart: another tile's would show.
    p["tab"] = np.ldexp(p["tab"], (np.arange(rows) // 64 % 7)[:, None]).astype(np.float32)
    y, ran = kernels_of(lambda: lin.run(p, dtype, "none"))
    assert ran == {"q4_linear_many": 1}
    lin.check(y, p, dtype, "none")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("wide", [0, 5, 16])
def test_epilogue_in_place_and_strided(lib, act, dtype, wide):
    # y = act(x W^T + b) + y over rows of y that are dense, odd and of whole vectors apart.
    from gptq_post_weight_gb300 import _lib

    tokens, rows, n = 1500, 4099, 1056
    p = lin.problem(tokens, rows, n, dtype, 31, bias=True, residual=True)
    out = torch.zeros(tokens, rows + wide, dtype=lin.DT[dtype], device="cuda")
    out[:, :rows] = lin.dev(p["residual"], lin.DT[dtype])
    y = out[:, :rows]
    x = torch.full((tokens, n + 24), float("nan"), dtype=lin.DT[dtype], device="cuda")
    x[:, 16:16 + n] = lin.dev(p["x"], lin.DT[dtype])
    got, ran = kernels_of(lambda: _lib.q4tp_linear(
        x[:, 16:16 + n], lin.dev(p["nib"]), lin.dev(p["rungs"]), lin.dev(p["tab"]),
        bias=lin.dev(p["bias"], lin.DT[dtype]), act=act, residual=y, out=y))
    _lib.serve_check()
    assert got is y and not out[:, rows:].any() and ran == {"q4_linear_many": 1}
    lin.check(y, p, dtype, act)


def test_zero_rows_large_rungs_and_another_stream(lib):
    tokens, rows, n = 1500, 4099, 1056
    p = lin.problem(tokens, rows, n, "f16", 32)
    p["tab"][[0, 255, 256, 4098]] = 0
    p["rungs"][np.random.default_rng(33).integers(0, p["rungs"].size, 500)] = 200  # counts as scale 0
    y, ran = kernels_of(lambda: lin.run(p, "f16", "none"))
    assert ran == {"q4_linear_many": 1}
    lin.check(y, p, "f16", "none")
    assert not y[:, [0, 255, 256, 4098]].any()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = lin.run(p, "f16", "none", stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, again)


def test_waits_run_out(lib):
    from gptq_post_weight_gb300 import _lib

    p = lin.problem(1500, 4099, 1056, "bf16", 34)
    try:
        _lib.test_set_wait(1_000_000, no_loads=True)
        with pytest.raises(_lib.GptqError) as ei:
            lin.run(p, "bf16", "none")
        assert ei.value.code == 6
    finally:
        _lib.test_set_wait()
    y, ran = kernels_of(lambda: lin.run(p, "bf16", "none"))
    assert ran == {"q4_linear_many": 1}
    lin.check(y, p, "bf16", "none")
