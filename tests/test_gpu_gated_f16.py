"""gptq_q4tp_gated of f16 above 8 tokens, whose weights enter partly as two numbers:
waits that run out, strided inputs and outputs, and sums taken again from a strided x."""
import numpy as np
import pytest

import test_gpu_gated as gated
import test_gpu_linear as lin
from oracle import serve

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,inner,n", [(9, 40, 96), (100, 128, 608), (1500, 2051, 1056)])
def test_waits_run_out(lib, tokens, inner, n):
    from gptq_post_weight_gb300 import _lib

    p = gated.problem(tokens, inner, n, "f16", 23)
    want = gated.run(p, "f16", "silu")
    try:
        _lib.test_set_wait(1_000_000, no_loads=True)
        with pytest.raises(_lib.GptqError) as ei:
            gated.run(p, "f16", "silu")
        assert ei.value.code == 6
    finally:
        _lib.test_set_wait()
    assert torch.equal(gated.run(p, "f16", "silu"), want)


@pytest.mark.parametrize("tokens,inner,n", [(1, 203, 352), (9, 203, 352), (90, 203, 352), (1500, 2051, 1056)])
def test_strides_and_infinite_activations(lib, tokens, inner, n):
    from gptq_post_weight_gb300 import _lib

    p = gated.problem(tokens, inner, n, "f16", 13, bias=True)
    p["nib"][:] |= 0x11  # no code is 8: no weight 0
    if tokens > 8:
        p["x"][2, 3], p["x"][7, n - 1], p["x"][5, 130] = np.inf, -np.inf, np.inf
    plain = gated.run(p, "f16", "none")
    wide = torch.full((tokens, n + 40), float("nan"), dtype=torch.float16, device="cuda")
    wide[:, 8:8 + n] = lin.dev(p["x"], torch.float16)
    out = torch.zeros(tokens, inner + 5, dtype=torch.float16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = _lib.q4tp_gated(wide[:, 8:8 + n], lin.dev(p["nib"]), lin.dev(p["rungs"]), lin.dev(p["tab"]),
                        bias=lin.dev(p["bias"], torch.float16), act="none", out=out[:, :inner], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, plain) and not out[:, inner:].any()
    if tokens > 8:
        some = [2, 5, 7]
        want = serve.gated(p["x"][some], p["nib"], p["rungs"], p["tab"], p["bias"], "none")
        assert np.isinf(want).all()
        np.testing.assert_array_equal(y[some].float().cpu().numpy(), want.astype(np.float32))
        assert torch.isfinite(y[[0, 1, 3, 4, 6, 8]]).all()
