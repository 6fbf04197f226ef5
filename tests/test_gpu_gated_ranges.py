"""gptq_q4tp_gated above 8 tokens where the rungs of one row, or the rows' ladders,
lie far apart.  Tolerances: test_gpu_gated.py's, which grant a weight half a step of f16.
"""
import numpy as np
import pytest

import test_gpu_gated as gated
from oracle import serve

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SHAPES = [(12, 70, 256), (45, 250, 1056), (1500, 2051, 256)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("apart", [12, 16, 20, 22])
@pytest.mark.parametrize("tokens,inner,n", SHAPES)
def test_rungs_of_a_row_far_apart(lib, tokens, inner, n, apart, dtype):
    # Every other group has a rung 2^-apart of its neighbours', and x as much larger
    # there: either half of the columns makes half of a sum.
    p = gated.problem(tokens, inner, n, dtype, 41)
    rungs = p["rungs"].reshape(2 * inner, n // 32)
    rungs[:] = rungs // 2 * 2
    rungs[:, 1::2] += 1
    p["rungs"] = rungs.reshape(-1)
    p["tab"][:, 1::2] = np.ldexp(p["tab"][:, 0::2], -apart)
    x = p["x"].reshape(tokens, n // 32, 32)
    x[:, 0::2] = np.ldexp(x[:, 0::2], -apart // 2)
    x[:, 1::2] = np.ldexp(x[:, 1::2], apart - apart // 2 - 1)
    p["x"] = serve.round_to(x.reshape(tokens, n), dtype)
    p["tab"] = np.ldexp(p["tab"], apart // 2).astype(np.float32)
    gated.check(gated.run(p, dtype, "none"), p, dtype, "none")


@pytest.mark.parametrize("tokens,inner,n", SHAPES)
def test_smallest_and_largest_ladders(lib, tokens, inner, n):
    # Rows of the gate near the lower end of f32 against rows of the up projection as
    # far the other way, and large ones of the gate alone.
    p = gated.problem(tokens, inner, n, "bf16", 43)
    size = np.zeros(2 * inner, dtype=int)
    size[0:inner:3], size[inner::3], size[1:inner:3] = -128, 95, 60
    p["tab"] = np.ldexp(p["tab"], size[:, None]).astype(np.float32)
    p["x"] = np.ldexp(p["x"], 20)
    gated.check(gated.run(p, "bf16", "none"), p, "bf16", "none")
