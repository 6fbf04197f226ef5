"""The angles of gptq_rotary next to the quarters of a turn, where the sine or the
cosine vanishes and an error of the angle is all that is left, and all around.

Tolerance, with x = (1, 0) so that a pair becomes gain (cos, sin), gain a power of
two: the angle is rounded to 2^-32 of a turn (pi 2^-32) and its rest over the
nearest quarter, at most an eighth of a turn, to f32 (half of 2^-27 of a turn: pi
2^-27); sine and cosine are good to two f32 steps (2^-22 of them), and the result rounds
to T: half a step, 2^-8 (bf16) or 2^-11 (f16) of it, or half of f16's smallest number.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("position", [1, -1, 7001, 123456789012345])
def test_angles_near_the_quarters(lib, position, layout, dtype):
    from gptq_post_weight_gb300 import _lib

    r = np.random.default_rng(abs(position) % 1000)
    pairs, gain = 512, 4096.0
    # 2^64ths of a turn: eighths of a turn, and steps of 2^-32 of one and parts of them beside.
    near = [k * 2 ** 61 + sign * int(step * 2 ** 32) for k in range(8) for sign in (1, -1)
            for step in (0, 0.4, 0.6, 1, 7, 15.5, 31, 33, 63, 64, 65, 97, 127, 129, 1000.3, 1e6, 2e8)]
    turn = near + [int(v) for v in r.integers(0, 2 ** 63, pairs - len(near))]
    back = pow(position, -1, 2 ** 64)
    turns = [((t * back) % 2 ** 64 + 2 ** 63) % 2 ** 64 - 2 ** 63 for t in turn]
    x = torch.zeros(1, 1, 2 * pairs, dtype=DT[dtype], device="cuda")
    first, second = (slice(0, pairs), slice(pairs, None)) if layout == "half" else (slice(0, None, 2), slice(1, None, 2))
    x[..., first] = 1
    y = _lib.rotary(x, torch.tensor([position], device="cuda"), torch.tensor(turns, device="cuda"), layout=layout,
                    gain=gain).double().cpu().numpy()[0, 0]
    angle = np.array([2 * math.pi * ((t + 2 ** 63) % 2 ** 64 - 2 ** 63) / 2 ** 64 for t in turn])
    for got, want in ((y[first], gain * np.cos(angle)), (y[second], gain * np.sin(angle))):
        err = gain * math.pi * (2.0 ** -27 + 2.0 ** -32) + 2.0 ** -22 * np.abs(want)
        tol = err + HALF[dtype] * (np.abs(want) + err) + 2.0 ** -25
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), [(hex(turn[i]), got[i], want[i], tol[i]) for i in np.flatnonzero(bad)[:4]]
