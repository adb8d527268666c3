"""The angles of gdn_rope, on pairs (1, 0), which become (cosine, sine), against 50 decimal digits.

Tolerance of an element, from the stated precision: the angle to 2^-32 of a turn and |p| 2^-52 / min(factor, 1) of a turn for
its frequency (2 pi of that in the result); and of the value itself 2^-21: the reduced angle as a float 2^-24, sine or
cosine 2 ulp (2^-22), the product with 1 and the magnitude 1, the sum with 0 and the store none."""
import math
from decimal import Decimal, getcontext

import pytest
import torch

from hybrid_gated_deltanet_gb300 import binding as gb
from parts_cases import i32

pytestmark = pytest.mark.gpu
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494")


def _turns(p, theta, i, rot, factor):
    """p theta^(-2i/rot) / factor / 2 pi, less the nearest whole turn."""
    getcontext().prec = 60
    f = (Decimal(theta).ln() * (-2 * i) / rot).exp() / Decimal(factor)
    t = p * f / (2 * PI)
    return float(t - t.to_integral_value())


# 355 is 113 pi less 3e-5, so that odd multiples end just short of half a turn, and even ones of a whole one
NEAR_HALF_TURNS = [355 * m for m in (1, -1, 3, 5, 7, 9, 11, 13, -15, 17, 19, 21, 2, 4, -6, 101, 1001)]
POSITIONS = NEAR_HALF_TURNS + [0, 1, -1, 11, 344, -344, 12345, (1 << 20) - 1, 1 << 20, -(1 << 20), 10 ** 9 + 7, 2 ** 31 - 1, -2 ** 31]


@pytest.mark.parametrize("heads", [1, 3])  # the form for many tokens (a thread walks over all heads) and the one for few
@pytest.mark.parametrize("layout", [gb.ROPE_HALF, gb.ROPE_INTERLEAVED])
@pytest.mark.parametrize("theta,factor", [(10000.0, 1.0), (5e5, 8.0), (1e7, 0.25), (10000.0, 2.0 ** -10)])
def test_rope_angles(theta, factor, layout, heads):
    rot = 96
    x = torch.zeros((len(POSITIONS), heads, 128), device="cuda")
    first = slice(0, rot // 2) if layout == gb.ROPE_HALF else slice(0, rot, 2)
    second = slice(rot // 2, rot) if layout == gb.ROPE_HALF else slice(1, rot, 2)
    x[..., first] = 1.0
    gb.gdn_rope(gb.gdn_rope_plan(gb.RopeConfig(128, rot, theta, layout, gb.F32, factor)), i32(POSITIONS), x, None)
    t = torch.tensor([[_turns(p, theta, i, rot, factor) for i in range(rot // 2)] for p in POSITIONS], dtype=torch.float64)
    slack = 2 * math.pi * (2.0 ** -32 + torch.tensor(POSITIONS).double().abs() * 2.0 ** -52 / min(factor, 1.0))[:, None, None]
    got = x.cpu().double()
    for part, want in ((first, torch.cos(2 * math.pi * t)), (second, torch.sin(2 * math.pi * t))):
        want = want[:, None].expand(-1, heads, -1)
        err = (got[..., part] - want).abs()
        bad = ~(err <= slack + 2.0 ** -21 * want.abs() + 2.0 ** -50)  # (the 64-bit sine of the oracle: 2^-50)
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, at {bad.nonzero()[0].tolist()}, off by {float(err[bad].max()):.3e}"
