"""GPU tests of the rotary calls at their limits: angles of far positions from frequencies to the last
unit, and gradients."""
import decimal
import math

import numpy as np
import pytest
import torch

from test_gpu_rope import F32, f64, i32, rand, sv  # noqa: F401

pytestmark = pytest.mark.gpu

TAU = decimal.Decimal("6.28318530717958647692528676655900576839433879875021164194988918461563281257242")


@pytest.mark.parametrize("at", [1, 131071, 2 ** 31 - 2, -70000, -2 ** 31])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_far_positions_to_the_bound(sv, at, base):  # noqa: F811
    """At any position a component is off by no more than 2^-21 of its pair's length: a frequency's
    half unit of 2^-64 of a turn is 2^-31 radians at most."""
    rot = 64
    with decimal.localcontext() as c:
        c.prec = 70
        turns = [(-(decimal.Decimal(2 * i) / rot) * decimal.Decimal(base).ln()).exp() / TAU
                 for i in range(rot // 2)]
        angle = np.array([[2 * math.pi * float(p * x % 1) for x in turns] for p in (at, at + 1)])
    x = rand((1, 2, 3, rot), 1, F32)
    xs, c, s = f64(x), np.cos(angle)[None, :, None], np.sin(angle)[None, :, None]
    a, b = xs[..., :rot // 2], xs[..., rot // 2:]
    want, size = np.concatenate([a * c - b * s, b * c + a * s], -1), np.hypot(a, b)
    size = np.concatenate([size, size], -1)
    rope = sv.Rope(rot, base=base)
    for kw in (dict(pos=i32([[at, at + 1]])), dict(start=i32([at]))):
        got = f64(sv.sv_rope(rope, x, **kw))
        assert (np.abs(got - want) <= size * 2.0 ** -21 + np.abs(want) * 2.0 ** -24 * 1.001).all()
