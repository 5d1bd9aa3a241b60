"""The attention-side operators where their inputs are unusual: far positions, scales that no write makes, rows that
no sequence covers, other streams."""
from __future__ import annotations

import math
import random
from fractions import Fraction

import pytest
import torch

from turns import TWO_PI

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def m():
    from int4_routed_expert_gb300 import build as b
    b.build()
    import int4_routed_expert_gb300 as mod
    mod.load()
    return mod


def test_rope_angles_at_far_positions(m):
    """Rotating (1, 0) gives the cosine and the sine themselves.  Off by at most 2 ulp of the library's function
    (2^-23) and half an ulp of the step by the derivatives (2^-25); the angle's 2^-32 turns are 2^-29."""
    r = random.Random(5)
    freq = [1.0] + [r.uniform(0.5, 1.2) for _ in range(95)] + [math.exp(r.uniform(-16, 0)) for _ in range(32)]
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, 2 ** 30 + 7, -1999999999, 4000037, 131071, 1000, 1, 0]
    rope = m.Rope(256, inv_freq=freq, amplitude=1.0)
    x = torch.zeros(len(pos), 1, 256, device=DEV)
    x[..., :128] = 1
    y = rope.apply(x, torch.tensor(pos, dtype=torch.int32, device=DEV)).double().cpu()
    for t, p in enumerate(pos):
        angle = [float(p * Fraction(f) % TWO_PI) for f in freq]
        want = torch.tensor([math.cos(a) for a in angle] + [math.sin(a) for a in angle], dtype=torch.float64)
        assert float((y[t, 0] - want).abs().max()) <= 2.0 ** -23 + 2.0 ** -25 + 2.0 ** -29
