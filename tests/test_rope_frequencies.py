"""rope_frequencies' "yarn" pair by pair against the method's published formula, in 64 bits."""
from __future__ import annotations

import math

import pytest

import exact_io_aware_101_b200 as ea


@pytest.mark.parametrize("rot,base,factor,length,fast,slow", [
    (128, 10000.0, 16.0, 4096, 32.0, 1.0), (64, 500000.0, 4.0, 8192, 32.0, 1.0), (32, 10000.0, 40.0, 2048, 8.0, 2.0),
    (2, 10000.0, 4.0, 64, 32.0, 1.0),
])
def test_blend_is_linear_in_the_turns(rot, base, factor, length, fast, slow):
    got, attention = ea.rope_frequencies(rot, base=base, scaling="yarn", factor=factor, original_length=length,
                                         beta_fast=fast, beta_slow=slow, device="cpu")
    assert attention == 0.1 * math.log(factor) + 1.0
    between = 0
    for i in range(rot // 2):
        theta = base ** (-2.0 * i / rot)
        turns = length * theta / (2.0 * math.pi)          # the length over the pair's wavelength
        ramp = min(1.0, max(0.0, (turns - slow) / (fast - slow)))
        between += 0.0 < ramp < 1.0
        want = (1.0 - ramp) * theta / factor + ramp * theta
        assert abs(float(got[i]) - want) <= 1e-13 * want  # a few 64-bit roundings
    assert between or rot == 2
