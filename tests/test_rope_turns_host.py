"""The rotation's table scaled by parts: which ramp it is."""
import decimal

import numpy as np
import pytest


@pytest.mark.parametrize("rot,base,factor,length,fast,slow", [
    (64, 10000.0, 8.0, 4096, 32.0, 1.0), (128, 500000.0, 32.0, 8192, 32.0, 1.0), (128, 1e6, 4.0, 32768, 4.0, 0.5),
    (96, 500000.0, 8.0, 8192, 4.0, 1.0)])
def test_parts_ramp_over_turns(rot, base, factor, length, fast, slow):
    """A pair keeps the share (turns - slow) / (fast - slow) of its rate, within [0, 1], turns in `length` positions;
    the rest of the rate is divided by factor.  (Not a ramp over the pairs' numbers.)"""
    from lora_serving_amd import mlora as m
    got = m.mlora_rope_turns(rot, base, m.MLORA_ROPE_PARTS, factor=factor, orig_len=length, fast=fast,
                             slow=slow).numpy().view(np.uint64)
    decimal.getcontext().prec = 50
    D = decimal.Decimal
    pi = D("3.1415926535897932384626433832795028841971693993751")
    between = 0
    for i in range(rot // 2):
        f = D(base) ** (D(-2 * i) / rot) / (2 * pi)
        keep = min(D(1), max(D(0), (length * f - D(slow)) / (D(fast) - D(slow))))
        between += 0 < keep < 1
        want = (f * keep + f / D(factor) * (1 - keep)) * 2 ** 64
        # half a unit of the fixed point; a 64-bit significand's power, ramp and products (some 2^-64, relative to f)
        assert abs(int(got[i]) - want) <= D(0.5) + f * 2 ** 64 * D(2.0 ** -60)
    assert between >= 2
