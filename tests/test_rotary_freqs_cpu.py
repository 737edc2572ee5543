"""Frequencies of MOE_ROTARY_RAMP against their formula, for trained contexts from a few positions to very long ones."""
import math

import numpy as np
import pytest

from routed_expert_execution_amd import moe


def _ramp(rot, base, context, factor, fast, slow):
    """64 bits: pair i keeps 1 - t_i of its frequency and t_i of that divided by factor."""
    half = rot // 2
    turning = lambda n: rot / 2 * math.log(context / (2 * math.pi * n)) / math.log(base)  # the pair that turns n times
    low, high = max(math.floor(turning(fast)), 0), min(math.ceil(turning(slow)), rot - 1)
    i = np.arange(half, dtype=np.float64)
    plain = base ** (-2 * i / rot)
    if high <= 0:  # no pair turns more than `slow` times
        t = np.ones(half)
    elif low >= half:
        t = np.zeros(half)
    else:
        t = np.clip((i - low) / (high - low), 0, 1)
    return plain * ((1 - t) + t / factor)


@pytest.mark.parametrize("rot,base,context,factor,fast,slow", [
    (128, 10000.0, 2048, 4, 32, 1), (128, 10000.0, 131072, 4, 32, 1), (64, 10000.0, 65536, 4, 32, 1), (64, 10000.0, 4096, 8, 32, 1), (128, 500000.0, 8192, 8, 32, 1),
    (96, 1e6, 32768, 2.5, 16, 2), (128, 10000.0, 1 << 30, 4, 32, 1), (2, 10000.0, 4096, 4, 32, 1), (64, 10000.0, 100, 4, 32, 1), (64, 10000.0, 6, 4, 32, 1), (64, 10000.0, 1, 4, 32, 1),
    (64, 10.0, 1e9, 4, 32, 1), (256, 10000.0, 1e5, 16, 1.5, 1.25)])
def test_ramp_is_its_formula(rot, base, context, factor, fast, slow):
    got, scale = moe.moe_rotary_freqs(rot, base, moe.MOE_ROTARY_RAMP, factor, context, fast, slow)
    want = _ramp(rot, base, context, factor, fast, slow)
    # the result's rounding to fp32 (2^-24), and the power's and the ramp's in 64 bits
    assert (np.abs(got - want) <= 2.0 ** -24 * want * (1 + 1e-6) + 1e-13 * want).all(), (got / want)
    assert abs(scale - (0.1 * math.log(factor) + 1)) <= 2.0 ** -24 * scale


@pytest.mark.parametrize("rot,context", [(128, 131072), (64, 65536), (64, 100), (64, 6), (128, 4096)])
def test_ramp_divides_wholly_only_what_turns_slowly(rot, context):
    factor, fast, slow = 4.0, 32.0, 1.0
    got, _ = moe.moe_rotary_freqs(rot, 10000.0, moe.MOE_ROTARY_RAMP, factor, context, fast, slow)
    plain, _ = moe.moe_rotary_freqs(rot)
    turns = context * plain.astype(np.float64) / (2 * math.pi)
    share = got / plain
    assert np.allclose(share[turns >= fast], 1, rtol=2.0 ** -22)
    # the last pair of the ramp is rounded outwards: a pair that turns less than `slow` times by up to one step of the pairs' numbers
    step = 10000.0 ** (2 / rot)
    assert np.allclose(share[turns * step <= slow], 1 / factor, rtol=2.0 ** -22)
    assert (share[turns > slow] > 1 / factor * (1 + 1e-3)).all()
