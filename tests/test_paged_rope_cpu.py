"""RopeSpec's frequencies against their definitions, pair by pair."""
import math

import pytest

import causal_sliding_window_rope_b200 as cs


@pytest.mark.parametrize("R,base,original,factor", [(128, 1e4, 65536, 4.0), (64, 1e4, 65536, 4.0), (16, 1e4, 32768, 4.0),
                                                    (128, 1e4, 2048, 4.0), (128, 5e5, 8192, 8.0), (32, 1e4, 10 ** 9, 2.0)])
def test_ramped_frequencies(R, base, original, factor):
    """Pairs between the one that turns beta_fast = 32 times within the original length (rounded down) and the one that
    turns beta_slow = 1 times (rounded up) are mixed along a straight line, also where the line ends past the last pair;
    so a pair that turns more than once keeps a part of its frequency, and the last of many turns keeps all of it."""
    got = cs.RopeSpec(R, scaling="yarn", factor=factor, base=base, original_length=original).frequencies
    pair_of = lambda turns: R * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
    low, high = max(0, math.floor(pair_of(32))), min(R - 1, math.ceil(pair_of(1)))
    for i, f in enumerate(got):
        w = base ** (-2 * i / R)
        ramp = min(1.0, max(0.0, (i - low) / (high - low))) if high > low else float(i > low)
        assert f == pytest.approx(w * (1 - ramp) + w / factor * ramp, rel=1e-12, abs=0.0), i
        turns = original * w / (2 * math.pi)
        if turns > 1.0:
            assert f > w / factor * (1 + 1e-9), (i, turns)


@pytest.mark.parametrize("factor,want", [(0.25, 1.0), (1.0, 1.0), (4.0, 1 + 0.1 * math.log(4.0))])
def test_a_context_that_is_not_stretched_keeps_cos_and_sin(factor, want):
    assert cs.RopeSpec(64, scaling="yarn", factor=factor, original_length=2048).attention_factor == pytest.approx(want)
