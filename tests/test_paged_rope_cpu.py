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


@pytest.mark.parametrize("kw,want", [
    (dict(), 5e5), (dict(base=2e4), 2e4), (dict(base=10000.0), 1e4),
    (dict(scaling="linear", factor=4.0), 5e5), (dict(scaling="ntk", factor=2.0), 5e5),
    (dict(scaling="yarn", factor=4.0, original_length=8192), 5e5),
])
def test_the_layers_base_is_the_default(kw, want, monkeypatch):
    """What attn_paged_append hands to the library: frequencies of the layer's base unless the RopeSpec names one."""
    seen = []

    class Calls:
        @staticmethod
        def append(*a):
            s = cs.CswattnRope.from_address(a[10].address)
            seen.append([s.frequencies[i] for i in range(s.rotary_dim // 2)])
    monkeypatch.setattr(cs, "_paged", Calls)
    rope = cs.RopeSpec(64, **kw)
    for base in (5e5, 1e4, 5e5):
        spec = cs.LayerSpec(1, 16, 2, 1, 64, 16, has_ve=False, rope_base=base)
        cs.attn_paged_append(spec, *[None] * 8, rope=rope)
        explicit = cs.RopeSpec(64, **{**kw, "base": want if want != 5e5 else base})
        assert seen[-1] == list(explicit.frequencies)
    assert seen[0] == seen[2] and (seen[0] != seen[1]) == (want == 5e5)
    own = cs.RopeSpec(16, frequencies=[0.5] * 8)
    cs.attn_paged_append(cs.LayerSpec(1, 16, 2, 1, 64, 16, has_ve=False, rope_base=5e5), *[None] * 8, rope=own)
    assert seen[-1] == [0.5] * 8
