"""rotary_frequencies: turns per position in units of 2^-64 (no GPU)."""
import math

import pytest

from w4afp8_mixture_experts_gb300 import rotary_frequencies, rotary_yarn_scale


def _radians(t):
    return [2 * math.pi * v * 2.0 ** -64 for v in t.tolist()]


def _close(a, b):
    # a fraction of a turn has 64 bits: 2 pi 2^-64 radians, beside fp64 roundings
    return all(abs(x - y) <= 1e-15 * abs(y) + 4e-19 for x, y in zip(a, b)) and len(a) == len(b)


@pytest.mark.parametrize("dim", [2, 64, 128])
def test_plain_and_linear(dim):
    want = [10000.0 ** (-2 * i / dim) for i in range(dim // 2)]
    assert _close(_radians(rotary_frequencies(dim, device="cpu")), want)
    assert _close(_radians(rotary_frequencies(dim, scaling="linear", factor=8.0, device="cpu")), [w / 8 for w in want])


def test_ntk():
    base = 5e5 * 4.0 ** (64 / 62)
    want = [base ** (-2 * i / 64) for i in range(32)]
    assert _close(_radians(rotary_frequencies(64, 5e5, scaling="ntk", factor=4.0, device="cpu")), want)


def test_yarn_keeps_fast_and_divides_slow():
    got = _radians(rotary_frequencies(64, scaling="yarn", factor=40.0, length=4096, device="cpu"))
    plain = [10000.0 ** (-2 * i / 64) for i in range(32)]
    for f, p in zip(got, plain):
        turns = p * 4096 / (2 * math.pi)
        # the ramp begins and ends at whole pairs, which lie 10000^(2 / 64) = 1.334 apart: at most 32 * 1.334 = 42.7 turns
        # and at least 1 / 1.334 = 0.75
        if turns > 42.7:
            assert _close([f], [p])
        elif turns < 0.74:
            assert _close([f], [p / 40])
        else:
            assert p / 40 * (1 - 1e-12) <= f <= p * (1 + 1e-12)
    assert rotary_yarn_scale(40.0) == pytest.approx(0.1 * math.log(40) + 1) and rotary_yarn_scale(1.0) == 1.0


def test_given_frequencies_keep_whole_turns_out():
    f = [0.5, 4.0, -1.0, 7.0]  # 7 radians are a turn and more, -1 a turn backwards
    got = rotary_frequencies(8, inv_freq=f, device="cpu")
    for t, v in zip(got.tolist(), f):
        a = 2 * math.pi * t * 2.0 ** -64
        assert abs(math.sin(a - v)) <= 1e-15 * 8 and math.cos(a - v) > 0


@pytest.mark.parametrize("kw", [dict(dim=3), dict(dim=0), dict(dim=8, scaling="cubic"), dict(dim=8, factor=0.0),
                                dict(dim=8, base=1.0), dict(dim=2, scaling="ntk"), dict(dim=8, inv_freq=[1.0]),
                                dict(dim=4, inv_freq=[1.0, math.inf]), dict(dim=8, length=0),
                                dict(dim=8, factor=math.nan)])
def test_refusals(kw):
    with pytest.raises(ValueError):
        rotary_frequencies(device="cpu", **kw)


@pytest.mark.parametrize("dim,base,factor", [(64, 10000.0, 8.0), (128, 5e5, 4.0), (4, 100.0, 2.0)])
def test_given_frequencies_are_scaled_like_those_of_a_base(dim, base, factor):
    f = [base ** (-2 * i / dim) for i in range(dim // 2)]
    for scaling in ("none", "linear", "ntk"):
        want = _radians(rotary_frequencies(dim, base, scaling=scaling, factor=factor, device="cpu"))
        assert _close(_radians(rotary_frequencies(dim, base, scaling=scaling, factor=factor, inv_freq=f, device="cpu")), want)


def test_ntk_of_given_frequencies():
    # the first pair keeps its frequency, the last is divided by factor, whatever the frequencies are
    got = _radians(rotary_frequencies(8, scaling="ntk", factor=8.0, inv_freq=[1.0, 0.3, 0.2, 0.1], device="cpu"))
    assert _close(got, [1.0, 0.3 * 8.0 ** (-1 / 3), 0.2 * 8.0 ** (-2 / 3), 0.1 / 8.0])
    with pytest.raises(ValueError, match="ntk"):
        rotary_frequencies(2, scaling="ntk", inv_freq=[1.0], device="cpu")


@pytest.mark.parametrize("dim,base", [(64, 10000.0), (128, 5e5)])
def test_yarn_of_given_frequencies_of_the_same_base(dim, base):
    # their places among the base's pairs are logarithms, off by 1e-13 at most: as much of the blend's width of 10 pairs
    f = [base ** (-2 * i / dim) for i in range(dim // 2)]
    want = _radians(rotary_frequencies(dim, base, scaling="yarn", factor=40.0, device="cpu"))
    got = _radians(rotary_frequencies(dim, base, scaling="yarn", factor=40.0, inv_freq=f, device="cpu"))
    assert all(abs(x - y) <= 1e-12 * y for x, y in zip(got, want))


@pytest.mark.parametrize("f", [[500000.0 ** (-2 * i / 64) for i in range(32)], [0.9 ** i for i in range(32)],
                               [1e-5 * (i + 1) for i in range(32)], [0.0] + [-0.8 ** i for i in range(31)]])
def test_yarn_of_given_frequencies_goes_by_their_own_turns(f):
    # the default base's pairs lie 10000^(2 / 64) = 1.334 apart, so that the blend ends within 42.7 and 0.75 turns
    got = _radians(rotary_frequencies(64, scaling="yarn", factor=40.0, length=4096, inv_freq=f, device="cpu"))
    for g, p in zip(got, f):
        turns = abs(p) * 4096 / (2 * math.pi)
        if turns > 42.7:
            assert _close([g], [p])
        elif turns < 0.74:
            assert _close([g], [p / 40])
        else:
            assert abs(p) / 40 * (1 - 1e-12) <= abs(g) <= abs(p) * (1 + 1e-12)
