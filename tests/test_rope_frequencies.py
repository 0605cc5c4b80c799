"""Scalings of rotary frequencies against what their description says of each pair."""
import math

import numpy as np
import pytest

import attention_backward_gb300 as ab


@pytest.mark.parametrize("R,length,base,slow,fast", [
    (64, 131072, 1e4, 1.0, 32.0), (64, 65536, 1e4, 1.0, 32.0), (128, 131072, 1e4, 1.0, 32.0), (16, 32768, 1e4, 1.0, 32.0),
    (32, 1 << 20, 1e4, 1.0, 32.0), (64, 8192, 1e4, 1.0, 32.0), (64, 100, 1e4, 1.0, 32.0), (16, 4, 1e4, 1.0, 32.0),
    (2, 4096, 1e4, 1.0, 32.0), (128, 262144, 5e5, 2.0, 16.0), (64, 10 ** 9, 1e4, 1.0, 32.0)])
def test_parts_by_turns(R, length, base, slow, fast):
    """Pairs that turn fewer than ``slow`` times in ``length`` positions are divided by the
    factor, those that turn more than ``fast`` times left, the others in between; where the pairs
    that turn ``slow`` and ``fast`` times lie among the first R, the ramp is the line between
    them (their places rounded outwards)."""
    factor = 4.0
    f = np.array(ab.rope_frequencies(R, base)[0])
    got = np.array(ab.rope_frequencies(R, base, "parts", factor, length, fast, slow)[0]) / f
    turns = f * length / (2 * math.pi)
    assert (np.diff(got) <= 1e-15).all()
    assert np.allclose(got[turns < slow], 1 / factor, rtol=1e-14)
    assert (got[turns > fast * base ** (2 / R)] == 1).all()  # (a pair further on: rounded places)
    between = (turns > slow * base ** (2 / R)) & (turns < fast)
    between[0] = False  # (the ramp begins at the first pair, with nothing taken off, where that turns too seldom)
    assert (got[between] > 1 / factor).all() and (got[between] < 1).all()
    at = [R / 2 * math.log(length / (2 * math.pi * t), base) for t in (fast, slow)]
    if 0 <= at[0] and at[1] <= R - 1:
        a, e = math.floor(at[0]), math.ceil(at[1])
        part = np.clip((np.arange(R // 2) - a) / (e - a), 0, 1)
        assert np.allclose(got, 1 - part + part / factor, rtol=1e-13)


def test_parts_whose_slowest_pair_turns():
    """64 columns, 131072 positions: the last pair turns 2.78 times, two thirds along the ramp."""
    f, p = ab.rope_frequencies(64)[0], ab.rope_frequencies(64, scaling="parts", factor=4.0, original_length=131072)[0]
    assert f[-1] * 131072 / (2 * math.pi) > 2.7
    a, e = 22, 35  # floor and ceiling of the pairs that turn 32 times and once
    part = (31 - a) / (e - a)
    assert abs(p[-1] / f[-1] - (1 - part + part / 4)) < 1e-13


@pytest.mark.parametrize("factor,scale", [(0.5, 1.0), (1.0, 1.0), (1e-3, 1.0), (math.e, 1.1), (40.0, 1 + math.log(40.0) / 10)])
def test_parts_never_scale_the_result_down(factor, scale):
    assert abs(ab.rope_frequencies(64, scaling="parts", factor=factor, original_length=4096)[1] - scale) < 1e-15
