"""Frequencies of rotary positions: closed forms at both ends and in between."""
import math

import pytest

from precision_rl_rollout_gb300.positions import rope_frequencies


def test_plain():
    f, m = rope_frequencies(8, base=16.0)
    assert f == [1.0, 0.5, 0.25, 0.125] and m == 1.0
    assert rope_frequencies(2)[0] == [1.0]


def test_linear_and_base():
    plain = rope_frequencies(128)[0]
    assert rope_frequencies(128, scaling="linear", factor=4)[0] == [x / 4 for x in plain]
    f, m = rope_frequencies(128, scaling="base", factor=4)
    assert m == 1.0 and f[0] == 1.0
    assert f[-1] == pytest.approx(plain[-1] / 4, rel=1e-12)             # the slowest pair reaches the longer context
    assert all(b <= a for a, b in zip(plain, f))
    assert rope_frequencies(2, scaling="base", factor=8)[0] == [1.0]    # one pair: nothing to stretch


def test_bands():
    R, trained, factor = 128, 4096, 8.0
    plain = rope_frequencies(R)[0]
    f, m = rope_frequencies(R, scaling="bands", factor=factor, trained=trained)
    assert m == pytest.approx(0.1 * math.log(8) + 1)
    for a, b in zip(plain, f):
        turns = trained * a / (2 * math.pi)
        if turns >= 32:
            assert b == a
        elif turns <= 1:
            assert b == pytest.approx(a / factor, rel=1e-15)
        else:
            k = (turns - 1) / 31
            assert b == pytest.approx(a * (k + (1 - k) / factor), rel=1e-14) and a / factor < b < a
    assert rope_frequencies(R, scaling="bands", factor=1.0, trained=trained)[0] == pytest.approx(plain, rel=1e-15)


@pytest.mark.parametrize("kw", [dict(R=3), dict(R=0), dict(R=8, base=0.0), dict(R=8, factor=0.5),
                                dict(R=8, scaling="other"), dict(R=8, scaling="bands", factor=2.0),
                                dict(R=8, scaling="bands", factor=2.0, trained=10, slow=2.0, fast=2.0)])
def test_refusals(kw):
    with pytest.raises(ValueError):
        rope_frequencies(**kw)
