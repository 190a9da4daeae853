"""The element checks of the GPU tests, on the CPU: a NaN or an infinity is out
of every tolerance, wherever it stands. The mistakes are planted in the
oracle's own gradient.
"""
import numpy as np
import pytest

import oracle
from gpu_common import assert_close, assert_within


def _gradient():
    rng = np.random.default_rng(1)
    l = rng.standard_normal((6, 5)).astype(np.float32)
    ids = np.argsort(-l, axis=1, kind="stable")[:, :2]
    return oracle.route_backward(l, ids, rng.standard_normal((6, 2)), True)


def test_what_is_within_passes():
    g = _gradient()
    assert_within(g, g, 0.0)
    assert_within(g + 1e-9, g, 2e-9)
    assert_within(0.0, np.zeros((2, 0)), 1.0)
    assert_close(g, g, (0.0, 0.0))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_what_is_no_number_does_not(value):
    g = _gradient()
    for at in ((0, 0), (3, 2), (5, 4)):
        bad = g.copy()
        bad[at] = value
        for args in ((bad, g, 1e30), (g, bad, 1e30), (bad, bad, 1e30)):
            with pytest.raises(AssertionError):
                assert_within(*args)
        with pytest.raises(AssertionError):
            assert_within(g, g, np.where(np.isfinite(bad), 1.0, value))
        with pytest.raises(AssertionError):
            assert_close(bad, g, (1.0, 1.0))
    with pytest.raises(AssertionError):
        assert_within(np.full_like(g, value), g, 1e30)


def test_one_step_past_the_allowance_does_not():
    g = _gradient()
    bad = g.copy()
    bad[2, 1] += 1e-6
    with pytest.raises(AssertionError):
        assert_within(bad, g, 0.9e-6)
