"""The comparison of the attention's GPU tests says so when an output is not a
number: Python's max and a running maximum would drop it."""

import numpy as np
import pytest

from parity_util import over_bound

NAN, INF = float("nan"), float("inf")


def test_within_and_over():
    ref = np.arange(6.0).reshape(2, 3)
    assert over_bound(ref, ref, 0.0) == 0
    assert over_bound(ref + 0.5, ref, 0.5) <= 0
    assert over_bound(ref - 1, ref, 0.25) == 0.75
    worse = ref.copy()
    worse[1, 2] += 3
    assert over_bound(worse, ref, np.ones((2, 3))) == 2
    assert over_bound(np.zeros((0, 4)), np.zeros((0, 4)), 0.0) <= 0


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("at", [0, 3, 5])
def test_what_is_not_finite_is_over(bad, at):
    ref = np.arange(6.0)
    for which in range(3):
        args = [ref.copy(), ref.copy(), np.full(6, 1e9)]
        args[which][at] = bad
        assert over_bound(*args) == INF
    assert max(-1.0, NAN) == -1.0          # what a running maximum makes of it
