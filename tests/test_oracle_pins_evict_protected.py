"""Pins of the eviction's oracle for protected tokens next to weights that are
not finite, worked out by hand."""
import math

from oracle import paged as O


def test_protected_tokens_come_before_every_weight():
    order = [3, 0, 1, 2]
    for w in (math.nan, math.inf, 7.0):
        # order 0 is a sink, order 3 the newest; both stay whatever the others gathered
        assert O.evict_source([-1.0, -2.0, w, w], order, 4, 2, 3, 1, 1) == [0, 1]
        assert O.evict_source([math.nan, -2.0, w, w], order, 4, 3, 3, 1, 1) == [0, 1, 2]
    # among the others a NaN is above infinity, and infinity above the rest
    assert O.evict_source([1.0, math.inf, math.nan, 2.0], [0, 1, 2, 3], 4, 1, 3, 0, 0) == [2]
    assert O.evict_source([1.0, math.inf, 5.0, math.nan], [0, 1, 2, 3], 4, 2, 3, 0, 0) == [3, 1]
