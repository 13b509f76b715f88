"""GPU tests of the eviction's protected tokens next to weights that are not
finite, bit for bit against the oracle's choice."""
import numpy as np
import pytest

from gpu_case import log
from test_gpu_paged import _evict

pytestmark = pytest.mark.gpu

@pytest.mark.parametrize("value", [np.nan, -np.nan, np.inf])
@pytest.mark.parametrize("lens,budget,recent,sinks", [
    ([300, 41], 40, 10, 4),       # several leave; one leaves
    ([5000, 2001], 2000, 100, 1),
    ([9000], 20, 30, 4),          # more protected tokens than the budget
])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_protects_against_weights_that_are_not_finite(gpu, value, lens, budget, recent, sinks, in_place):
    """The first and the last tokens stay first, also where every other weight
    is a NaN or infinite: those only come before the finite weights."""
    log(f"evict protected {value} {lens} -> {budget} in place:{in_place}")

    def most(s):
        s[np.random.default_rng(1).random(s.shape) < 0.9] = value

    def every(s):
        s[:] = value

    for weights in (most, every):
        _evict(gpu, lens, budget, recent, sinks, hk=1, dim=16, page=24, seed=budget, weights=weights, in_place=in_place)
