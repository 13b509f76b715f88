"""GPU tests of the eviction on both sides of 65536 tokens a head, up to which
a workgroup keeps a head's keys in registers; beyond, every pass reads them
again. Bit for bit against the oracle's choice."""
import numpy as np
import pytest

from gpu_case import log
from test_gpu_paged import _evict

pytestmark = pytest.mark.gpu


def _same(s):
    s[:] = 0.25


def _near(s):
    s[:] = 1.0 + s / 64  # one magnitude: more share the first 8 bits than are kept in LDS


def _few(s):
    s[:] = np.round(s * 4) / 4


def _odd(s):
    s[:] = np.random.default_rng(3).choice([0.0, -0.0, np.inf, -np.inf, np.nan, -np.nan, 1e-45, -3.0, 2.0], s.shape)


WEIGHTS = {"distinct": None, "same": _same, "near": _near, "few": _few, "odd": _odd}


@pytest.mark.parametrize("n", [65536, 65537, 100003])
@pytest.mark.parametrize("weights", list(WEIGHTS))
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_around_the_registers_limit(gpu, n, weights, in_place):
    """A long head next to a shorter one."""
    log(f"evict {n} {weights} in place:{in_place}")
    _evict(gpu, [n, 9500], 9000, 100, 4, ct="i8", hk=1, dim=16, page=32, seed=n % 100 + len(weights),
           weights=WEIGHTS[weights], in_place=in_place)


@pytest.mark.parametrize("n,budget", [(65538, 65536), (70001, 69000), (100003, 60000), (70001, 3)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_a_few_and_nearly_all(gpu, n, budget, in_place):
    log(f"evict {n} -> {budget} in place:{in_place}")
    _evict(gpu, [n], budget, budget // 3, 1, ct="bf16", hk=1, dim=16, page=24, seed=budget % 97, in_place=in_place)
