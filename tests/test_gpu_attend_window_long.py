"""GPU tests of the attention with a short window on a long cache, weights
gathered: the decay of what lies before the window is most of the work.
Tolerances as in test_gpu_paged."""
import pytest

from gpu_case import log
from test_gpu_paged import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,hk", [(3, 1), (16, 8)])  # few heads, and many
@pytest.mark.parametrize("window", [100, 512, 1000])
@pytest.mark.parametrize("before", [4096, 4097, 9000])   # slots before the window
@pytest.mark.parametrize("qt,ct", [("bf16", "i8"), ("f32", "bf16")])
def test_short_windows_on_long_caches(gpu, batch, hk, window, before, qt, ct):
    log(f"attend window {window} before {before} {batch}x{hk} {qt} {ct}")
    cap = window + before
    lens = [cap, 0, window, window + 1, cap - 1, 1, 4099, 40]
    page = 16 if cap % 16 == 0 else 1
    c = Case(gpu, batch, hk, 1, 16, page, [lens[i % len(lens)] for i in range(batch)], qt, ct, seed=window + before,
             window=window, scores=True, per_seq=cap // page, spare=3)
    try:
        c.check(c.attend())
        assert gpu.dq_kv_take_errors(c.ctx) == 0
    finally:
        c.close()
