"""The decoding example over its budget: every step's attention and gathered
weights against the fp64 oracle on the cache as the attention read it, before
and after evictions have moved its rows. Tolerances as in test_gpu_paged."""
import os
import sys

import numpy as np
import pytest

from gpu_case import log
from oracle import paged as O
from test_gpu_paged import HALF, U, _close

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_every_step_of_the_example(gpu, monkeypatch):
    import torch

    import paged_decode

    log("example: every step")
    batch, width, budget, page, dim, hq, hk = 3, 128, 40, 8, 32, 4, 2
    layer = paged_decode.Layer(batch, width, hq, hk, dim, budget, page_size=page, sinks=2, recent=8)
    held = {}
    attend, evict = gpu.dq_kv_attend, gpu.dq_kv_evict

    def attend_seen(*a, **k):
        held["scores"] = layer.scores.clone()
        attend(*a, **k)

    def evict_seen(*a, **k):
        held.update(k=layer.k.clone(), v=layer.v.clone(), ks=layer.ks.clone(), vs=layer.vs.clone(),
                    gathered=layer.scores.clone(), lens=layer.lens.clone())
        evict(*a, **k)

    monkeypatch.setattr(gpu, "dq_kv_attend", attend_seen)
    monkeypatch.setattr(gpu, "dq_kv_evict", evict_seen)
    try:
        g = torch.Generator(device="cuda").manual_seed(5)
        layer.prompt(torch.randn((batch, 30, width), generator=g, device="cuda").bfloat16())
        x = torch.randn((batch, width), generator=g, device="cuda").bfloat16()
        f = lambda t: t.float().cpu().numpy()  # noqa: E731
        for step in range(30):
            x = layer.step(x)
            q, y, _ = layer.seen
            lens = held["lens"].tolist()
            assert lens == [min(31 + step, budget + 1)] * batch
            want, _, ws, mass, reach = O.attend(f(q), lens, layer.table.cpu().numpy(), f(held["k"]), f(held["v"]),
                                                f(held["ks"]), f(held["vs"]), dim ** -0.5, page)
            dp = 2 * (reach * (4 * np.sqrt(dim) + 16) * U + (lens[0] / 128 + 64) * U)
            _close(f(y), want, HALF["bf16"] * np.abs(want) + (2 * dp + 2.0 ** -16)[..., None] * mass, f"out {step}")
            at = slice(0, lens[0])
            full = np.float64(np.float32(0.99)) * f(held["scores"])[:, :, at] + ws[:, :, at]
            worst = dp.reshape(batch, hk, hq // hk).max(-1)[..., None]
            _close(f(held["gathered"])[:, :, at], full, 2 * U * np.abs(full) + 2 * U + worst * ws[:, :, at], f"weights {step}")
        assert layer.lens.tolist() == [budget] * batch and gpu.dq_kv_take_errors(layer.kv) == 0
    finally:
        layer.release()
