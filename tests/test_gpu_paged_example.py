"""The decoding example end to end: the quantized projections, the append, the
attention and the eviction as one program, each step's attention checked
against the fp64 oracle on the cache that it read."""
import os
import sys

import numpy as np
import pytest

from gpu_case import log
from oracle import paged as O

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_decoding_over_the_budget(gpu):
    import torch

    import paged_decode

    log("example: decoding over the budget")
    batch, width, budget, page = 3, 128, 40, 8
    layer = paged_decode.Layer(batch, width, 4, 2, 32, budget, page_size=page, sinks=2, recent=8)
    try:
        g = torch.Generator(device="cuda").manual_seed(3)
        layer.prompt(torch.randn((batch, 30, width), generator=g, device="cuda").bfloat16())
        x = torch.randn((batch, width), generator=g, device="cuda").bfloat16()
        for step in range(25):
            before = int(layer.lens[0])
            x = layer.step(x)
            q, y, lens = layer.seen
            assert lens.tolist() == [before + 1] * batch
            assert torch.isfinite(x.float()).all()
            if before + 1 <= budget:
                f = lambda t: t.float().cpu().numpy()  # noqa: E731
                want, _, _, mass, _ = O.attend(f(q), lens.tolist(), layer.table.cpu().numpy(), f(layer.k), f(layer.v),
                                               f(layer.ks), f(layer.vs), 32 ** -0.5, page)
                # half a step of bf16 and the weights' rounding
                assert (np.abs(f(y) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -12 * mass).all()
                total = layer.scores[:, :, :before + 1].sum(-1).cpu().numpy()
                steps = step + 1
                assert np.allclose(total, 2 * (1 - 0.99 ** steps) / 0.01, rtol=1e-4)  # two query heads a step
            assert layer.lens.tolist() == [min(before + 1, budget)] * batch
        # the first two and the last eight tokens of 55 are still there, and every number once
        order = layer.order[:, :, :budget].cpu().numpy()
        for b in range(batch):
            for h in range(2):
                held = set(order[b, h].tolist())
                assert len(held) == budget and {0, 1} <= held and set(range(47, 55)) <= held and max(held) == 54
        assert gpu.dq_kv_take_errors(layer.kv) == 0
    finally:
        layer.release()
