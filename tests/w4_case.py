"""Random cases of products with 4-bit weights for the tests: inputs on the
host, the call, and the comparison with the fp64 oracle."""
from __future__ import annotations

import numpy as np

from oracle import experts as X

ROUND = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # half a step, relative to the value
SMALL = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -25}  # and below the normal values


def code(dq, name):
    return {"f32": dq.DQ_F32, "bf16": dq.DQ_BF16, "f16": dq.DQ_F16}[name]


def dtype(torch, name):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def make(torch, seed, experts, N, K, group, x_rows, type="bf16", scale="bf16", zeros=True, bias=True, gated=False):
    """Host tensors; x and the scales hold values of their types."""
    r = np.random.default_rng(seed)
    rows, G = N * (2 if gated else 1), -(-K // group)
    c = dict(experts=experts, N=N, K=K, group=group, type=type, scale=scale, gated=gated)
    c["codes"] = torch.from_numpy(r.integers(0, 256, (experts, rows, (K + 1) // 2), dtype=np.uint8))
    c["scales"] = torch.from_numpy(r.uniform(-0.4, 1.0, (experts, rows, G)) / np.sqrt(K) / 4).to(dtype(torch, scale))
    c["zeros"] = torch.from_numpy(r.integers(0, 256, (experts, rows, (G + 1) // 2), dtype=np.uint8)) if zeros else None
    c["bias"] = torch.from_numpy(r.normal(0, 0.5, (experts, rows)).astype(np.float32)) if bias else None
    c["x"] = torch.from_numpy(r.normal(0, 1, (x_rows, K)) * r.choice([1, 1, 1, 8], K)).to(dtype(torch, type))
    return c


def handle(dq, c, y, max_rows):
    h = dq.dq_w4_init(c["experts"], c["N"], c["K"], c["group"], code(dq, c["type"]), code(dq, c["scale"]),
                      code(dq, y), c["gated"], max_rows)
    dev = [None if c[n] is None else c[n].cuda() for n in ("codes", "scales", "zeros", "bias")]
    dq.dq_w4_set_w(h, *dev)
    return h


def want(c, e, x):
    """(the oracle's rows for expert e, how far fp32 sums may be from them)"""
    part = [None if c[n] is None else c[n][e].double().numpy() if c[n].is_floating_point() else c[n][e].numpy()
            for n in ("codes", "scales", "zeros", "bias")]
    W = X.weights(part[0], part[1], part[2], c["K"], c["group"])
    x = x.double().numpy()
    pieces = 3 if c["type"] == "f32" else 1
    return (X.product(x, W, part[3], c["gated"]),
            X.product_bound(x, part[0], part[1], part[2], c["K"], c["group"], pieces, part[3], c["gated"]))


def check(got, ref, bound, y, what):
    got = got.double().cpu().numpy()
    err = np.abs(got - ref)
    # y's own rounding counts on the value that was rounded, which the sums' error can have moved
    ok = err <= bound + ROUND[y] * (np.abs(ref) + bound) + SMALL[y]
    assert ok.all(), (f"{what}: {(~ok).sum()} of {ok.size} outside, first at {np.argwhere(~ok)[0].tolist()}, "
                      f"worst {np.nanmax(err / (bound + ROUND[y] * np.abs(ref) + 1e-30)):.3g} of the bound")
