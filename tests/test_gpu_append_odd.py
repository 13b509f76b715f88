"""GPU test of the append and the rotation of neighbouring pairs out of tensors
that are aligned to their elements alone: odd offsets and strides, which leave
one pair a lane. Tolerances as in test_gpu_paged."""
import numpy as np
import pytest

from gpu_case import log
from oracle import paged as O
from test_gpu_paged import Case, HALF, U, _close, _np, _types

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("qt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("ct", ["bf16", "f16", "i8"])
@pytest.mark.parametrize("dim,rot", [(16, 6), (80, 36), (128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_from_odd_places(gpu, qt, ct, dim, rot, interleaved):
    import torch

    log(f"append odd {qt}->{ct} {dim}/{rot} {interleaved}")
    r = np.random.default_rng(dim + rot)
    batch, hk, group, page = 5, 2, 2, 8
    hq, heads = hk * group, hk * group + 2 * hk
    axis, freq = [i % 2 for i in range(rot // 2)], [0.9 ** i for i in range(rot // 2)]
    c = Case(gpu, batch, hk, group, dim, page, [9] * batch, qt, ct, seed=dim)
    rope = gpu.dq_rope_init(dim, rot, axis, freq, interleaved)
    try:
        x = torch.from_numpy(r.normal(0, 1, (batch, heads, dim)).astype(np.float32)).to(_types(torch)[qt])
        wide = torch.full((batch, heads + 1, dim + 3), float("nan"), dtype=x.dtype, device="cuda")
        part = wide[:, :heads, 1:dim + 1]
        part.copy_(x)
        pos = r.integers(0, 40000, (2, batch)).astype(np.int32)
        index = torch.tensor([0, 8, 3, 7, 5], dtype=torch.int32, device="cuda")
        # one element past an aligned place, as the outputs of a smaller allocation are
        q_out = torch.full((batch * hq * dim + 1,), float("nan"), dtype=x.dtype, device="cuda")[1:].view(batch, hq, dim)
        gpu.dq_kv_append(c.ctx, part[:, hq:hq + hk], part[:, hq + hk:], index, *c.cache(), q=part[:, :hq], q_out=q_out,
                         rope=rope, positions=torch.from_numpy(pos).cuda())
        k, v = (torch.empty((batch, hk, dim), dtype=x.dtype, device="cuda") for _ in range(2))
        gpu.dq_kv_read(c.ctx, index, *c.cache(), k_out=k, v_out=v)
        torch.cuda.synchronize()
        assert gpu.dq_kv_take_errors(c.ctx) == 0
        x = _np(x)
        big = np.abs(x).max(-1, keepdims=True)
        turned = O.rotate(x, pos, axis, freq, interleaved)
        _close(_np(q_out), turned[:, :hq], HALF[qt] * np.abs(turned[:, :hq]) + 6 * U * big[:, :hq], "q")
        for name, got, want, b in (("k", k, turned[:, hq:hq + hk], big[:, hq:hq + hk]),
                                   ("v", v, x[:, hq + hk:], big[:, hq + hk:])):
            if ct == "i8":
                tol = 0.5 * np.abs(want).max(-1, keepdims=True) / 127 * (1 + 2.0 ** -20) + 18 * U * b
            else:
                tol = HALF[ct] * np.abs(want) + 6 * U * b + 2.0 ** -25 * (ct == "f16")
            _close(_np(got), want, tol + HALF[qt] * (np.abs(want) + tol), name)
        assert torch.isnan(wide[:, heads:]).all() and torch.isnan(wide[:, :, 0]).all()
    finally:
        gpu.dq_rope_release(rope)
        c.close()
