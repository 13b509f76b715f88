"""GPU test of rotary positions far from 0 over the whole range of frequencies
that the calls accept, against rational arithmetic."""
import numpy as np
import pytest

from exact_angle import cos_sin
from gpu_case import log
from test_gpu_paged import U, _close, _np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("freq", [1.0, 0.7, 1e-9, 10000.0 ** -0.37, 1e3, 1e6, 123456789.123, 1e9, -1e9])
def test_far_positions_at_every_frequency(gpu, freq):
    """(1, 0) turns into (cos, sin), rounded to fp32 once: half a step, and what
    the reduced angle is off by, 3e-13 (1e-15 for frequencies up to 1)."""
    import torch

    log(f"rope far {freq}")
    pos = np.array([2 ** 31 - 1, -2 ** 31, 2 ** 31 - 2, 2 ** 30 + 1, 1999999999, -1234567890, 16777217, 1, 0], np.int32)
    x = torch.zeros((len(pos), 1, 2), device="cuda")
    x[..., 0] = 1.0
    y, back = torch.empty_like(x), torch.empty_like(x)
    p = torch.from_numpy(pos).cuda()
    ctx = gpu.dq_rope_init(2, 2, [0], [freq])
    try:
        gpu.dq_rope_forward(ctx, x, p, y)
        gpu.dq_rope_forward(ctx, x, p, back, inverse=True)
        torch.cuda.synchronize()
        want = np.array([[cos_sin(t, freq)] for t in pos])
        tol = U * np.abs(want) + (1e-15 if abs(freq) <= 1 else 3e-13)
        _close(_np(y), want, tol, "forward")
        _close(_np(back), want * [1, -1], tol, "inverse")
    finally:
        gpu.dq_rope_release(ctx)


def test_append_turns_as_the_rotation_does(gpu):
    """The append's rotation of keys and queries at such angles is the same."""
    import torch

    log("append far")
    freq = [1e9, 0.7, 1e6, 1.0, 123456789.123, 1e-9, 1e3, -1e9]
    ctx = gpu.dq_kv_init(3, 2, 1, 16, 3, 8, 1, gpu.DQ_F32, gpu.DQ_BF16)
    rope = gpu.dq_rope_init(16, 16, [0] * 8, freq)
    try:
        g = torch.Generator().manual_seed(1)
        q, kv = torch.randn((3, 2, 16), generator=g).cuda(), torch.randn((3, 1, 16), generator=g).cuda()
        pos = torch.tensor([[2 ** 31 - 1, -2 ** 31, 1999999999]], dtype=torch.int32, device="cuda")
        table = torch.arange(3, dtype=torch.int32, device="cuda").view(3, 1)
        k, v = (torch.zeros((3, 1, 8, 16), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        q_out, want_q, want_k = torch.empty_like(q), torch.empty_like(q), torch.empty_like(kv)
        gpu.dq_kv_append(ctx, kv, kv, torch.zeros(3, dtype=torch.int32, device="cuda"), table, k, v, q=q, q_out=q_out,
                         rope=rope, positions=pos)
        gpu.dq_rope_forward(rope, q, pos, want_q)
        gpu.dq_rope_forward(rope, kv, pos, want_k)
        assert torch.equal(q_out, want_q) and torch.equal(k[:, :, 0], want_k.bfloat16())
        assert gpu.dq_kv_take_errors(ctx) == 0
    finally:
        gpu.dq_rope_release(rope)
        gpu.dq_kv_release(ctx)
