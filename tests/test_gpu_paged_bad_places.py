"""GPU tests of what the paged cache's calls give for pages and lengths that do
not exist, beyond the outputs: gathered weights and evictions."""
import pytest

from gpu_case import log
from test_gpu_paged import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("length", [300, 2000])  # whole heads, and shared ones
@pytest.mark.parametrize("window", [0, 100])
def test_weights_of_a_sequence_with_a_bad_page(gpu, length, window):
    """NaN for the tokens that are attended to, decayed before the window,
    other sequences and other slots as ever."""
    import torch

    log(f"bad page, weights {length} window {window}")
    c = Case(gpu, 3, 2, 2, 32, 8, [40, length, 9], "bf16", "i8", seed=1, window=window, scores=True)
    try:
        c.dev["table"][1, (length - 20) // 8] = 10 ** 6
        out, lse, so = c.attend()
        assert gpu.dq_kv_take_errors(c.ctx) > 0
        first = length - window if window else 0
        assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all() and torch.isnan(so[1, :, first:length]).all()
        assert torch.equal(so[1, :, :first].cpu(), c.scores[1, :, :first] * 0.9)
        assert bool((so[1, :, length:] == 7).all())
        c.check((out, lse, so), rows=[0, 2])
    finally:
        c.close()


def test_weights_of_a_length_out_of_range(gpu):
    import torch

    log("bad length, weights")
    for length in (-1, 10 ** 6):
        c = Case(gpu, 3, 2, 2, 32, 8, [40, 300, 9], "f16", "f16", seed=2, scores=True)
        try:
            c.dev["lens"][1] = length
            out, lse, so = c.attend()
            assert gpu.dq_kv_take_errors(c.ctx) > 0
            assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all() and bool((so[1] == 7).all())
            c.check((out, lse, so), rows=[0, 2])
        finally:
            c.close()


@pytest.mark.parametrize("in_place", [False, True])
def test_eviction_of_a_length_out_of_range(gpu, in_place):
    """Above the slots there are it counts as all of them, below zero as none;
    a head within its budget keeps what it has."""
    import torch

    log(f"evict bad length in place:{in_place}")
    c = Case(gpu, 3, 1, 1, 32, 8, [40, 40, 20], "bf16", "bf16", seed=1, per_seq=5)
    try:
        cap = c.cap
        s = torch.arange(cap, dtype=torch.float32, device="cuda").expand(3, 1, cap).contiguous()
        o = torch.arange(cap, dtype=torch.int32, device="cuda").expand(3, 1, cap).contiguous()
        n = torch.tensor([2 ** 31 - 1, -5, 20], dtype=torch.int32, device="cuda")
        newest = torch.full_like(n, 100)
        v = c.dev["v"].view(torch.int16).clone()
        so, oo, no = (s, o, n) if in_place else (torch.full_like(s, -7.0), torch.full_like(o, -7), torch.full_like(n, -7))
        gpu.dq_kv_evict(c.ctx, 30, n, newest, s, o, *c.cache(), so, oo, no)
        torch.cuda.synchronize()
        assert gpu.dq_kv_take_errors(c.ctx) > 0 and no.tolist() == [30, 0, 20]
        # the 30 largest of 40: slots 10 .. 39; those from 30 on move into 0 .. 9
        assert oo[0, 0, :30].tolist() == list(range(30, 40)) + list(range(10, 30))
        assert so[0, 0, :30].tolist() == oo[0, 0, :30].float().tolist()
        assert oo[2, 0, :20].tolist() == list(range(20))
        rest = [int(x) for x in oo[1, 0]]
        assert rest == (list(range(cap)) if in_place else [-7] * cap)
        got, table = c.dev["v"].view(torch.int16), c.table
        for to, src in zip(range(10), range(30, 40)):
            assert torch.equal(got[int(table[0, to // 8]), 0, to % 8], v[int(table[0, src // 8]), 0, src % 8])
    finally:
        c.close()
