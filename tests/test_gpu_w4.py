"""Products with 4-bit weights on the GPU against the fp64 oracle, at the
bound that the oracle derives for fp32 sums plus y's rounding."""
import numpy as np
import pytest

import w4_case as W
from gpu_case import log

pytestmark = pytest.mark.gpu


def _forward(gpu, torch, c, y="f32", x=None, max_rows=None):
    x = c["x"].cuda() if x is None else x
    h = W.handle(gpu, c, y, max_rows or max(1, x.shape[0]))
    try:
        out = torch.full((x.shape[0], c["N"]), 77.0, dtype=W.dtype(torch, y), device="cuda")
        gpu.dq_w4_forward(h, x, out)
        torch.cuda.synchronize()
        return out
    finally:
        gpu.dq_w4_release(h)


def _compare(gpu, torch, c, y="f32", what=""):
    log(f"w4 {what} rows {len(c['x'])} N {c['N']} K {c['K']} g {c['group']} {c['type']} {c['scale']} -> {y} "
        f"gated {c['gated']}")
    W.check(_forward(gpu, torch, c, y), *W.want(c, 0, c["x"]), y, what)


@pytest.mark.parametrize("type", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,N,K,group", [(1, 16, 128, 128), (1, 1, 1, 32), (3, 17, 31, 32), (16, 100, 300, 64),
                                            (17, 33, 129, 32), (33, 48, 1000, 256), (65, 20, 640, 128),
                                            (130, 130, 260, 64), (2, 257, 2050, 1024), (5, 40, 96, 128)])
def test_forward(gpu, type, rows, N, K, group):
    import torch

    for scale, y, zeros, bias, gated in (("f32", "f32", True, True, False), (type, type, False, False, False),
                                         ("bf16", type, True, False, True), ("f16", "f32", False, True, True)):
        c = W.make(torch, rows * 1000 + K, 1, N, K, group, rows, type, scale, zeros, bias, gated)
        _compare(gpu, torch, c, y)


@pytest.mark.parametrize("type", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows", [1, 40, 300, 700])
def test_larger(gpu, type, rows):
    """Several tiles of rows and columns, several blocks a wave."""
    import torch

    for group, gated, N, K in ((128, False, 520, 1536), (32, True, 264, 1160), (64, False, 300, 1283)):
        c = W.make(torch, rows + group, 1, N, K, group, rows, type, type, True, False, gated)
        _compare(gpu, torch, c, "f32")


@pytest.mark.parametrize("type", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows", [3, 200])
def test_strided_and_unaligned_x(gpu, type, rows):
    """Rows of a wider tensor, and from an element that is not 16-byte aligned."""
    import torch

    c = W.make(torch, 9, 1, 70, 384, 64, rows, type)
    for left, width in ((8, 400), (3, 391), (0, 385), (8, 392)):
        wide = torch.full((rows, width), float("nan"), dtype=c["x"].dtype, device="cuda")
        x = wide[:, left:left + 384]
        x.copy_(c["x"])
        log(f"w4 strided {type} {left} of {width}")
        W.check(_forward(gpu, torch, c, "f32", x), *W.want(c, 0, c["x"]), "f32", "strided")
    one = c["x"][:1].cuda().expand(rows, -1)
    ref, bound = W.want(c, 0, c["x"][:1])
    W.check(_forward(gpu, torch, c, "f32", one), ref.repeat(rows, 0), bound.repeat(rows, 0), "f32", "one row for all")


@pytest.mark.parametrize("type", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows", [5, 150])
def test_not_finite_stays_in_its_row(gpu, type, rows):
    import torch

    c = W.make(torch, 4, 1, 90, 500, 128, rows, type)
    ref, bound = W.want(c, 0, c["x"])
    x = c["x"].clone()
    x[1, 3], x[4, 499] = float("nan"), float("inf")
    got = _forward(gpu, torch, c, "f32", x.cuda())
    assert not torch.isfinite(got[1]).any() and not torch.isfinite(got[4]).any()
    keep = [i for i in range(rows) if i not in (1, 4)]
    W.check(got[keep], ref[keep], bound[keep], "f32", "other rows")


def test_fp16_subnormals_count(gpu):
    """fp16 values below the normal ones, and codes times them, are not lost."""
    import torch

    c = W.make(torch, 2, 1, 32, 128, 32, 4, "f16", "f32", True, False)
    c["x"] = (torch.arange(4 * 128).reshape(4, 128) % 37 * 2.0 ** -24).to(torch.float16)
    c["scales"] = c["scales"] * 2.0 ** 20
    _compare(gpu, torch, c, "f32", "subnormal")


def test_zero_rows_and_one_context_for_many_sizes(gpu):
    import torch

    c = W.make(torch, 6, 1, 48, 256, 64, 200, "bf16")
    ref, bound = W.want(c, 0, c["x"])
    h = W.handle(gpu, c, "f32", 200)
    x = c["x"].cuda()
    for rows in (0, 1, 200, 16, 17, 64, 65, 2):
        out = torch.full((201, 48), -5.0, device="cuda")
        gpu.dq_w4_forward(h, x[:rows], out[:rows])
        torch.cuda.synchronize()
        W.check(out[:rows], ref[:rows], bound[:rows], "f32", f"{rows} rows") if rows else None
        assert (out[rows:] == -5.0).all()
    gpu.dq_w4_release(h)


def _grouped(gpu, torch, c, counts, y="f32", row_index=None, lead=0, tail=0, h=None):
    """counts of each expert's rows, `lead` rows before them and `tail` behind."""
    rows = lead + sum(counts) + tail
    off = torch.tensor([lead + sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32)
    own = h is None
    h = W.handle(gpu, c, y, max(rows, 1)) if own else h
    out = torch.full((rows, c["N"]), 77.0, dtype=W.dtype(torch, y), device="cuda")
    idx = None if row_index is None else torch.tensor(row_index, dtype=torch.int32, device="cuda")
    gpu.dq_w4_forward_grouped(h, c["x"].cuda(), off.cuda(), out, row_index=idx)
    torch.cuda.synchronize()
    if own:
        gpu.dq_w4_release(h)
    return out


def _check_grouped(torch, c, counts, out, y="f32", row_index=None, lead=0):
    at = lead
    assert (out[:lead] == 77.0).all()
    for e, n in enumerate(counts):
        if n:
            src = range(at, at + n) if row_index is None else row_index[at:at + n]
            W.check(out[at:at + n], *W.want(c, e, c["x"][list(src)]), y, f"expert {e}")
        at += n
    assert (out[at:] == 77.0).all()


@pytest.mark.parametrize("type", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("counts", [[3], [0, 5, 0, 17, 1], [1] * 9, [40, 0, 70, 33], [0, 0, 130, 2, 0, 0, 1],
                                    [300, 20, 0, 500]])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped(gpu, type, counts, gather):
    import torch

    rows, N, K = sum(counts), 70, 200
    r = np.random.default_rng(rows)
    x_rows = 13 if gather else rows
    idx = r.integers(0, x_rows, rows).tolist() if gather else None
    for gated, y in ((False, "f32"), (True, type)):
        c = W.make(torch, rows + gated, len(counts), N, K, 64, x_rows, type, type, not gated, gated, gated)
        log(f"w4 grouped {counts} {type} -> {y} gather {gather} gated {gated}")
        _check_grouped(torch, c, counts, _grouped(gpu, torch, c, counts, y, idx), y, idx)


def test_grouped_rows_before_and_behind_are_left(gpu):
    import torch

    counts = [4, 0, 21]
    c = W.make(torch, 3, 3, 24, 160, 32, 25 + 7 + 40)
    out = _grouped(gpu, torch, c, counts, lead=7, tail=40)
    _check_grouped(torch, c, counts, out, lead=7)
    out = _grouped(gpu, torch, c, [0, 0, 0], tail=30)
    assert (out == 77.0).all()


def test_grouped_many_experts(gpu):
    """More than the 64 that are looked up at a time, rows of few of them."""
    import torch

    for experts in (65, 200, 1024):
        counts = [0] * experts
        for e in (0, 1, 63, 64, experts - 1):
            counts[e] += 2 + e % 3
        c = W.make(torch, experts, experts, 16, 40, 32, sum(counts), bias=False)
        log(f"w4 grouped {experts} experts")
        _check_grouped(torch, c, counts, _grouped(gpu, torch, c, counts))


def test_grouped_bad_rows_and_offsets(gpu):
    """A row that does not exist is NaN; offsets out of order or range stay
    inside y, and rows that they leave to one expert are that expert's."""
    import torch

    counts = [5, 20, 3]
    idx = np.random.default_rng(0).integers(0, 28, 28).tolist()
    idx[2], idx[9], idx[27] = -1, 28, 2 ** 31 - 1
    c = W.make(torch, 1, 3, 40, 128, 32, 28)
    out = _grouped(gpu, torch, c, counts, row_index=idx)
    for r in (2, 9, 27):
        assert torch.isnan(out[r]).all()
        out[r] = 0.0
    good = [r for r in range(28) if r not in (2, 9, 27)]
    for r in good:
        e = 0 if r < 5 else 1 if r < 25 else 2
        W.check(out[r:r + 1], *W.want(c, e, c["x"][idx[r]:idx[r] + 1]), "f32", f"row {r}")
    h = W.handle(gpu, c, "f32", 28)
    x = c["x"].cuda()
    for off, owner in (([-9, 4, 50, 60], {0: range(0, 4), 1: range(4, 28)}),
                       ([3, 3, -5, 10], {2: range(0, 10)}),
                       ([2 ** 31 - 1] * 4, {}), ([-2 ** 31] * 4, {}), ([0, 28, 28, 5], {0: range(28)})):
        out = torch.full((29, 40), 77.0, device="cuda")
        gpu.dq_w4_forward_grouped(h, x, torch.tensor(off, dtype=torch.int32, device="cuda"), out[:28])
        torch.cuda.synchronize()
        for e, rows in owner.items():
            W.check(out[list(rows)], *W.want(c, e, c["x"][list(rows)]), "f32", f"{off} expert {e}")
        rest = [r for r in range(29) if not any(r in v for v in owner.values())]
        assert (out[rest] == 77.0).all(), off
    gpu.dq_w4_release(h)


@pytest.mark.parametrize("rows", [1, 40, 260])
def test_replays_streams_and_repeats(gpu, rows):
    """Captured and replayed with eager calls between, on another stream, and
    twice: bit for bit the same."""
    import torch

    c = W.make(torch, rows, 1, 130, 1100, 64, rows, "bf16", "bf16", True, True, True)
    h = W.handle(gpu, c, "bf16", rows)
    x = c["x"].cuda()
    out = torch.empty((rows, 130), dtype=torch.bfloat16, device="cuda")
    gpu.dq_w4_forward(h, x, out)
    torch.cuda.synchronize()
    first = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        gpu.dq_w4_forward(h, x, out)
    side.synchronize()
    assert torch.equal(first, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gpu.dq_w4_forward(h, x, out)
    x2 = (x.float() * 0.5).to(x.dtype)
    keep = x.clone()
    for _ in range(3):
        x.copy_(x2)
        g.replay()
        torch.cuda.synchronize()
        half = out.clone()
        gpu.dq_w4_forward(h, x, out)
        torch.cuda.synchronize()
        assert torch.equal(half, out)
        x.copy_(keep)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, out)
    gpu.dq_w4_release(h)


def test_weights_can_be_set_again(gpu):
    import torch

    a = W.make(torch, 1, 1, 33, 140, 32, 6)
    b = W.make(torch, 2, 1, 33, 140, 32, 6, zeros=False, bias=False)
    h = W.handle(gpu, a, "f32", 6)
    for c in (b, a):
        gpu.dq_w4_set_w(h, *[None if c[n] is None else c[n].cuda() for n in ("codes", "scales", "zeros", "bias")])
        out = torch.empty((6, 33), device="cuda")
        gpu.dq_w4_forward(h, c["x"].cuda(), out)
        torch.cuda.synchronize()
        W.check(out, *W.want(c, 0, c["x"]), "f32", "set again")
    gpu.dq_w4_release(h)


@pytest.mark.parametrize("type,K,rows", [("f32", 16384, 700), ("bf16", 16390, 2100)])
def test_more_rows_than_are_prepared_at_once(gpu, type, K, rows):
    """Long rows that are prepared for the kernel in several parts, of one
    expert, of several, and by an index from fewer or more rows."""
    import torch

    counts = [rows // 2 - 3, 0, rows - rows // 2 - 10]
    c = W.make(torch, 1, 3, 20, K, 128, rows, type, "f32")
    log(f"w4 parts {type} {K} {rows}")
    out = _grouped(gpu, torch, c, counts, tail=13)
    _check_grouped(torch, c, counts, out)
    r = np.random.default_rng(5)
    for x_rows in (31, rows):
        idx = r.integers(0, x_rows, rows).tolist()
        d = dict(c, x=c["x"][:x_rows])
        out = _grouped(gpu, torch, d, counts, row_index=idx, tail=13)
        _check_grouped(torch, d, counts, out, row_index=idx)
    one = {n: v if n in ("x", "type", "scale", "N", "K", "group", "gated") else 1 if n == "experts" else v[:1]
           for n, v in c.items()}
    W.check(_forward(gpu, torch, one), *W.want(one, 0, c["x"]), "f32", "one expert")


@pytest.mark.parametrize("type", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows", [3, 16, 30, 44, 60, 200])
def test_what_the_chip_held_before_does_not_show(gpu, type, rows):
    """A K that ends inside a block and rows that end inside a tile, behind a
    call whose x was all NaN: what it left in the compute units' memory is not
    multiplied."""
    import torch

    c = W.make(torch, rows, 1, 4096, 168, 128, rows, type, bias=False)
    bad = W.make(torch, rows, 1, 4096, 2048, 128, 256, type, bias=False)
    hb, h = W.handle(gpu, bad, "f32", 256), W.handle(gpu, c, "f32", 256)
    x, nan = c["x"].cuda(), torch.full((256, 2048), float("nan"), dtype=c["x"].dtype, device="cuda")
    out, junk = torch.empty((rows, 4096), device="cuda"), torch.empty((256, 4096), device="cuda")
    ref, bound = W.want(c, 0, c["x"])
    for n in (256, 64, 48, 16, 2):
        gpu.dq_w4_forward(hb, nan[:n], junk[:n])
        gpu.dq_w4_forward(h, x, out)
        torch.cuda.synchronize()
        W.check(out, ref, bound, "f32", f"behind {n} rows of NaN")
    gpu.dq_w4_release(hb)
    gpu.dq_w4_release(h)


def test_refusals_with_a_context(gpu):
    """What a call refuses leaves y as it was."""
    import ctypes as C

    import torch

    lib = gpu.load()
    c = W.make(torch, 1, 2, 24, 64, 32, 10)
    h = gpu.dq_w4_init(2, 24, 64, 32, gpu.DQ_BF16, gpu.DQ_BF16, gpu.DQ_F32, False, 10)
    x, y = c["x"].cuda(), torch.full((10, 24), 5.0, device="cuda")
    off = torch.tensor([0, 4, 10], dtype=torch.int32, device="cuda")

    def refused(status, call):
        with pytest.raises(gpu.DQError) as e:
            call()
        assert e.value.status == status, e.value
        torch.cuda.synchronize()
        assert (y == 5.0).all()

    refused(gpu.DQ_ERR_STATE, lambda: gpu.dq_w4_forward_grouped(h, x, off, y))  # no weights yet
    gpu.dq_w4_set_w(h, *[None if c[n] is None else c[n].cuda() for n in ("codes", "scales", "zeros", "bias")])
    refused(gpu.DQ_ERR_ARG, lambda: gpu.dq_w4_forward(h, x, y))  # several experts
    refused(gpu.DQ_ERR_ARG, lambda: gpu.dq_w4_forward_grouped(h, x, off[:2].contiguous(), y))
    refused(gpu.DQ_ERR_TYPE, lambda: gpu.dq_w4_forward_grouped(h, x.float(), off, y))
    refused(gpu.DQ_ERR_TYPE, lambda: gpu.dq_w4_forward_grouped(h, x, off.long(), y))
    refused(gpu.DQ_ERR_TYPE, lambda: gpu.dq_w4_forward_grouped(h, x, off, y.bfloat16()))
    refused(gpu.DQ_ERR_ARG, lambda: gpu.dq_w4_forward_grouped(h, x[:, :63], off, y))
    refused(gpu.DQ_ERR_ARG, lambda: gpu.dq_w4_forward_grouped(h, x.t().contiguous().t(), off, y))
    refused(gpu.DQ_ERR_ARG, lambda: gpu.dq_w4_forward_grouped(h, x, off, y.t().contiguous().t()))
    refused(gpu.DQ_ERR_ARG, lambda: gpu.dq_w4_forward_grouped(h, x[:9], off, y))  # rows of x that are not there
    refused(gpu.DQ_ERR_ARG, lambda: gpu.dq_w4_forward_grouped(h, x, off, y, row_index=off))  # too short
    refused(gpu.DQ_ERR_ARG, lambda: gpu.dq_w4_forward_grouped(h, x, off, torch.empty((11, 24), device="cuda")))
    p, q = x.data_ptr(), y.data_ptr()
    st = torch.cuda.current_stream().cuda_stream
    assert lib.dq_w4_forward_grouped(h, 10, off.data_ptr(), 10, p + 1, 64, None, q, st) == gpu.DQ_ERR_ARG
    assert lib.dq_w4_forward_grouped(h, 10, off.data_ptr() + 2, 10, p, 64, None, q, st) == gpu.DQ_ERR_ARG
    assert lib.dq_w4_forward_grouped(h, 10, off.data_ptr(), 10, p, 64, None, q + 2, st) == gpu.DQ_ERR_ARG
    assert lib.dq_w4_forward_grouped(h, 10, off.data_ptr(), 10, p, -64, None, q, st) == gpu.DQ_ERR_ARG
    assert lib.dq_w4_forward_grouped(h, 10, None, 10, p, 64, None, q, st) == gpu.DQ_ERR_ARG
    assert lib.dq_w4_forward_grouped(h, 10, off.data_ptr(), 0, p, 64, None, q, st) == gpu.DQ_ERR_ARG
    assert lib.dq_w4_forward_grouped(h, -1, off.data_ptr(), 10, p, 64, None, q, st) == gpu.DQ_ERR_ARG
    assert lib.dq_w4_set_w(h, None, p, None, None, st) == gpu.DQ_ERR_ARG
    torch.cuda.synchronize()
    assert (y == 5.0).all()
    m = gpu.dq_moe_init(4, 8, 2, gpu.DQ_F32)
    l, i, w = torch.zeros((5, 8), device="cuda"), torch.zeros((5, 2), dtype=torch.int32, device="cuda"), torch.zeros((5, 2), device="cuda")
    o = torch.zeros(9, dtype=torch.int32, device="cuda")
    refused(gpu.DQ_ERR_ARG, lambda: gpu.dq_moe_route(m, l, i, w, o, i, i))  # five tokens
    refused(gpu.DQ_ERR_ARG, lambda: gpu.dq_moe_route(m, l[:4], i, w, o[:8].contiguous(), i, i))
    refused(gpu.DQ_ERR_TYPE, lambda: gpu.dq_moe_route(m, l[:4].half(), i, w, o, i, i))
    refused(gpu.DQ_ERR_ARG, lambda: gpu.dq_moe_combine(m, y, w, i, torch.empty((5, 24), device="cuda")))
    refused(gpu.DQ_ERR_ARG, lambda: gpu.dq_moe_combine(m, y, w, i, torch.empty((4, 20), device="cuda")))
    refused(gpu.DQ_ERR_TYPE, lambda: gpu.dq_moe_combine(m, y, w, i, y[:4], add=y[:4].half()))
    gpu.dq_moe_release(m)
    gpu.dq_w4_release(h)


def test_two_contexts_on_two_streams(gpu):
    """Calls that overlap, each on a context of its own, as alone."""
    import torch

    cases = [W.make(torch, i, 1, 200, 900, 64, 120, "bf16") for i in range(2)]
    hs = [W.handle(gpu, c, "f32", 120) for c in cases]
    xs = [c["x"].cuda() for c in cases]
    outs = [torch.empty((120, 200), device="cuda") for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for h, x, o, s in zip(hs, xs, outs, streams):
            gpu.dq_w4_forward(h, x, o, stream=s)
    torch.cuda.synchronize()
    for c, o, h in zip(cases, outs, hs):
        W.check(o, *W.want(c, 0, c["x"]), "f32", "overlapping")
        gpu.dq_w4_release(h)
