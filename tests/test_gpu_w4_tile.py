"""Products with 4-bit weights of many rows on the GPU, at sizes that fill the
chip with tiles (and so take the kernel for them), against the fp64 oracle at the
bound that it derives for fp32 sums plus y's rounding. The oracle computes some
columns of each tile of 16, and all of the last ones."""
import numpy as np
import pytest

import w4_case as W
from gpu_case import log

pytestmark = pytest.mark.gpu


def _columns(N, seed):
    r = np.random.default_rng(seed)
    pick = {int(t * 16 + r.integers(0, 16)) for t in range(N // 16)} | set(range(max(0, N - 17), N)) | {0, 15, 16}
    return sorted(c for c in pick if c < N)


def _some(torch, c, cols):
    """The same case with some of its columns."""
    rows = torch.tensor(cols + [c["N"] + n for n in cols] if c["gated"] else cols)
    return {**c, "N": len(cols), **{n: c[n][:, rows] for n in ("codes", "scales", "zeros", "bias") if c[n] is not None}}


def _run(gpu, torch, c, y, x=None, offsets=None, row_index=None, rows=None, h=None):
    x = c["x"].cuda() if x is None else x
    rows = rows or (len(row_index) if row_index is not None else len(x))
    own = h is None
    h = W.handle(gpu, c, y, rows) if own else h
    out = torch.full((rows, c["N"]), 77.0, dtype=W.dtype(torch, y), device="cuda")
    if offsets is None:
        gpu.dq_w4_forward(h, x, out)
    else:
        idx = None if row_index is None else torch.tensor(row_index, dtype=torch.int32, device="cuda")
        gpu.dq_w4_forward_grouped(h, x, torch.tensor(offsets, dtype=torch.int32, device="cuda"), out, row_index=idx)
    torch.cuda.synchronize()
    if own:
        gpu.dq_w4_release(h)
    return out


def _check(torch, c, out, y, offsets=None, row_index=None, seed=0, skip=()):
    cols = _columns(c["N"], seed)
    some = _some(torch, c, cols)
    offsets = [0, len(out)] if offsets is None else offsets
    for e in range(len(offsets) - 1):
        rows = [r for r in range(offsets[e], offsets[e + 1]) if r not in skip]
        if rows:
            src = rows if row_index is None else [row_index[r] for r in rows]
            ref, bound = W.want(some, e, c["x"][src])
            W.check(out[rows][:, cols], ref, bound, y, f"expert {e}")
    assert (out[:offsets[0]] == 77.0).all() and (out[offsets[-1]:] == 77.0).all()


KINDS = [("bf16", "bf16", "bf16", 128, True, True, False), ("bf16", "f32", "f32", 32, True, False, True),
         ("f16", "f16", "f16", 64, False, True, True), ("f16", "bf16", "f32", 256, True, True, False),
         ("f32", "f32", "f32", 64, True, False, False), ("f32", "f16", "f32", 128, False, False, True),
         ("bf16", "f16", "f32", 64, True, True, False), ("f16", "f32", "f16", 32, False, False, False),
         ("f32", "bf16", "bf16", 32, True, True, False)]


@pytest.mark.parametrize("type,scale,y,group,zeros,bias,gated", KINDS)
@pytest.mark.parametrize("rows,N,K", [(1100, 3100, 256), (1025, 2818, 392), (2049, 1600, 130), (4225, 2100, 256),
                                      (2177, 4130, 200)])
def test_forward(gpu, type, scale, y, group, zeros, bias, gated, rows, N, K):
    """Whole blocks of K, a K that ends inside one, rows that are copied first;
    the last two with a workgroup of 256 columns for every compute unit."""
    import torch

    N = N // 2 if gated else N
    c = W.make(torch, rows + K, 1, N, K, group, rows, type, scale, zeros, bias, gated)
    log(f"w4 tiles {rows} x {N} x {K} g {group} {type} {scale} -> {y} gated {gated}")
    _check(torch, c, _run(gpu, torch, c, y), y)


@pytest.mark.parametrize("type", ["bf16", "f16", "f32"])
def test_strides_and_one_row_for_all(gpu, type):
    import torch

    c = W.make(torch, 9, 1, 3000, 256, 64, 1100, type)
    h = W.handle(gpu, c, "f32", 1100)
    for left, width in ((8, 272), (3, 261), (0, 257)):
        wide = torch.full((1100, width), float("nan"), dtype=c["x"].dtype, device="cuda")
        x = wide[:, left:left + 256]
        x.copy_(c["x"])
        log(f"w4 tiles strided {type} {left} of {width}")
        _check(torch, c, _run(gpu, torch, c, "f32", x, h=h), "f32")
    one = dict(c, x=c["x"][:1].expand(1100, -1))
    _check(torch, one, _run(gpu, torch, one, "f32", c["x"][:1].cuda().expand(1100, -1), h=h), "f32")
    gpu.dq_w4_release(h)


@pytest.mark.parametrize("type", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped(gpu, type, gather):
    """Experts with no rows, one row, and rows on both sides of a tile's 128;
    rows before and behind theirs are left."""
    import torch

    for counts, lead, tail, sizes in (([0, 300, 1, 128, 129, 0, 255, 90], 5, 40, (3400, 1700)),
                                      ([700, 1, 0, 513, 900], 3, 30, (4400, 2200))):
        _grouped_case(gpu, torch, type, gather, counts, lead, tail, sizes)


def _grouped_case(gpu, torch, type, gather, counts, lead, tail, sizes):
    rows = lead + sum(counts) + tail
    offsets = [lead + sum(counts[:i]) for i in range(len(counts) + 1)]
    r = np.random.default_rng(3)
    for gated, N, K, x_rows in ((False, sizes[0], 256, 77), (True, sizes[1], 200, 2 * rows)):
        idx = r.integers(0, x_rows, rows).tolist() if gather else None
        c = W.make(torch, K, len(counts), N, K, 64, x_rows if gather else rows, type, "bf16", not gated, gated, gated)
        log(f"w4 tiles grouped {type} gather {gather} gated {gated}")
        _check(torch, c, _run(gpu, torch, c, "f32", None, offsets, idx, rows), "f32", offsets, idx)


@pytest.mark.parametrize("type", ["bf16", "f32"])
def test_bad_rows_and_offsets(gpu, type):
    import torch

    rows, N = 1200, 3000
    idx = np.random.default_rng(0).integers(0, 50, rows).tolist()
    bad = {2: -1, 130: 50, 777: 2 ** 31 - 1, 1199: -2 ** 31}
    for at, v in bad.items():
        idx[at] = v
    c = W.make(torch, 1, 2, N, 128, 32, 50, type)
    out = _run(gpu, torch, c, "f32", None, [0, 700, rows], idx)
    for at in bad:
        assert torch.isnan(out[at]).all()
    _check(torch, c, out, "f32", [0, 700, rows], idx, skip=bad)
    c = W.make(torch, 1, 2, N, 128, 32, rows, type)
    h = W.handle(gpu, c, "f32", rows)
    for off, owner in (([-5, 600, 2 ** 31 - 1], {0: range(600), 1: range(600, rows)}), ([900, 100, 1000], {1: range(100, 1000)}),
                       ([2 ** 31 - 1] * 3, {}), ([0, rows, -1], {0: range(rows)})):
        out = torch.full((rows + 1, N), 77.0, device="cuda")
        gpu.dq_w4_forward_grouped(h, c["x"].cuda(), torch.tensor(off, dtype=torch.int32, device="cuda"), out[:rows])
        torch.cuda.synchronize()
        cols = _columns(N, 1)
        for e, rr in owner.items():
            rr = list(rr)
            W.check(out[rr][:, cols], *W.want(_some(torch, c, cols), e, c["x"][rr]), "f32", f"{off} expert {e}")
        rest = [r for r in range(rows + 1) if not any(r in v for v in owner.values())]
        assert (out[rest] == 77.0).all(), off
    gpu.dq_w4_release(h)


@pytest.mark.parametrize("type", ["bf16", "f16", "f32"])
def test_not_finite_stays_in_its_row(gpu, type):
    import torch

    c = W.make(torch, 4, 1, 3000, 300, 128, 1100, type)
    x = c["x"].clone()
    x[1, 3], x[200, 299], x[1099, 0] = float("nan"), float("inf"), -float("inf")
    got = _run(gpu, torch, c, "f32", x.cuda())
    for r in (1, 200, 1099):
        assert not torch.isfinite(got[r]).any()
    cols = _columns(3000, 2)
    keep = [r for r in range(1100) if r not in (1, 200, 1099)]
    W.check(got[keep][:, cols], *W.want(_some(torch, c, cols), 0, c["x"][keep]), "f32", "other rows")


@pytest.mark.parametrize("type", ["bf16", "f32"])
def test_what_the_chip_held_before_does_not_show(gpu, type):
    """Rows that end inside a tile behind a call whose x was all NaN."""
    import torch

    c = W.make(torch, 5, 1, 3000, 256, 128, 1030, type, bias=False)
    h = W.handle(gpu, c, "f32", 1100)
    nan = torch.full((1100, 256), float("nan"), dtype=c["x"].dtype, device="cuda")
    for _ in range(3):
        junk = torch.empty((1100, 3000), device="cuda")
        gpu.dq_w4_forward(h, nan, junk)
        _check(torch, c, _run(gpu, torch, c, "f32", h=h), "f32")
    gpu.dq_w4_release(h)


@pytest.mark.parametrize("type,K,rows", [("f32", 16384, 700), ("bf16", 16390, 2100)])
def test_more_rows_than_are_prepared_at_once(gpu, type, K, rows):
    """Long rows that are prepared in several parts, of one expert, of several,
    and by an index from fewer or more rows."""
    import torch

    counts = [rows // 2 - 3, 0, rows - rows // 2 - 10]
    offsets = [0, counts[0], counts[0], counts[0] + counts[2]]
    N = 4300 if rows < 1000 else 1600
    c = W.make(torch, 1, 3, N, K, 128, rows, type, "f32", bias=False)
    log(f"w4 tiles in parts {type} {K} {rows}")
    _check(torch, c, _run(gpu, torch, c, "f32", None, offsets), "f32", offsets)
    r = np.random.default_rng(5)
    for x_rows in (31, rows):
        idx = r.integers(0, x_rows, rows).tolist()
        d = dict(c, x=c["x"][:x_rows])
        _check(torch, d, _run(gpu, torch, d, "f32", None, offsets, idx), "f32", offsets, idx)


@pytest.mark.parametrize("type,K", [("bf16", 384), ("f32", 200)])
def test_replays_streams_and_repeats(gpu, type, K):
    """Captured and replayed with eager calls between, on another stream, and
    twice: bit for bit the same."""
    import torch

    c = W.make(torch, 1, 1, 1600, K, 64, 1100, type, "bf16", True, True, True)
    h = W.handle(gpu, c, "bf16", 1100)
    x = c["x"].cuda()
    out = torch.empty((1100, 1600), dtype=torch.bfloat16, device="cuda")
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
    keep, half_x = x.clone(), (x.float() * 0.5).to(x.dtype)
    for _ in range(3):
        x.copy_(half_x)
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
