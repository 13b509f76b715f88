"""GPU tests of the attention over a paged cache where keys or queries are
infinite: a token whose score is -infinity weighs nothing whatever the types,
one whose score is +infinity or NaN shows. Tolerances as in test_gpu_paged."""
import numpy as np
import pytest

from gpu_case import log
from oracle import paged as O
from test_gpu_paged import Case, HALF, U, _close, _np

pytestmark = pytest.mark.gpu

PAIRS = [("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16"), ("f32", "f16"), ("f16", "bf16"), ("bf16", "f16")]


def _expect(c, keep, b, h):
    """The head's output and lse over the tokens `keep` of sequence b, and their bounds."""
    k = O.sequence(_np(c.k), None, c.table, b, c.lens[b], c.page)[h // c.group][keep]
    v = O.sequence(_np(c.v), None, c.table, b, c.lens[b], c.page)[h // c.group][keep]
    q = _np(c.q)[b, h]
    s = c.sm * (k @ q)
    lse = s.max() + np.log(np.exp(s - s.max()).sum())
    p = np.exp(s - lse)
    ds = c.sm * (np.abs(k) @ np.abs(q)).max() * (4 * np.sqrt(c.dim) + 16) * U
    sums = (c.lens[b] / 128 + 64) * U
    # the weights' own pieces: 2^-20 where the output is fp32
    tol = HALF[c.qt] * np.abs(p @ v) + (4 * (ds + sums) + (2.0 ** -20 if c.qt == "f32" else 2.0 ** -16)) * (p @ np.abs(v))
    return p @ v, tol, lse, ds + sums + 2.0 ** -20 + 2 * U * abs(lse), p, 2 * (ds + sums)


@pytest.mark.parametrize("qt,ct", PAIRS)
@pytest.mark.parametrize("dim", [32, 80, 128])
@pytest.mark.parametrize("one", [False, True])
def test_keys_of_infinity(gpu, qt, ct, dim, one):
    """Every product of the token is -infinity (queries of both signs, keys of
    the opposite infinity), in the whole row or in one place: as a cache
    without it. A sequence of nothing else: zeros, lse -infinity."""
    import torch

    log(f"attend keys of infinity {qt} {ct} dim {dim} one:{one}")
    c = Case(gpu, 2, 2, 1, dim, 8, [700 if one else 300, 5], qt, ct, seed=dim + one, scores=True)
    try:
        sign = torch.sign(c.q.float())
        assert bool((sign != 0).all())
        for b, n in enumerate(c.lens):
            for t in range(n):
                if b == 1 or t % 3:
                    p, s = O.place(c.table, b, t, 8)
                    inf = (-float("inf") * sign[b]).to(c.k.dtype)
                    at = t % dim if one else slice(None)
                    c.k[p, :, s, at] = inf[:, at]
        c.dev["k"] = c.k.cuda()
        out, lse, so = c.attend()
        assert not out[1].any() and torch.isneginf(lse[1]).all()
        assert torch.equal(so[1, :, :5].cpu(), 0.9 * c.scores[1, :, :5])
        keep = [t for t in range(c.lens[0]) if t % 3 == 0]
        for h in range(2):
            want, tol, wl, dl, w, dw = _expect(c, keep, 0, h)
            _close(_np(out)[0, h], want, tol, "out")
            _close(_np(lse)[0, h], wl, dl, "lse")
            got = np.zeros(c.lens[0])
            got[keep] = w
            full = 0.9 * _np(c.scores)[0, h, :c.lens[0]] + got
            _close(_np(so)[0, h, :c.lens[0]], full, 2 * U * np.abs(full) + 2 * U + dw * got, "scores")
        assert gpu.dq_kv_take_errors(c.ctx) == 0
    finally:
        c.close()


@pytest.mark.parametrize("qt,ct", PAIRS)
def test_keys_whose_score_is_not_a_number(gpu, qt, ct):
    """A score of +infinity, infinities of both signs and a NaN show in their
    head and in no other."""
    import torch

    log(f"attend not a number {qt} {ct}")
    for what in ("up", "both", "nan"):
        c = Case(gpu, 2, 2, 2, 64, 16, [200, 33], qt, ct, seed=3)
        try:
            c.q = c.q.abs() + 0.5
            p, s = O.place(c.table, 0, 77, 16)
            if what == "nan":
                c.dev["k"][p, 1, s, 5] = float("nan")
            else:
                c.dev["k"][p, 1, s, 5] = float("inf")
                if what == "both":
                    c.dev["k"][p, 1, s, 6] = -float("inf")
            c.dev["q"] = c.q.cuda()
            out, lse, _ = c.attend()
            assert torch.isnan(out[0, 2:]).all() and torch.isnan(lse[0, 2:]).all()
            assert torch.isfinite(out[0, :2]).all() and torch.isfinite(lse[0, :2]).all()
            c.check((out, lse, None), rows=[1])
        finally:
            c.close()


@pytest.mark.parametrize("qt,ct", PAIRS + [("f32", "i8"), ("f16", "i8"), ("bf16", "i8")])
def test_queries_of_infinity(gpu, qt, ct):
    """An infinite value of a query against keys of one sign there: scores of
    -infinity weigh nothing, +infinity shows; other heads do not see it. On an
    int8 cache a query that is split into pieces counts as NaN instead."""
    import torch

    log(f"attend infinite query {qt} {ct}")
    c = Case(gpu, 1, 2, 2, 64, 16, [150], qt, ct, seed=4)
    try:
        for t in range(150):
            p, s = O.place(c.table, 0, t, 16)
            c.k[p, 0, s, 9] = -3 if ct == "i8" else -1.5
        c.q[0, 0, 9] = float("inf")
        c.q[0, 1, 9] = -float("inf")
        c.dev["k"], c.dev["q"] = c.k.cuda(), c.q.cuda()
        out, lse, _ = c.attend()
        if ct == "i8" and qt != "bf16":
            assert torch.isnan(out[0, 0]).all() and bool(torch.isnan(lse[0, 0]))
        else:
            assert not out[0, 0].any() and bool(torch.isneginf(lse[0, 0]))
        assert torch.isnan(out[0, 1]).all() and bool(torch.isnan(lse[0, 1]))
        assert torch.isfinite(out[0, 2:]).all() and torch.isfinite(lse[0, 2:]).all()
    finally:
        c.close()
