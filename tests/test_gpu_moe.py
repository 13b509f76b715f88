"""The experts' router, the sum of their results, and a whole layer of experts
on the GPU against the fp64 oracle."""
import numpy as np
import pytest

import w4_case as W
from gpu_case import log
from oracle import experts as X

pytestmark = pytest.mark.gpu


def _route(gpu, torch, logits, top_k, type="f32", sigmoid=False, normalize=True, scale=1.0, h=None, max_tokens=None):
    tokens, experts = logits.shape
    own = h is None
    if own:
        h = gpu.dq_moe_init(max_tokens or max(1, tokens), experts, top_k, W.code(gpu, type),
                            gpu.DQ_MOE_SIGMOID if sigmoid else gpu.DQ_MOE_SOFTMAX, normalize, scale)
    i = lambda *s: torch.full(s, -7, dtype=torch.int32, device="cuda")  # noqa: E731
    ids, off, tok, row = i(tokens, top_k), i(experts + 1), i(tokens * top_k), i(tokens, top_k)
    w = torch.full((tokens, top_k), -7.0, device="cuda")
    gpu.dq_moe_route(h, logits, ids, w, off, tok, row)
    torch.cuda.synchronize()
    if own:
        gpu.dq_moe_release(h)
    return [t.cpu().numpy() for t in (ids, w, off, tok, row)]


def _check_route(got, want, what):
    ids, w, off, tok, row = want
    assert np.array_equal(got[0], ids), what
    assert np.array_equal(got[2], off) and np.array_equal(got[4], row), what
    assert np.array_equal(got[3][:len(tok)], tok) and (got[3][len(tok):] == -7).all(), what
    assert np.array_equal(np.isnan(got[1]), np.isnan(w)), what
    # in units of 2^-24 of a weight: the argument of exp is a difference of at
    # most 16 with one rounding (16), exp itself (4); the sum of up to 1024 such
    # terms adds its 22 roundings a term (16 in a lane, 6 across); the same for
    # the term above it (20), quotient and factor (2): below 64
    err = np.abs(got[1] - w)
    assert (err[~np.isnan(w)] <= 64 * 2.0 ** -24 * np.abs(w[~np.isnan(w)]) + 2.0 ** -126).all(), what


@pytest.mark.parametrize("type", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("tokens,experts,top_k", [(1, 1, 1), (1, 8, 2), (7, 64, 6), (65, 65, 8), (130, 128, 1),
                                                  (33, 300, 32), (5, 1024, 10), (200, 16, 16), (64, 7, 7),
                                                  (1000, 40, 3)])
def test_route(gpu, type, tokens, experts, top_k):
    import torch

    r = np.random.default_rng(tokens * experts)
    logits = torch.from_numpy(r.normal(0, 2, (tokens, experts))).to(W.dtype(torch, type))
    for sigmoid, normalize, scale in ((False, True, 1.0), (False, False, 2.5), (True, True, 1.0), (True, False, 1.0)):
        log(f"route {tokens} x {experts} top {top_k} {type} sigmoid {sigmoid} normalize {normalize}")
        got = _route(gpu, torch, logits.cuda(), top_k, type, sigmoid, normalize, scale)
        _check_route(got, X.route(logits.double().numpy(), top_k, sigmoid, normalize, scale), type)


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_ties_masks_and_values_not_finite(gpu, type, sigmoid):
    import torch

    inf, nan = float("inf"), float("nan")
    r = np.random.default_rng(3)
    logits = r.integers(-2, 3, (300, 70)).astype(np.float64)  # nearly all tied
    logits[5], logits[6, 1:], logits[7, 3:] = -inf, -inf, -inf
    logits[8, 9], logits[9] = nan, nan
    logits[10, 4], logits[11, :3] = inf, inf
    logits[12] = torch.finfo(W.dtype(torch, type)).min
    logits[13] = np.where(r.random(70) < 0.9, -inf, 0.0)
    logits[14, :] = 0.0
    logits[14, ::2] = -0.0  # equal to 0
    x = torch.from_numpy(logits).to(W.dtype(torch, type))
    for normalize in (True, False):
        got = _route(gpu, torch, x.cuda(), 4, type, sigmoid, normalize)
        _check_route(got, X.route(x.double().numpy(), 4, sigmoid, normalize), f"{type} {sigmoid} {normalize}")


def test_route_strided_fewer_tokens_none_and_again(gpu):
    """Logits of a wider tensor, calls of other numbers of tokens on one context."""
    import torch

    r = np.random.default_rng(8)
    wide = torch.from_numpy(r.normal(0, 1, (500, 50)).astype(np.float32)).cuda()
    logits = wide[:, 7:39]
    h = gpu.dq_moe_init(500, 32, 5, gpu.DQ_F32)
    for tokens in (500, 1, 0, 64, 300, 500):
        got = _route(gpu, torch, logits[:tokens], 5, h=h)
        _check_route(got, X.route(logits[:tokens].double().cpu().numpy().reshape(tokens, 32), 5), f"{tokens} tokens")
    gpu.dq_moe_release(h)


def test_route_many_tokens(gpu):
    """Chunks of tokens, one expert that takes all, one that takes none."""
    import torch

    r = np.random.default_rng(11)
    logits = r.normal(0, 1, (5000, 24)).astype(np.float32)
    logits[:, 3], logits[:, 17] = 9.0, -np.inf
    got = _route(gpu, torch, torch.from_numpy(logits).cuda(), 3)
    _check_route(got, X.route(logits, 3), "many tokens")
    assert got[2][4] - got[2][3] == 5000 and got[2][18] == got[2][17]


@pytest.mark.parametrize("y", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
def test_combine(gpu, y, out):
    import torch

    r = np.random.default_rng(1)
    for tokens, top_k, N, add, cut in ((1, 1, 1, False, 0), (9, 3, 40, True, 0), (33, 8, 72, False, 0), (5, 2, 1027, True, 0),
                                       (300, 4, 64, True, 0), (7, 2, 48, True, 1)):
        rows = tokens * top_k
        h = gpu.dq_moe_init(tokens, 64, top_k, gpu.DQ_F32)
        yv = torch.from_numpy(r.normal(0, 1, (rows, N))).to(W.dtype(torch, y))
        row_of = r.permutation(rows).reshape(tokens, top_k).astype(np.int32)
        row_of[r.random((tokens, top_k)) < 0.1] = -1
        if tokens > 5:
            row_of[3], row_of[4, 0] = -1, -2 ** 31
        w = r.normal(0, 1, (tokens, top_k)).astype(np.float32)
        w[row_of < 0] = np.nan  # what has no row counts nothing whatever its weight
        av = torch.from_numpy(r.normal(0, 1, (tokens, N))).to(W.dtype(torch, out)) if add else None
        flat = torch.full((tokens * N + 8,), 77.0, dtype=W.dtype(torch, out), device="cuda")
        o = flat[cut:cut + tokens * N].view(tokens, N)  # cut: not 16-byte aligned
        log(f"combine {tokens} x {top_k} of {N} {y} -> {out}")
        gpu.dq_moe_combine(h, yv.cuda(), torch.from_numpy(w).cuda(), torch.from_numpy(row_of).cuda(), o,
                           add=None if av is None else av.cuda())
        torch.cuda.synchronize()
        a = None if av is None else av.double().numpy()
        want = X.combine(yv.double().numpy(), w, row_of, a)
        # one rounding a product and a sum, relative to the magnitudes' sum; then out's
        size = X.combine(np.abs(yv.double().numpy()), np.abs(w), row_of, None if a is None else np.abs(a))
        err = np.abs(o.double().cpu().numpy() - want)
        bound = (2 * top_k + 1) * 2.0 ** -24 * size
        assert (err <= bound + W.ROUND[out] * (np.abs(want) + bound) + W.SMALL[out]).all()
        assert (flat[:cut] == 77.0).all() and (flat[cut + tokens * N:] == 77.0).all()
        gpu.dq_moe_release(h)


def test_combine_rows_that_do_not_exist_and_in_place(gpu):
    import torch

    h = gpu.dq_moe_init(4, 8, 2, gpu.DQ_F32)
    y = torch.arange(12.0, device="cuda").view(3, 4)
    row_of = torch.tensor([[0, 1], [2, 3], [-1, -1], [2 ** 31 - 1, 0]], dtype=torch.int32, device="cuda")
    out = torch.ones((4, 4), device="cuda")
    gpu.dq_moe_combine(h, y, torch.full((4, 2), 0.5, device="cuda"), row_of, out, add=out)
    torch.cuda.synchronize()
    assert torch.equal(out[0], 1 + 0.5 * (y[0] + y[1])) and torch.equal(out[2], torch.ones(4, device="cuda"))
    assert torch.isnan(out[1]).all() and torch.isnan(out[3]).all()
    gpu.dq_moe_release(h)


def _layer(gpu, torch, tokens, experts, top_k, width, hidden, seed, type="bf16"):
    """Everything a layer of experts needs, on the device, and its call."""
    up = W.make(torch, seed, experts, hidden, width, 64, tokens, type, type, True, False, True)
    down = W.make(torch, seed + 1, experts, width, hidden, 32, 1, type, type, False, True, False)
    shared = W.make(torch, seed + 2, 1, width, width, 128, 1, type, type, True, False, False)
    r = np.random.default_rng(seed)
    s = dict(up=up, down=down, shared=shared, tokens=tokens, experts=experts, top_k=top_k)
    s["h_up"] = W.handle(gpu, up, type, tokens * top_k)
    s["h_down"] = W.handle(gpu, down, "f32", tokens * top_k)
    s["h_shared"] = W.handle(gpu, shared, type, tokens)
    s["moe"] = gpu.dq_moe_init(tokens, experts, top_k, gpu.DQ_F32)
    s["x"] = up["x"].cuda()
    s["logits"] = torch.from_numpy(r.normal(0, 1, (tokens, experts)).astype(np.float32)).cuda()
    dt, i32 = W.dtype(torch, type), dict(dtype=torch.int32, device="cuda")
    s["ids"], s["row_of"] = torch.empty((tokens, top_k), **i32), torch.empty((tokens, top_k), **i32)
    s["weights"] = torch.empty((tokens, top_k), device="cuda")
    s["offsets"], s["row_token"] = torch.empty(experts + 1, **i32), torch.empty(tokens * top_k, **i32)
    s["mid"] = torch.zeros((tokens * top_k, hidden), dtype=dt, device="cuda")
    s["y"] = torch.zeros((tokens * top_k, width), device="cuda")
    s["out"] = torch.empty((tokens, width), dtype=dt, device="cuda")
    return s


def _run_layer(gpu, s):
    gpu.dq_moe_route(s["moe"], s["logits"], s["ids"], s["weights"], s["offsets"], s["row_token"], s["row_of"])
    gpu.dq_w4_forward_grouped(s["h_up"], s["x"], s["offsets"], s["mid"], row_index=s["row_token"])
    gpu.dq_w4_forward_grouped(s["h_down"], s["mid"], s["offsets"], s["y"])
    gpu.dq_w4_forward(s["h_shared"], s["x"], s["out"])
    gpu.dq_moe_combine(s["moe"], s["y"], s["weights"], s["row_of"], s["out"], add=s["out"])


def _free_layer(gpu, s):
    for n in ("h_up", "h_down", "h_shared"):
        gpu.dq_w4_release(s[n])
    gpu.dq_moe_release(s["moe"])


def _layer_want(torch, s):
    """Each step of the layer by the oracle, from what the step before left on
    the device, so that each has its own bound."""
    ids, w, off, tok, row = X.route(s["logits"].double().cpu().numpy(), s["top_k"])
    assert np.array_equal(s["ids"].cpu().numpy(), ids) and np.array_equal(s["offsets"].cpu().numpy(), off)
    mid, x = s["mid"].cpu(), s["x"].cpu()
    for e in range(s["experts"]):
        a, b = off[e], off[e + 1]
        if a < b:
            W.check(mid[a:b], *W.want(s["up"], e, x[tok[a:b]]), s["up"]["type"], f"up {e}")
            W.check(s["y"][a:b], *W.want(s["down"], e, mid[a:b]), "f32", f"down {e}")
    y = s["y"].double().cpu().numpy()
    ref, bound = W.want(s["shared"], 0, x)
    t = s["up"]["type"]
    # the shared expert's rows were rounded once before the sum, then the sum
    want = X.combine(y, w, row, ref)
    size = X.combine(np.abs(y), np.abs(w), row, np.abs(ref))
    # the weights' own error (as tested above): 64 roundings
    d = bound + W.ROUND[t] * (np.abs(ref) + bound) + (2 * s["top_k"] + 65) * 2.0 ** -24 * size
    err = np.abs(s["out"].double().cpu().numpy() - want)
    assert (err <= d + W.ROUND[t] * (np.abs(want) + d) + W.SMALL[t]).all()


@pytest.mark.parametrize("tokens,type", [(1, "bf16"), (6, "f16"), (50, "bf16"), (40, "f32"), (400, "bf16")])
def test_layer_of_experts(gpu, tokens, type):
    import torch

    log(f"layer of experts, {tokens} tokens, {type}")
    s = _layer(gpu, torch, tokens, 12, 3, 160, 96, tokens, type)
    _run_layer(gpu, s)
    torch.cuda.synchronize()
    _layer_want(torch, s)
    _free_layer(gpu, s)


def test_layer_of_experts_replays(gpu):
    """The whole layer captured, replayed on other tokens with eager calls
    between, against the eager results bit for bit."""
    import torch

    s = _layer(gpu, torch, 30, 10, 2, 128, 64, 5)
    sets = []
    for i in range(3):
        x = (torch.randn(s["x"].shape, generator=torch.Generator().manual_seed(i))).to(s["x"].dtype).cuda()
        sets.append((x, torch.randn(s["logits"].shape, generator=torch.Generator().manual_seed(50 + i)).cuda()))
    eager = []
    for x, l in sets:
        s["x"].copy_(x)
        s["logits"].copy_(l)
        _run_layer(gpu, s)
        torch.cuda.synchronize()
        eager.append(s["out"].clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _run_layer(gpu, s)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _run_layer(gpu, s)
    for _ in range(3):
        for (x, l), want in zip(sets, eager):
            s["x"].copy_(x)
            s["logits"].copy_(l)
            s["out"].zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(s["out"], want)
            _run_layer(gpu, s)
            torch.cuda.synchronize()
            assert torch.equal(s["out"], want)
    _free_layer(gpu, s)


def test_route_more_chunks_than_one_workgroup_sums(gpu):
    """Over 16384 tokens, where the chunks' counts are summed by a launch of
    their own; and fewer tokens on the same context afterwards."""
    import torch

    r = np.random.default_rng(21)
    logits = torch.from_numpy(r.normal(0, 1, (17001, 6)).astype(np.float32))
    logits[100:200] = -np.inf
    h = gpu.dq_moe_init(17001, 6, 2, gpu.DQ_F32)
    for tokens in (17001, 16385, 16384, 300):
        got = _route(gpu, torch, logits[:tokens].cuda(), 2, h=h)
        _check_route(got, X.route(logits[:tokens].double().numpy(), 2), f"{tokens} tokens")
    gpu.dq_moe_release(h)
