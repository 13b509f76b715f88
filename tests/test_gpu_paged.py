"""GPU tests of rotary positions and the paged key-value cache (append, read,
attention of one new token, eviction) against the fp64 oracle, over types,
head layouts, lengths from zero on, odd page sizes, windows, strided inputs,
values that are not finite in places that must not count, and places that do
not exist.

Tolerances, set from the arithmetic: u = 2^-24 is half a step of fp32, h(t)
half a step of the output's type. A rotation takes two products and a sum of
fp32 values whose cos and sin are rounded once: 3 u (|a| + |b|), plus h. A
score is a dot product of D fp32 terms: its error is 4 sqrt(D) + 16 steps of
the largest sum of |q k| (rounding errors of D terms spread as sqrt(D); four
deviations, and 16 for the scaling, the maximum and exp). The weights' error
relative to themselves is twice that and the sums' (n / 128 + 64) u, once for
the numerator and once for the denominator; the values they are multiplied
with keep them to 2^-16 (16-bit outputs) or 2^-20 (fp32)."""
import numpy as np
import pytest

from gpu_case import log
from oracle import paged as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def _types(torch):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "i8": torch.int8}


def _code(dq, name):
    return {"f32": dq.DQ_F32, "bf16": dq.DQ_BF16, "f16": dq.DQ_F16, "i8": dq.DQ_I8}[name]


def _np(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def _close(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        ok = same | (np.abs(got - want) <= tol)
    assert ok.all(), (f"{what}: {(~ok).sum()} of {ok.size} beyond the bound, first at {np.argwhere(~ok)[0]}: "
                      f"{got[~ok][0]} for {want[~ok][0]}")


# ------------------------------------------------------------------ rotary

@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("interleaved,inverse", [(False, False), (True, True), (False, True)])
@pytest.mark.parametrize("tokens,heads,dim,rot,axes", [(1, 1, 2, 2, 1), (5, 3, 64, 64, 3), (3, 7, 80, 40, 2),
                                                       (4, 2, 10, 6, 1), (257, 33, 128, 64, 3), (2, 1, 1024, 1024, 8)])
def test_rope(gpu, kind, interleaved, inverse, tokens, heads, dim, rot, axes):
    import torch

    log(f"rope {kind} {tokens}x{heads}x{dim} rot:{rot} axes:{axes} {interleaved} {inverse}")
    g = torch.Generator().manual_seed(tokens + dim)
    x = torch.randn((tokens, heads, dim), generator=g).to(_types(torch)[kind])
    pos = torch.randint(-3, 1 << 20, (axes, tokens), generator=g, dtype=torch.int32)
    axis = [i % axes for i in range(rot // 2)]
    if rot // 2 < axes:
        pos = pos[:rot // 2].contiguous()
    freq = [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    ctx = gpu.dq_rope_init(dim, rot, axis, freq, interleaved)
    try:
        y = torch.empty_like(x, device="cuda")
        gpu.dq_rope_forward(ctx, x.cuda(), pos.cuda(), y, inverse=inverse)
        # out of a wider tensor, with an odd offset, and in place
        wide = torch.zeros((tokens, heads + 2, dim + 3), dtype=x.dtype, device="cuda")
        part = wide[:, 1:heads + 1, 1:dim + 1]
        part.copy_(x)
        gpu.dq_rope_forward(ctx, part, pos.cuda(), part, inverse=inverse)
        torch.cuda.synchronize()
        want = O.rotate(_np(x), pos.numpy(), axis, freq, interleaved, inverse)
        tol = HALF[kind] * np.abs(want) + 3 * U * 2 * np.abs(_np(x)).max(-1, keepdims=True)
        _close(_np(y), want, tol, "rope")
        assert torch.equal(part.contiguous(), y)
        assert not wide[:, 0].any() and not wide[:, -1].any() and not wide[:, :, 0].any() and not wide[:, :, -2:].any()
        if rot < dim:
            assert torch.equal(y[..., rot:].cpu(), x[..., rot:])
        assert "rotary" in gpu.dq_rope_info(ctx)
    finally:
        gpu.dq_rope_release(ctx)


def test_rope_far_positions_and_no_tokens(gpu):
    """Positions of 31 bits: the angle keeps its place within a turn."""
    import torch

    log("rope far positions")
    ctx = gpu.dq_rope_init(4, 4, [0, 0], [1.0, 0.7])
    try:
        x = torch.tensor([[[1.0, 2.0, 3.0, 4.0]]], device="cuda").expand(4, 1, 4).contiguous()
        pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 0, 123456789], dtype=torch.int32, device="cuda")
        y = torch.empty_like(x)
        gpu.dq_rope_forward(ctx, x, pos, y)
        want = O.rotate(_np(x), pos.cpu().numpy()[None], [0, 0], [1.0, 0.7])
        _close(_np(y), want, U * np.abs(want) + 3 * U * 8, "far")
        assert torch.equal(y[2], x[2])
        none = torch.empty((0, 1, 4), device="cuda")
        gpu.dq_rope_forward(ctx, none, torch.empty((1, 0), dtype=torch.int32, device="cuda"), none)
    finally:
        gpu.dq_rope_release(ctx)


def test_rope_gradient_by_differences(gpu):
    """The inverse pass is the gradient: against differences in fp32 of a
    large enough step (the map is linear, so any step is exact up to rounding)."""
    import torch

    log("rope gradient")
    dim, freq, axis = 16, [1.0 / (i + 1) for i in range(6)], [0, 1, 0, 1, 0, 1]
    for il in (False, True):
        ctx = gpu.dq_rope_init(dim, 12, axis, freq, il)
        try:
            pos = torch.tensor([[7, 1000], [3, 9]], dtype=torch.int32, device="cuda")
            g = torch.randn((2, 1, dim), generator=torch.Generator().manual_seed(1)).cuda()
            dx = torch.empty_like(g)
            gpu.dq_rope_forward(ctx, g, pos, dx, inverse=True)
            for d in range(dim):
                e = torch.zeros_like(g)
                e[..., d] = 1.0
                up, down = torch.empty_like(g), torch.empty_like(g)
                gpu.dq_rope_forward(ctx, e, pos, up)
                gpu.dq_rope_forward(ctx, -e, pos, down)
                diff = ((up - down).double() * g.double()).sum(-1) / 2
                _close(_np(diff), _np(dx[..., d]), 8 * U * float(g.abs().max()) * 2, f"gradient {d}")
        finally:
            gpu.dq_rope_release(ctx)


# ------------------------------------------------------------------- cache

class Case:
    """A cache whose unused slots and pages hold NaN (int8: NaN scales), with
    block table entries that no call may follow set to bad ones."""

    def __init__(self, gpu, batch, hk, group, dim, page, lens, qt, ct, seed=0, window=0, scores=False, spare=2,
                 per_seq=None, ctx_batch=None):
        import torch

        self.dq, self.torch = gpu, torch
        self.batch, self.hk, self.group, self.dim, self.page, self.window = batch, hk, group, dim, page, window
        self.hq, self.qt, self.ct, self.lens = hk * group, qt, ct, list(lens)
        r = np.random.default_rng(seed)
        need = [-(-n // page) for n in self.lens]
        self.per_seq = per_seq or max(1, max(need)) + 1
        self.cap = self.per_seq * page
        self.pages = sum(need) + spare
        perm = r.permutation(self.pages)
        table = np.full((batch, self.per_seq), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
            first = max(0, self.lens[b] - window) if window else 0
            table[b, :first // page] = self.pages + 5 if b % 2 else -7
        self.table = table
        shape = (self.pages, hk, page, dim)
        used = np.zeros(shape[:3], bool)
        for b, n in enumerate(self.lens):
            first = max(0, n - window) if window else 0
            for t in range(first, n):
                used[table[b, t // page], :, t % page] = True
        self.k_scale = self.v_scale = None
        for name in ("k", "v"):
            x = r.normal(0, 1, shape).astype(np.float32)
            if name == "k":
                x[..., ::max(1, dim // 4)] += 1.5
            if ct == "i8":
                codes = np.clip(np.rint(x * 40), -127, 127).astype(np.int8)
                codes[~used] = 127
                scale = r.uniform(0.01, 0.04, shape[:3]).astype(np.float32)
                scale[~used] = np.nan
                setattr(self, name, torch.from_numpy(codes))
                setattr(self, name + "_scale", torch.from_numpy(scale))
            else:
                x[~used] = np.nan if name == "k" else np.inf
                setattr(self, name, torch.from_numpy(x).to(_types(torch)[ct]))
        self.q = (torch.from_numpy(r.normal(0, 1.5, (batch, self.hq, dim)).astype(np.float32))).to(_types(torch)[qt])
        self.sm = dim ** -0.5
        self.scores = torch.from_numpy(r.random((batch, hk, self.cap)).astype(np.float32)) if scores else None
        self.ctx = gpu.dq_kv_init(ctx_batch or batch, self.hq, hk, dim, self.pages, page, self.per_seq,
                                  _code(gpu, qt), _code(gpu, ct), scores)
        self.dev = {}
        for n in ("k", "v", "k_scale", "v_scale", "q", "scores"):
            t = getattr(self, n)
            self.dev[n] = None if t is None else t.cuda()
        self.dev["table"] = torch.from_numpy(table).cuda()
        self.dev["lens"] = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def cache(self):
        d = self.dev
        return d["table"], d["k"], d["v"], d["k_scale"], d["v_scale"]

    def attend(self, **more):
        torch, d = self.torch, self.dev
        out = torch.full((self.batch, self.hq, self.dim), 7.0, dtype=_types(torch)[self.qt], device="cuda")
        lse = torch.full((self.batch, self.hq), 7.0, device="cuda")
        so = None
        if self.scores is not None:
            so = torch.full((self.batch, self.hk, self.cap), 7.0, device="cuda")
            more = dict(scores=d["scores"], scores_out=so, decay=0.9, **more)
        self.dq.dq_kv_attend(self.ctx, more.pop("q", d["q"]), d["lens"], *self.cache(), out, self.sm, lse=lse,
                             window=self.window, **more)
        torch.cuda.synchronize()
        return out, lse, so

    def check(self, got, rows=None):
        out, lse, so = got
        f = lambda t: None if t is None else t.float().numpy() if t.is_floating_point() else t.numpy()  # noqa: E731
        want, wl, ws, mass, reach = O.attend(f(self.q), self.lens, self.table, f(self.k), f(self.v), f(self.k_scale),
                                             f(self.v_scale), self.sm, self.page, self.window)
        n = max(self.lens)
        ds = reach * (4 * np.sqrt(self.dim) + 16) * U
        sums = (n / 128 + 64) * U
        dp = 2 * (ds + sums)
        keep = 2.0 ** -20 if self.qt == "f32" else 2.0 ** -16
        rows = list(range(self.batch)) if rows is None else rows
        tol = HALF[self.qt] * np.abs(want) + (2 * dp + keep)[..., None] * mass
        _close(_np(out)[rows], want[rows], tol[rows], "out")
        with np.errstate(invalid="ignore"):
            _close(_np(lse)[rows], wl[rows], (ds + sums + 2.0 ** -20 + 2 * U * np.abs(wl))[rows], "lse")
        if so is not None:
            held = np.arange(self.cap)[None, None] < np.array(self.lens)[:, None, None]
            full = np.where(held, 0.9 * _np(self.scores) + ws, 7.0)
            worst = dp.reshape(self.batch, self.hk, self.group).max(-1)[..., None]
            _close(_np(so)[rows], full[rows], (2 * U * np.abs(full) + 2 * U + worst * ws)[rows], "scores")

    def close(self):
        self.dq.dq_kv_release(self.ctx)


def _run(case, **more):
    try:
        case.check(case.attend(**more))
        assert case.dq.dq_kv_take_errors(case.ctx) == 0
    finally:
        case.close()


# --------------------------------------------------------------- refusals

def test_refusals_with_a_context(gpu):
    """Every refusal leaves the outputs alone and launches nothing."""
    import torch

    log("refusals")
    c = Case(gpu, 2, 2, 2, 32, 8, [9, 3], "bf16", "i8", scores=False)
    other = Case(gpu, 2, 2, 2, 32, 8, [9, 3], "bf16", "bf16")
    rope64 = gpu.dq_rope_init(64, 64, [0] * 32, [1.0] * 32)
    try:
        d = c.dev
        out = torch.full((2, 4, 32), 7.0, dtype=torch.bfloat16, device="cuda")
        state = torch.zeros((2, 2, c.cap), device="cuda")

        def refused(status, fn, *a, **k):
            with pytest.raises(gpu.DQError) as e:
                fn(*a, **k)
            assert e.value.status == status, str(e.value)

        def attend(ctx=c.ctx, q=d["q"], cache=c.cache(), out=out, sm=0.1, **k):
            gpu.dq_kv_attend(ctx, q, d["lens"], *cache, out, sm, **k)

        ARG, STATE = gpu.DQ_ERR_ARG, gpu.DQ_ERR_STATE
        refused(STATE, attend, scores=state, scores_out=state)
        refused(ARG, attend, window=-1)
        refused(ARG, attend, sm=float("nan"))
        refused(ARG, attend, sm=float("inf"))
        refused(ARG, attend, scores=state)
        refused(ARG, attend, out=None)
        refused(ARG, attend, cache=c.cache()[:3] + (None, None))
        refused(ARG, attend, ctx=other.ctx, cache=other.cache()[:3] + c.cache()[3:])
        refused(ARG, attend, cache=(None,) + c.cache()[1:])
        refused(ARG, attend, q=torch.zeros((3, 4, 32), dtype=torch.bfloat16, device="cuda"),
                out=torch.zeros((3, 4, 32), dtype=torch.bfloat16, device="cuda"))
        odd = torch.zeros(2 * 4 * 32 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(2, 4, 32)
        refused(ARG, attend, out=odd)
        shifted = torch.zeros(d["k"].numel() + 1, dtype=torch.int8, device="cuda")[1:]
        refused(ARG, attend, cache=(c.cache()[0], shifted) + c.cache()[2:])

        kv = torch.zeros((3, 2, 32), dtype=torch.bfloat16, device="cuda")
        q = torch.zeros((3, 4, 32), dtype=torch.bfloat16, device="cuda")
        idx = torch.zeros(3, dtype=torch.int32, device="cuda")
        pos = torch.zeros((1, 3), dtype=torch.int32, device="cuda")
        refused(ARG, gpu.dq_kv_append, c.ctx, kv, kv, idx, *c.cache())                      # 3 tokens, no seq_ids
        refused(ARG, gpu.dq_kv_append, c.ctx, kv, kv, None, *c.cache(), seq_ids=idx)
        refused(ARG, gpu.dq_kv_append, c.ctx, kv, kv, idx, *c.cache(), seq_ids=idx, q=q)    # no q_out
        refused(ARG, gpu.dq_kv_append, c.ctx, kv, kv, idx, *c.cache(), seq_ids=idx, rope=rope64, positions=pos)
        refused(ARG, gpu.dq_kv_append, c.ctx, kv, kv, idx, *c.cache()[:3], seq_ids=idx)     # no scales
        refused(ARG, gpu.dq_kv_read, c.ctx, idx, *c.cache(), seq_ids=idx)                   # nothing to write
        refused(ARG, gpu.dq_kv_read, c.ctx, idx, *c.cache(), k_out=kv)
        st = torch.zeros((2, 2, c.cap), dtype=torch.int32, device="cuda")
        ev = (d["lens"], d["lens"], state, st, *c.cache(), state, st)
        refused(ARG, gpu.dq_kv_evict, c.ctx, 0, *ev, d["lens"])
        refused(ARG, gpu.dq_kv_evict, c.ctx, 4, *ev, d["lens"], recent=-1)
        refused(ARG, gpu.dq_kv_evict, c.ctx, 4, *ev, d["lens"], sinks=-1)
        refused(ARG, gpu.dq_kv_evict, c.ctx, 4, *ev, None)
        rope = gpu.dq_rope_init(32, 32, [0] * 16, [1.0] * 16)
        x8 = torch.zeros((2, 1, 32), dtype=torch.int8, device="cuda")
        refused(gpu.DQ_ERR_TYPE, gpu.dq_rope_forward, rope, x8, idx, x8)
        refused(gpu.DQ_ERR_TYPE, gpu.dq_rope_forward, rope, x8, idx, x8, type_=gpu.DQ_I8)
        x, y = (torch.zeros((2, 2, 32), device="cuda") for _ in range(2))
        refused(ARG, gpu.dq_rope_forward, rope, x, None, y)
        refused(ARG, gpu.dq_rope_forward, rope, x, idx, x.transpose(0, 1))
        gpu.dq_rope_release(rope)
        torch.cuda.synchronize()
        assert bool((out == 7).all()) and gpu.dq_kv_take_errors(c.ctx) == 0
        assert torch.equal(d["k"].cpu(), c.k) and "paged cache" in gpu.dq_kv_info(c.ctx)
    finally:
        gpu.dq_rope_release(rope64)
        c.close()
        other.close()


# -------------------------------------------------------- append and read

@pytest.mark.parametrize("qt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("ct", ["bf16", "f16", "i8"])
@pytest.mark.parametrize("dim,rot,il,page", [(16, 16, False, 1), (64, 32, True, 8), (80, 80, False, 24),
                                             (96, 36, False, 16), (128, 128, True, 64), (256, 256, False, 5)])
def test_append_and_read(gpu, qt, ct, dim, rot, il, page):
    """Prompt chunks of ragged sequences out of a fused projection, padding
    tokens among them; the slots that are not named keep what they hold."""
    import torch

    log(f"append {qt}->{ct} {dim}/{rot} {il} page {page}")
    r = np.random.default_rng(dim + page)
    batch, hk, group = 3, 2, 3
    hq = hk * group
    c = Case(gpu, batch, hk, group, dim, page, [20, 33, 1], qt, ct, seed=dim)
    rope = gpu.dq_rope_init(dim, rot, [i % 2 for i in range(rot // 2)], [0.9 ** i for i in range(rot // 2)], il)
    try:
        places = [(b, t) for b in range(batch) for t in range(c.lens[b])]
        pick = [places[i] for i in r.permutation(len(places))[:31]]
        seq = np.array([b for b, _ in pick] + [0, 1], np.int32)
        idx = np.array([t for _, t in pick] + [-1, -5], np.int32)   # two padding tokens
        n = len(idx)
        fused = torch.from_numpy(r.normal(0, 1, (n, hq + 2 * hk, dim)).astype(np.float32)).to(_types(torch)[qt])
        fused[3, hq:] = 0                                            # rows of zeros
        pos = r.integers(0, 40000, (2, n)).astype(np.int32)
        f = fused.cuda()
        q_out = torch.empty((n, hq, dim), dtype=f.dtype, device="cuda")
        before = [None if t is None else t.clone() for t in c.cache()]
        seq_t, idx_t = torch.from_numpy(seq).cuda(), torch.from_numpy(idx).cuda()
        gpu.dq_kv_append(c.ctx, f[:, hq:hq + hk], f[:, hq + hk:], idx_t, *c.cache(), seq_ids=seq_t, q=f[:, :hq],
                         q_out=q_out, rope=rope, positions=torch.from_numpy(pos).cuda())
        k_out, v_out = (torch.empty((n, hk, dim), dtype=f.dtype, device="cuda") for _ in range(2))
        gpu.dq_kv_read(c.ctx, idx_t, *c.cache(), k_out=k_out, v_out=v_out, seq_ids=seq_t)
        torch.cuda.synchronize()
        assert gpu.dq_kv_take_errors(c.ctx) == 0
        x = fused.double().numpy()
        axis, freq = [i % 2 for i in range(rot // 2)], [0.9 ** i for i in range(rot // 2)]
        big = np.abs(x).max(-1, keepdims=True)
        want_q = O.rotate(x[:, :hq], pos, axis, freq, il)
        _close(_np(q_out), want_q, HALF[qt] * np.abs(want_q) + 6 * U * big[:, :hq], "q")
        want = {"k": O.rotate(x[:, hq:hq + hk], pos, axis, freq, il), "v": x[:, hq + hk:]}
        for name, back, heads in (("k", k_out, slice(hq, hq + hk)), ("v", v_out, slice(hq + hk, None))):
            w, b = want[name], big[:, heads]
            if ct == "i8":
                # half a step, the scale's and the quotient's rounding (3 u of the row's largest), the rotation's
                step = np.abs(w).max(-1, keepdims=True) / 127
                tol = 0.5 * step * (1 + 2.0 ** -20) + (3 + 6 * (name == "k")) * 2 * U * b
            else:
                tol = HALF[ct] * np.abs(w) + 6 * U * b + 2.0 ** -25 * (ct == "f16")  # fp16's subnormal step
            tol = tol + HALF[qt] * (np.abs(w) + tol)
            _close(_np(back)[:31], w[:31], tol[:31], name)
            assert not back[31:].any()
            if ct == "i8" and name == "v":
                # no rotation: the codes and scales of the definition, bit for bit
                codes, scale = O.quantize_rows(fused.float().numpy()[:31, heads])
                got_c, got_s = c.dev["v"].cpu().numpy(), c.dev["v_scale"].cpu().numpy()
                for i in range(31):
                    p, s = O.place(c.table, seq[i], idx[i], page)
                    assert np.array_equal(got_c[p, :, s], codes[i]) and np.array_equal(got_s[p, :, s], scale[i])
        # everything else is as it was
        mask = torch.ones(c.k.shape[:3], dtype=torch.bool)
        for i in range(31):
            p, s = O.place(c.table, seq[i], idx[i], page)
            mask[p, :, s] = False
        for old, new in zip(before[1:], c.cache()[1:]):
            if old is not None:
                kind = torch.int32 if old.element_size() == 4 else torch.int16 if old.element_size() == 2 else torch.int8
                assert torch.equal(old.view(kind).cpu()[mask], new.view(kind).cpu()[mask])
    finally:
        gpu.dq_rope_release(rope)
        c.close()


def test_append_one_token_each_without_rotation(gpu):
    """The serving step without seq_ids, queries or rotation; a row that is not
    finite, one whose scale underflows and places that do not exist."""
    import torch

    log("append step")
    for ct in ("i8", "bf16"):
        c = Case(gpu, 5, 1, 1, 32, 4, [6, 6, 6, 6, 6], "f32", ct)
        try:
            r = np.random.default_rng(1)
            k = r.normal(0, 1, (5, 1, 32)).astype(np.float32)
            v = k * 2
            k[0, 0, 5] = np.nan
            k[1, 0, 7] = -np.inf
            k[2, 0] = 1e-45
            idx = np.array([5, 4, 3, c.cap, 2 ** 31 - 1], np.int32)
            idx_t = torch.from_numpy(idx).cuda()
            gpu.dq_kv_append(c.ctx, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), idx_t, *c.cache())
            assert gpu.dq_kv_take_errors(c.ctx) > 0
            assert gpu.dq_kv_take_errors(c.ctx) == 0
            ko, vo = (torch.empty((5, 1, 32), device="cuda") for _ in range(2))
            gpu.dq_kv_read(c.ctx, idx_t, *c.cache(), k_out=ko, v_out=vo)
            assert gpu.dq_kv_take_errors(c.ctx) > 0
            ko, vo = ko.cpu().numpy(), vo.cpu().numpy()
            assert np.isnan(ko[3:]).all() and np.isnan(vo[3:]).all()
            if ct == "i8":
                assert np.isnan(ko[:2]).all() and not ko[2].any()
                assert np.abs(vo[:3] - v[:3]).max() <= np.abs(v).max() / 127
            else:
                assert np.isnan(ko[0, 0, 5]) and ko[1, 0, 7] == -np.inf and np.isfinite(ko[0, 0, :5]).all()
                assert np.array_equal(vo[:3], torch.from_numpy(v[:3]).bfloat16().float().numpy())
            # a sequence that does not exist
            bad_seq = torch.tensor([5, -1], dtype=torch.int32, device="cuda")
            old = c.dev["v"].clone()
            gpu.dq_kv_append(c.ctx, torch.from_numpy(k[3:]).cuda(), torch.from_numpy(v[3:]).cuda(),
                             torch.zeros(2, dtype=torch.int32, device="cuda"), *c.cache(), seq_ids=bad_seq)
            assert gpu.dq_kv_take_errors(c.ctx) > 0
            assert torch.equal(old.view(torch.int8), c.dev["v"].view(torch.int8))
        finally:
            c.close()


# --------------------------------------------------------------- attention

@pytest.mark.parametrize("qt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("ct", ["bf16", "f16", "i8"])
@pytest.mark.parametrize("scores", [False, True])
def test_attend_types(gpu, qt, ct, scores):
    log(f"attend {qt} {ct} scores:{scores}")
    _run(Case(gpu, 3, 2, 4, 64, 16, [37, 0, 300], qt, ct, seed=5, scores=scores))


@pytest.mark.parametrize("dim", [16, 32, 48, 64, 80, 96, 112, 128, 160, 192, 240, 256])
@pytest.mark.parametrize("ct", ["bf16", "f16", "i8"])
def test_attend_head_sizes(gpu, dim, ct):
    log(f"attend dim {dim} {ct}")
    qt = "bf16" if ct == "i8" else ct
    _run(Case(gpu, 2, 2, 2, dim, 24, [131, 5], qt, ct, seed=dim, scores=dim % 32 == 0))


@pytest.mark.parametrize("hk,group", [(1, 1), (3, 1), (2, 5), (1, 8), (2, 15), (1, 16), (2, 17), (1, 40)])
@pytest.mark.parametrize("qt,ct", [("f32", "i8"), ("bf16", "bf16")])
def test_attend_head_layouts(gpu, hk, group, qt, ct):
    log(f"attend heads {hk}x{group} {qt} {ct}")
    _run(Case(gpu, 2, hk, group, 32, 8, [77, 140], qt, ct, seed=hk + group, scores=True))


@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 32, 64, 100, 128, 500])
def test_attend_page_sizes_and_lengths(gpu, page):
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 0, 384]
    log(f"attend page {page}")
    _run(Case(gpu, len(lens), 1, 2, 32, page, lens, "bf16", "bf16", seed=page, scores=page == 24))


@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 100, 128, 129, 300, 1000])
@pytest.mark.parametrize("qt,ct", [("f16", "f16"), ("f32", "i8")])
def test_attend_windows(gpu, window, qt, ct):
    """Pages before the window may be gone: their entries are bad."""
    log(f"attend window {window} {qt} {ct}")
    _run(Case(gpu, 4, 2, 3, 48, 8, [400, 33, 1, 128], qt, ct, seed=window, window=window, scores=True))


@pytest.mark.parametrize("ct", ["bf16", "f16", "i8"])
def test_attend_long_sequences(gpu, ct):
    """Split over many workgroups and joined, next to short ones."""
    log(f"attend long {ct}")
    qt = "bf16" if ct == "i8" else ct
    _run(Case(gpu, 5, 2, 4, 128, 32, [9001, 3, 130, 0, 4000], qt, ct, seed=3, scores=True))
    _run(Case(gpu, 1, 1, 8, 64, 64, [20011], "f32", ct, seed=4))


@pytest.mark.parametrize("dim", [16, 48, 64, 80, 96, 128, 144, 192, 208, 256])
@pytest.mark.parametrize("qt,ct", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "i8"), ("f32", "i8"), ("f32", "bf16"),
                                   ("f32", "f16"), ("bf16", "f16"), ("f16", "i8")])
def test_attend_split_types_and_head_sizes(gpu, dim, qt, ct):
    """Room for more than 512 tokens: heads are split over workgroups."""
    log(f"attend split {qt} {ct} dim {dim}")
    _run(Case(gpu, 4, 1, 3, dim, 16, [700, 0, 1309, 5], qt, ct, seed=dim, scores=dim in (48, 128), per_seq=90))


@pytest.mark.parametrize("scores", [False, True])
@pytest.mark.parametrize("batch,hk,page,lens", [(300, 2, 8, (1, 9, 600, 0, 130)), (700, 1, 16, (33, 0, 0, 257)),
                                                (513, 1, 1, (3, 5, 0))])
def test_attend_many_sequences(gpu, batch, hk, page, lens, scores):
    """More sequences than a workgroup has threads, and more heads than
    workgroups; short ones whole, longer ones split."""
    log(f"attend {batch} sequences scores:{scores}")
    n = [lens[i % len(lens)] for i in range(batch)]
    _run(Case(gpu, batch, hk, 2, 16, page, n, "bf16", "i8", seed=batch, scores=scores))


@pytest.mark.parametrize("qt,ct,dim", [("bf16", "bf16", 64), ("bf16", "i8", 128), ("f32", "f16", 32),
                                       ("f32", "i8", 256)])
@pytest.mark.parametrize("batch,per_seq,window", [(15, 64, 0), (16, 64, 0), (16, 65, 0), (16, 130, 1024),
                                                  (16, 130, 1025), (66, 64, 0)])
def test_attend_many_heads(gpu, batch, per_seq, window, qt, ct, dim):
    """Either side of 128 heads, of 1024 slots and of a window of 1024: whole
    heads of up to eight units, or shared ones; more heads than workgroups."""
    log(f"attend {batch} sequences of {per_seq} pages window {window} {qt} {ct} {dim}")
    lens = [16 * per_seq, 0, 1, 1023, 513, 640, 129, 1000, 16 * per_seq - 1]
    _run(Case(gpu, batch, 8, 2, dim, 16, [lens[i % len(lens)] for i in range(batch)], qt, ct, seed=batch + per_seq,
              window=window, scores=dim != 64, per_seq=per_seq))


@pytest.mark.parametrize("scores", [False, True])
def test_attend_more_units_than_rounds(gpu, scores):
    """Enough tokens that workers take runs that cross sequences and heads."""
    log(f"attend runs scores:{scores}")
    r = np.random.default_rng(7)
    _run(Case(gpu, 12, 8, 1, 16, 64, [int(x) for x in r.integers(2000, 9000, 12)], "bf16", "bf16", seed=6,
              scores=scores))


@pytest.mark.parametrize("length", [100, 1000])
def test_attend_many_query_heads_with_weights(gpu, length):
    """Several tiles of query heads, more than are summed at a time."""
    log(f"attend 70 heads {length}")
    _run(Case(gpu, 2, 1, 70, 32, 16, [length, 17], "f32", "f16", seed=length, scores=True))
    _run(Case(gpu, 2, 1, 70, 32, 16, [length, 17], "bf16", "bf16", seed=length))


def test_attend_repeats_bit_for_bit(gpu):
    """The same call twice gives the same bits: parts are joined in order."""
    import torch

    log("attend repeats")
    c = Case(gpu, 6, 2, 4, 64, 16, [3000, 5, 700, 0, 1999, 2500], "bf16", "i8", seed=3, scores=True)
    try:
        first = c.attend()
        for _ in range(5):
            for a, b in zip(first, c.attend()):
                assert torch.equal(a, b)
    finally:
        c.close()


def test_attend_peaked_and_shifted_scores(gpu):
    """One token far above the others, all scores far below zero, growing
    scores (the running maximum moves at every step) and a negative scale."""
    import torch

    log("attend peaked")
    for qt, ct in (("bf16", "bf16"), ("f16", "f16"), ("f32", "i8"), ("f32", "f16")):
        for mode in range(4):
            c = Case(gpu, 1, 1, 3, 64, 16, [700], qt, ct, seed=mode)
            x = c.k.float() * (0.1 if mode != 3 else 1.0)
            for t in range(700):
                p, s = O.place(c.table, 0, t, 16)
                if mode == 0 and t == 333:
                    x[p, :, s] = 3.0 if ct != "i8" else 100
                if mode == 2:
                    x[p, :, s] = (t / 200.0) if ct != "i8" else t // 6
            if mode == 1:
                x = x - (2.0 if ct != "i8" else 40.0)
            if mode == 3:
                c.sm = -c.sm
            c.q = c.q.abs()
            c.k = x.round().clamp(-127, 127).to(torch.int8) if ct == "i8" else x.to(c.k.dtype)
            c.dev["k"], c.dev["q"] = c.k.cuda(), c.q.cuda()
            log(f"  {qt} {ct} mode {mode}")
            _run(c)


def test_attend_extreme_magnitudes(gpu):
    """Queries near both ends of their type, scales of an int8 cache over many
    powers of two: nothing overflows or is lost on the way."""
    import torch

    log("attend extremes")
    for qt, ct, up in (("f32", "f16", 1e30), ("f32", "f16", 1e-30), ("bf16", "f16", 1e30), ("f32", "bf16", 1e30),
                       ("bf16", "i8", 1e-30), ("f32", "i8", 1e20), ("f16", "bf16", 1e3)):
        c = Case(gpu, 2, 1, 4, 64, 16, [200, 1], qt, ct, seed=7)
        c.q = (c.q.float() * up).to(c.q.dtype)
        c.sm = 0.1 / up
        if ct == "i8":
            r = np.random.default_rng(3)
            c.v_scale = c.v_scale * torch.from_numpy((10.0 ** r.integers(-8, 8, tuple(c.v_scale.shape))).astype(np.float32))
            if qt == "bf16":
                c.v_scale = c.v_scale * 1e-20
        c.dev["q"] = c.q.cuda()
        c.dev["v_scale"] = None if c.v_scale is None else c.v_scale.cuda()
        log(f"  {qt} {ct} {up}")
        _run(c)


def test_attend_what_is_not_finite(gpu):
    """A NaN or infinite row that is attended to shows in the output; the rows
    of other sequences and heads do not."""
    log("attend not finite")
    import torch

    for qt, ct in (("bf16", "bf16"), ("f32", "f16"), ("f32", "i8")):
        c = Case(gpu, 3, 2, 2, 32, 8, [40, 40, 40], qt, ct, seed=1)
        try:
            p, s = O.place(c.table, 1, 17, 8)
            if ct == "i8":
                c.dev["v_scale"][p, 1, s] = float("nan")
            else:
                c.dev["v"][p, 1, s, 3] = float("nan")
            out, lse, _ = c.attend()
            c.check((out, lse, None), rows=[0, 2])
            assert torch.isnan(out[1, 2:, 3]).all() and torch.isfinite(out[1, :2]).all() and torch.isfinite(lse).all()
            if ct == "i8":
                c.dev["k_scale"][p, 0, s] = float("inf")
            else:
                c.dev["k"][p, 0, s] = float("inf")
            out, lse, _ = c.attend()
            c.check((out, lse, None), rows=[0, 2])
            # the row's score decides: -infinity weighs nothing, anything else not finite shows
            row = c.dev["k"][p, 0, s].double()
            dot = (c.dev["q"][1, :2].double() * row).sum(-1) * (float("inf") if ct == "i8" else 1)
            for h in range(2):
                shows = not bool(torch.isneginf(dot[h]))
                assert bool(torch.isnan(lse[1, h])) == shows and bool(torch.isnan(out[1, h]).all()) == shows
        finally:
            c.close()


def test_attend_scores_of_minus_infinity(gpu):
    """Tokens whose score is -infinity weigh nothing; when all do, the output
    is zero and lse -infinity."""
    import torch

    log("attend -inf")
    for qt, ct in (("bf16", "bf16"), ("f16", "f16")):
        c = Case(gpu, 2, 1, 2, 32, 8, [300, 5], qt, ct, seed=2, scores=True)
        c.q = c.q.abs() + 0.5
        for b, n in enumerate(c.lens):
            for t in range(n):
                if b == 1 or t % 3:
                    p, s = O.place(c.table, b, t, 8)
                    c.k[p, 0, s] = -float("inf")
        c.dev["q"], c.dev["k"] = c.q.cuda(), c.k.cuda()
        try:
            out, lse, so = c.attend()
            assert not out[1].any() and torch.isneginf(lse[1]).all()
            assert torch.allclose(so[1, 0, :5].cpu(), 0.9 * c.scores[1, 0, :5])
            # the same as a cache of the other tokens alone
            keep = [t for t in range(300) if t % 3 == 0]
            k = torch.stack([c.k[O.place(c.table, 0, t, 8)[0], 0, t % 8] for t in keep]).double()
            v = torch.stack([c.v[O.place(c.table, 0, t, 8)[0], 0, t % 8] for t in keep]).double()
            w = torch.softmax(c.sm * c.q[0].double() @ k.T, -1) @ v
            assert float((out[0].cpu().double() - w).abs().max()) <= HALF[qt] * float(w.abs().max()) + 1e-3
            assert torch.isfinite(so[0, 0, :300]).all()
        finally:
            c.close()


def test_attend_bad_pages_and_lengths(gpu):
    """Entries that name no page and lengths out of range: NaN for the
    sequences that need them, a count, and the others as ever."""
    import torch

    log("attend bad pages")
    for bad_page in (-1, 10 ** 6, -2 ** 31):
        c = Case(gpu, 4, 2, 2, 32, 8, [40, 300, 0, 9], "bf16", "i8", seed=1, scores=True)
        try:
            c.dev["table"][1, 20] = bad_page
            out, lse, so = c.attend()
            assert c.dq.dq_kv_take_errors(c.ctx) > 0
            assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
            c.check((out, lse, so), rows=[0, 2, 3])
        finally:
            c.close()
    c = Case(gpu, 3, 1, 2, 32, 8, [40, 16, 9], "f16", "f16", seed=1)
    try:
        c.dev["table"][2] = c.dev["table"][0]  # entries that exist for the length that is too long
        c.dev["lens"].copy_(torch.tensor([40, -3, 2 ** 31 - 1], dtype=torch.int32))
        out, lse, _ = c.attend()
        assert c.dq.dq_kv_take_errors(c.ctx) > 0
        c.check((out, lse, None), rows=[0])
        assert torch.isnan(out[1:]).all() and torch.isnan(lse[1:]).all()
    finally:
        c.close()


def test_attend_strided_queries_smaller_batches_and_streams(gpu):
    """Queries out of a fused projection, fewer sequences than the context
    has, no lse, weights gathered in place, on a stream of the caller's."""
    import torch

    log("attend strided")
    c = Case(gpu, 3, 2, 2, 64, 8, [70, 200, 9], "bf16", "bf16", seed=8, scores=True, ctx_batch=7)
    try:
        c.check(c.attend())
        fused = torch.zeros((3, 9, 65), dtype=torch.bfloat16, device="cuda")
        q = fused[:, 2:6, 1:]
        q.copy_(c.dev["q"])
        c.check(c.attend(q=q))
        want = c.attend()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        out = torch.empty_like(want[0])
        state = c.dev["scores"].clone()
        torch.cuda.synchronize()
        gpu.dq_kv_attend(c.ctx, c.dev["q"], c.dev["lens"], *c.cache(), out, c.sm, scores=state, scores_out=state,
                         decay=0.9, stream=side)
        side.synchronize()
        assert torch.equal(out, want[0])
        for b, n in enumerate(c.lens):
            assert torch.equal(state[b, :, :n], want[2][b, :, :n])
            assert torch.equal(state[b, :, n:], c.dev["scores"][b, :, n:])
        none = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
        gpu.dq_kv_attend(c.ctx, none, c.dev["lens"], *c.cache(), none, c.sm)
    finally:
        c.close()


@pytest.mark.parametrize("ct", ["bf16", "i8"])
def test_offsets_beyond_32_bits(gpu, ct):
    """A cache of more than 4 GiB: append, read, attention and eviction at its
    far end."""
    import torch

    log(f"far offsets {ct}")
    dim, page, hk = 256, 64, 2
    elem = 1 if ct == "i8" else 2
    pages = (5 << 30) // (dim * page * hk * elem)
    k = torch.empty((pages, hk, page, dim), dtype=_types(torch)[ct], device="cuda")
    v = torch.empty_like(k)
    ks = vs = None
    if ct == "i8":
        ks, vs = (torch.empty((pages, hk, page), device="cuda") for _ in range(2))
    ctx = gpu.dq_kv_init(1, 4, hk, dim, pages, page, 3, gpu.DQ_BF16, _code(gpu, ct), True)
    try:
        table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device="cuda")
        n, cap = 150, 3 * page
        g = torch.Generator().manual_seed(1)
        kn, vn = (torch.randn((n, hk, dim), generator=g).bfloat16() for _ in range(2))
        q = torch.randn((1, 4, dim), generator=g).bfloat16()
        idx = torch.arange(n, dtype=torch.int32, device="cuda")
        seq = torch.zeros_like(idx)
        gpu.dq_kv_append(ctx, kn.cuda(), vn.cuda(), idx, table, k, v, ks, vs, seq_ids=seq)
        ko, vo = (torch.empty((n, hk, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        gpu.dq_kv_read(ctx, idx, table, k, v, ks, vs, ko, vo, seq_ids=seq)
        bound = 2.0 ** -8 + (0.5 / 127 if ct == "i8" else 0)
        for back, x in ((ko, kn), (vo, vn)):
            err = (back.cpu().double() - x.double()).abs()
            assert float((err / x.double().abs().amax(-1, keepdim=True)).max()) <= bound * (1 + 2.0 ** -8)
        out = torch.empty((1, 4, dim), dtype=torch.bfloat16, device="cuda")
        sc = torch.zeros((1, hk, cap), device="cuda")
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        gpu.dq_kv_attend(ctx, q.cuda(), lens, table, k, v, ks, vs, out, dim ** -0.5, scores=sc, scores_out=sc)
        for h in range(4):
            s = ko[:, h // 2].cpu().double() @ q[0, h].double() * dim ** -0.5
            w = torch.softmax(s, 0) @ vo[:, h // 2].cpu().double()
            # read rows are rounded to bf16 once more than the cache's int8 values
            assert float((out[0, h].cpu().double() - w).abs().max()) <= 0.02
        assert torch.allclose(sc[0].sum(-1).cpu(), torch.full((hk,), 2.0), atol=1e-4)
        order = torch.arange(cap, dtype=torch.int32, device="cuda").expand(1, hk, cap).contiguous()
        so, oo, lo = torch.zeros_like(sc), torch.zeros_like(order), torch.zeros_like(lens)
        gpu.dq_kv_evict(ctx, 100, lens, lens - 1, sc, order, table, k, v, ks, vs, so, oo, lo, recent=20, sinks=2)
        gpu.dq_kv_read(ctx, idx[:100], table, k, v, ks, vs, ko[:100], vo[:100], seq_ids=seq[:100])
        torch.cuda.synchronize()
        assert int(lo) == 100 and gpu.dq_kv_take_errors(ctx) == 0
        for h in range(hk):
            src = O.evict_source(sc[0, h, :n].cpu().numpy(), np.arange(n), n, 100, n - 1, 20, 2)
            assert oo[0, h, :100].tolist() == src
            err = (vo[:100, h].cpu().double() - vn[src, h].double()).abs()
            assert float((err / vn[src, h].double().abs().amax(-1, keepdim=True)).max()) <= bound * (1 + 2.0 ** -8)
    finally:
        gpu.dq_kv_release(ctx)


# ---------------------------------------------------------------- eviction

def _evict(gpu, lens, budget, recent=0, sinks=0, ct="bf16", hk=2, dim=32, page=8, seed=0, in_place=False, ties=False,
           weights=None):
    import torch

    r = np.random.default_rng(seed)
    batch = len(lens)
    c = Case(gpu, batch, hk, 1, dim, page, lens, "bf16", ct, seed=seed)
    try:
        scores = r.random((batch, hk, c.cap)).astype(np.float32) ** 4
        if ties:
            scores = np.round(scores * 4) / 4
        if weights is not None:
            weights(scores)
        order = np.argsort(r.random((batch, hk, c.cap)), -1).astype(np.int32) * 2
        newest = np.array([2 * n - 2 for n in lens], np.int32)
        old = [None if t is None else t.clone().cpu() for t in c.cache()]
        s, o, n = torch.from_numpy(scores).cuda(), torch.from_numpy(order).cuda(), c.dev["lens"].clone()
        so = s if in_place else torch.full_like(s, 7.0)
        oo = o if in_place else torch.full_like(o, 7)
        no = n if in_place else torch.full_like(n, 7)
        gpu.dq_kv_evict(c.ctx, budget, n, torch.from_numpy(newest).cuda(), s, o, *c.cache(), so, oo, no,
                        recent=recent, sinks=sinks)
        torch.cuda.synchronize()
        assert gpu.dq_kv_take_errors(c.ctx) == 0
        so, oo = so.cpu().numpy(), oo.cpu().numpy()
        assert no.tolist() == [min(x, budget) for x in lens]
        bits = lambda t: t.view(torch.int8).reshape(t.shape[:3] + (-1,)) if t.dim() == 4 else t.view(torch.int32)  # noqa
        new = [None if t is None else bits(t.cpu()) for t in c.cache()[1:]]
        was = [None if t is None else bits(t) for t in old[1:]]
        want = [None if t is None else t.clone() for t in was]
        for b, m in enumerate(lens):
            for h in range(hk):
                src = O.evict_source(scores[b, h], order[b, h], m, budget, newest[b], recent, sinks)
                k = len(src)
                assert np.array_equal(so[b, h, :k], scores[b, h, src], equal_nan=True)
                assert np.array_equal(oo[b, h, :k], order[b, h, src])
                rest_s, rest_o = (scores[b, h, k:], order[b, h, k:]) if in_place else (7.0, 7)
                assert np.array_equal(so[b, h, k:], np.broadcast_to(rest_s, so[b, h, k:].shape), equal_nan=True)
                assert np.array_equal(oo[b, h, k:], np.broadcast_to(rest_o, oo[b, h, k:].shape))
                for j, f in enumerate(src):
                    if j != f:
                        (pj, sj), (pf, sf) = O.place(c.table, b, j, page), O.place(c.table, b, f, page)
                        for x, y in zip(want, was):
                            if x is not None:
                                x[pj, h, sj] = y[pf, h, sf]
        for x, y in zip(new, want):
            assert x is None or torch.equal(x, y)
    finally:
        c.close()


@pytest.mark.parametrize("ct", ["bf16", "f16", "i8"])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(gpu, ct, in_place):
    log(f"evict {ct} in place:{in_place}")
    _evict(gpu, [65, 64, 3, 0, 130, 63], 64, recent=9, sinks=4, ct=ct, seed=1, in_place=in_place)


@pytest.mark.parametrize("lens,budget,recent,sinks", [
    ([1, 2, 3], 1, 0, 0), ([40], 39, 0, 0), ([40], 40, 5, 5), ([200, 90], 10, 100, 0),   # more protected than fit
    ([1100, 1024, 1025], 1024, 128, 4), ([3000], 1500, 0, 1), ([2500, 5], 7, 3, 2), ([4097, 4096], 2000, 64, 4),
    ([8200, 8191, 7000], 4000, 100, 0), ([9001, 2], 8999, 1, 1)])
@pytest.mark.parametrize("ties", [False, True])
def test_evict_lengths(gpu, lens, budget, recent, sinks, ties):
    log(f"evict {lens} -> {budget} recent {recent} sinks {sinks} ties {ties}")
    _evict(gpu, lens, budget, recent, sinks, dim=16, page=24, seed=len(lens) + budget, ties=ties)


def test_evict_odd_weights(gpu):
    """Equal weights, zeros of both signs, infinities and NaN."""
    log("evict odd weights")

    def same(s):
        s[:] = 0.25

    def odd(s):
        r = np.random.default_rng(3)
        s[:] = r.choice([0.0, -0.0, np.inf, -np.inf, np.nan, -np.nan, 1e-45, -3.0, 2.0], s.shape)

    _evict(gpu, [300, 257], 128, 10, 4, weights=same, seed=2)
    _evict(gpu, [300, 257], 128, 10, 4, weights=odd, seed=3)
    _evict(gpu, [300, 257], 200, 0, 0, weights=odd, seed=4, in_place=True)


def test_evict_long(gpu):
    log("evict long")
    _evict(gpu, [33000, 9000], 2048, 512, 4, ct="i8", hk=1, dim=16, page=32, seed=5)


@pytest.mark.parametrize("n", [2, 65, 1025, 9000, 40001])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_one_token_over(gpu, n, in_place):
    """The least weight leaves wherever it is: first, last, in the middle, of
    several equal ones the last; and none but the protected are left."""
    log(f"evict one of {n} in place:{in_place}")

    def least(at):
        def put(s):
            s[:] = s + 0.5
            s[..., at] = 0.125
        return put

    for at in ([0], [n - 1], [n // 2], [n // 3, n // 2], [0, n - 1]):
        _evict(gpu, [n, n - 1], n - 1, 0, 0, dim=16, page=32, hk=1, seed=n, weights=least(at), in_place=in_place)
    _evict(gpu, [n], n - 1, n // 2, 1, ct="i8", dim=16, page=32, hk=1, seed=n, in_place=in_place)
    _evict(gpu, [n], n - 1, 2 * n, 0, ct="i8", dim=16, page=32, hk=1, seed=n, in_place=in_place)


def test_evict_long_ties(gpu):
    """Beyond what the registers hold, with equal weights among those that
    decide and weights of one magnitude."""
    log("evict long, ties")

    def same(s):
        s[:] = 0.25

    def near(s):
        s[:] = 1.0 + s / 64

    _evict(gpu, [34000], 3000, 100, 4, ct="f16", hk=1, dim=16, page=32, seed=6, ties=True, in_place=True)
    _evict(gpu, [33000, 20000], 9000, 100, 4, ct="f16", hk=1, dim=16, page=32, seed=7, weights=same)
    _evict(gpu, [33000, 20000], 9000, 100, 4, ct="f16", hk=1, dim=16, page=32, seed=8, weights=near)


def test_evict_places_that_do_not_exist(gpu):
    """A bad page is not followed (its rows stay), a length out of range is cut
    to what a sequence can hold, and both are counted."""
    import torch

    log("evict bad places")
    c = Case(gpu, 2, 1, 1, 32, 8, [40, 40], "bf16", "bf16", seed=1)
    try:
        old = c.dev["v"].clone()
        s = torch.arange(c.cap, dtype=torch.float32, device="cuda").expand(2, 1, c.cap).contiguous()
        o = torch.zeros((2, 1, c.cap), dtype=torch.int32, device="cuda")
        c.dev["table"][0, 4] = 10 ** 6
        n = torch.tensor([40, -2], dtype=torch.int32, device="cuda")
        out = torch.empty_like(n)
        gpu.dq_kv_evict(c.ctx, 8, n, n, s, o, *c.cache(), s, o, out)
        torch.cuda.synchronize()
        assert out.tolist() == [8, 0] and gpu.dq_kv_take_errors(c.ctx) > 0
        assert torch.equal(old.view(torch.int16), c.dev["v"].view(torch.int16))
        assert s[0, 0, :8].tolist() == [32.0 + i for i in range(8)]
    finally:
        c.close()


# ------------------------------------------------------------ graph capture

def test_decoding_step_replays(gpu):
    """Append, attention with gathered weights and eviction captured once and
    replayed, with eager calls between: every replay equals the eager result."""
    import torch

    log("graph decoding step")
    c = Case(gpu, 3, 2, 2, 64, 16, [520, 33, 129], "bf16", "i8", seed=9, scores=True)
    rope = gpu.dq_rope_init(64, 64, [i % 3 for i in range(32)], [0.8 ** i for i in range(32)])
    try:
        dev = c.dev
        r = np.random.default_rng(2)
        qkv = torch.empty((3, 8, 64), dtype=torch.bfloat16, device="cuda")
        pos = torch.empty((3, 3), dtype=torch.int32, device="cuda")
        index = dev["lens"] - 1
        q_out = torch.empty((3, 4, 64), dtype=torch.bfloat16, device="cuda")
        order = torch.arange(c.cap, dtype=torch.int32, device="cuda").expand(3, 2, c.cap).contiguous()
        outs = [q_out, torch.empty_like(q_out), torch.empty((3, 4), device="cuda"), torch.zeros((3, 2, c.cap), device="cuda"),
                torch.zeros((3, 2, c.cap), device="cuda"), torch.zeros_like(order), torch.zeros_like(dev["lens"])]
        start = [t.clone() for t in c.cache()[1:]]

        def run():
            gpu.dq_kv_append(c.ctx, qkv[:, 4:6], qkv[:, 6:], index, *c.cache(), q=qkv[:, :4], q_out=q_out, rope=rope,
                             positions=pos)
            gpu.dq_kv_attend(c.ctx, q_out, dev["lens"], *c.cache(), outs[1], c.sm, lse=outs[2], scores=dev["scores"],
                             scores_out=outs[3], decay=0.5)
            gpu.dq_kv_evict(c.ctx, 100, dev["lens"], index, outs[3], order, *c.cache(), outs[4], outs[5], outs[6],
                            recent=10, sinks=2)

        sets = [(torch.from_numpy(r.normal(0, 1, qkv.shape).astype(np.float32)).bfloat16().cuda(),
                 torch.from_numpy(r.integers(0, 5000, (3, 3)).astype(np.int32)).cuda()) for _ in range(3)]

        def load(i):
            for o in outs:
                o.zero_()
            for t, s in zip(c.cache()[1:], start):
                t.copy_(s)
            qkv.copy_(sets[i][0])
            pos.copy_(sets[i][1])

        def result():
            torch.cuda.synchronize()
            return [t.clone().view(torch.uint8) for t in outs + list(c.cache()[1:])]

        eager = []
        for i in range(3):
            load(i)
            run()
            eager.append(result())
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        torch.cuda.synchronize()
        for _ in range(2):
            for i in range(3):
                load(i)
                g.replay()
                for a, b in zip(result(), eager[i]):
                    assert torch.equal(a, b)
                load(i)
                run()
                for a, b in zip(result(), eager[i]):
                    assert torch.equal(a, b)
        assert gpu.dq_kv_take_errors(c.ctx) == 0
    finally:
        gpu.dq_rope_release(rope)
        c.close()
