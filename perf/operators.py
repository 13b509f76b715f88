"""The operators of autoregressive decoding over a paged key-value cache, as
they are measured: rotary positions with several axes, the append of new keys
and values to the cache (rotated, and quantized per row for an int8 cache),
the attention of one new token over the cache, and the eviction of the tokens
that gathered the least attention.

Shapes. B sequences, Hq query heads, Hk key-value heads (Hq a multiple of
Hk), head size D. The cache is [pages, Hk, page_size, D]; token t of sequence
b lies in page block_table[b, t // page_size] at slot t % page_size. An int8
cache has one fp32 scale for every row of D codes, [pages, Hk, page_size].

  rotary    pair i of a token turns by pos[axis(i)] * inv_freq[i]
            (a, b) -> (a cos - b sin, b cos + a sin); the gradient's pass
            turns by the opposite angle
  append    k rotated, v as it is; int8: scale = max|row| / 127 (1 for a row
            of zeros), code = clamp(rne(row / scale), -127, 127)
  attention s_t = sm_scale * q . k_t for the tokens t in [len - window, len),
            p = softmax(s), out = sum_t p_t v_t, lse = log sum_t exp(s_t);
            no token: out = 0, lse = -inf. Weight gathered by a token:
            scores' = decay * scores + sum of p_t over its key-value head's
            query heads
  eviction  of len > budget tokens the first `sinks` and the last `recent`
            (by their running number) stay, then those with the largest
            weights, ties to the lowest slot; the tokens kept at slots from
            budget on move, in order, into the slots freed below it
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "i8": torch.int8}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2, "i8": 1}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of a small batch: the launch itself counts
        dict(name="rope_step", op="rope", tokens=4, heads=10, head_dim=64, rotary_dim=64, axes=1,
             spread=False, interleaved=False, inverse=False, type="f16", fused=True),
        # the queries and keys of a clip's frames, read out of a fused projection
        dict(name="rope_video", op="rope", tokens=8205, heads=40, head_dim=128, rotary_dim=128, axes=3,
             spread=False, interleaved=False, inverse=False, type="bf16", fused=True),
        # the gradient's pass of a partial rotation of neighbouring pairs, in fp32
        dict(name="rope_grad", op="rope", tokens=4099, heads=16, head_dim=80, rotary_dim=64, axes=3,
             spread=True, interleaved=True, inverse=True, type="f32", fused=False),
        # one new token of every sequence in a serving batch, quantized as it is stored
        dict(name="append_step_i8", op="append", batch=32, tokens=32, q_heads=32, kv_heads=8,
             head_dim=128, axes=3, page_size=16, pages_per_seq=64, type="bf16", cache="i8"),
        # a chunk of prompts of several sequences
        dict(name="append_prompt", op="append", batch=3, tokens=6001, q_heads=32, kv_heads=8,
             head_dim=128, axes=1, page_size=64, pages_per_seq=64, type="bf16", cache="bf16"),
        # one short sequence: latency
        dict(name="attend_short", op="attend", batch=1, q_heads=8, kv_heads=2, head_dim=64, max_len=37,
             page_size=16, ragged=False, window=0, scores=False, type="f16", cache="f16"),
        # an ordinary serving batch, sequences of different lengths
        dict(name="attend_batch", op="attend", batch=32, q_heads=32, kv_heads=8, head_dim=128,
             max_len=4096, page_size=16, ragged=True, window=0, scores=False, type="bf16",
             cache="bf16"),
        # one long document, a page size that a length ends inside
        dict(name="attend_long", op="attend", batch=1, q_heads=32, kv_heads=4, head_dim=128,
             max_len=131071, page_size=64, ragged=False, window=0, scores=False, type="bf16",
             cache="bf16"),
        # a full int8 cache whose weights are gathered for the eviction: the largest
        dict(name="attend_i8_scores", op="attend", batch=48, q_heads=32, kv_heads=8, head_dim=128,
             max_len=20479, page_size=32, ragged=True, window=0, scores=True, type="bf16",
             cache="i8"),
        # heads of their own, a sliding window, an odd head size, fp32 queries on an int8 cache
        dict(name="attend_window_f32", op="attend", batch=9, q_heads=12, kv_heads=12, head_dim=96,
             max_len=5003, page_size=24, ragged=True, window=1000, scores=True, type="f32", cache="i8"),
        # one token over the budget in every sequence: the steady state of decoding
        dict(name="evict_step", op="evict", batch=16, kv_heads=8, head_dim=128, max_len=1025, budget=1024,
             recent=128, sinks=4, page_size=16, ragged=False, cache="i8"),
        # long prompts cut down to the budget at once
        dict(name="evict_prompt", op="evict", batch=8, kv_heads=8, head_dim=128, max_len=32768, budget=2048,
             recent=512, sinks=4, page_size=32, ragged=True, cache="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "evict"])
    if op == "rope":
        d = rng.choice([32, 64, 80, 96, 128, 192, 256])
        heads = _log(rng, 1, 48)
        return dict(op=op, tokens=_log(rng, 1, min(16000, int(1e8 / (heads * d)))), heads=heads, head_dim=d,
                    rotary_dim=rng.choice([d, d // 2]), axes=rng.choice([1, 2, 3]),
                    spread=rng.random() < 0.5, interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5,
                    type=rng.choice(["bf16", "f16", "f32"]), fused=rng.random() < 0.5)
    kv = rng.choice([1, 2, 4, 5, 8])
    d = rng.choice([32, 64, 80, 96, 128, 192, 256])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    if op == "append":
        batch = _log(rng, 1, 64)
        hq = kv * rng.choice([1, 2, 4, 7, 8])
        tokens = batch if rng.random() < 0.5 else max(batch, _log(rng, 1, min(8000, int(6e7 / (2 * (hq + kv) * d)))))
        # int8 rows are handed back as the values they stand for, in the query's 16-bit type
        types = rng.choice([("bf16", "i8"), ("f16", "i8"), ("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16")])
        return dict(op=op, batch=batch, tokens=tokens, q_heads=hq, kv_heads=kv,
                    head_dim=d, axes=rng.choice([1, 3]), page_size=page,
                    pages_per_seq=-(-tokens // batch) // page + rng.randint(1, 16), type=types[0], cache=types[1])
    if op == "attend":
        batch = _log(rng, 1, 64)
        most = min(150000, int(3e8 / (batch * kv * d)))
        length = _log(rng, 1, most)
        types = rng.choice([("bf16", "bf16"), ("f16", "f16"), ("bf16", "i8"), ("f16", "i8"), ("f32", "i8"),
                            ("f32", "bf16"), ("f32", "f16")])
        return dict(op=op, batch=batch, q_heads=kv * rng.choice([1, 2, 4, 5, 8, 16]), kv_heads=kv, head_dim=d,
                    max_len=length, page_size=page, ragged=rng.random() < 0.7,
                    window=rng.choice([0, 0, 0, 1 + length // 3]), scores=rng.random() < 0.4,
                    type=types[0], cache=types[1])
    batch = _log(rng, 1, 32)
    length = _log(rng, 32, min(100000, int(3e8 / (batch * kv * d))))
    budget = max(8, int(length * rng.choice([0.05, 0.25, 0.5, 0.98])))
    return dict(op=op, batch=batch, kv_heads=kv, head_dim=d, max_len=length, budget=budget,
                recent=budget // rng.choice([2, 8, 100]), sinks=rng.choice([0, 4]), page_size=page,
                ragged=rng.random() < 0.5, cache=rng.choice(["bf16", "f16", "i8"]))


# ------------------------------------------------------------------ inputs

def _axis_of_pair(case):
    """The position axis of each pair: in turn, or in blocks of which the
    first axis has the larger rest (16, 24, 24 for 64 pairs on three axes)."""
    pairs, axes = case.get("rotary_dim", case["head_dim"]) // 2, case["axes"]
    if case.get("spread"):
        return [i % axes for i in range(pairs)]
    share = pairs * 3 // (4 * axes - 4) if axes > 1 else 0
    first = pairs - share * (axes - 1)
    return [0 if i < first else 1 + (i - first) // share for i in range(pairs)]


def _inv_freq(case):
    r = case.get("rotary_dim", case["head_dim"])
    return [10000.0 ** (-2.0 * i / r) for i in range(r // 2)]


def _positions(gen, axes, tokens, dev):
    """Running numbers on one axis; frames, rows and columns on several."""
    start = int(torch.randint(0, 50000, (1,), generator=gen, device=dev))
    n = torch.arange(tokens, device=dev)
    rows, cols = 18, 32
    grid = [n + start] if axes == 1 else [start + n // (rows * cols), start + n // cols % rows, start + n % cols]
    return torch.stack([g.to(torch.int32) for g in grid[:axes]])


def _lengths(case):
    """The lengths that the case's sequences have, in some order: the longest
    first, the others spread over [1/4, 1] of it, and an empty place in a
    ragged batch of 8 or more."""
    n, top = case["batch"], case["max_len"]
    if not case["ragged"]:
        return [top] * n
    spread = [max(1, round(top * (1 - 0.75 * (i * 0.6180339887498949 % 1.0)))) for i in range(n)]
    return spread[:-1] + [0] if n >= 8 else spread


def _randn(gen, shape, dtype, dev):
    return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)


def _cache(gen, case, pages, dev):
    """Keys with a few strong channels, values around zero; the block table
    puts the pages of a sequence in no order."""
    shape = (pages, case["kv_heads"], case["page_size"], case["head_dim"])
    s = {}
    for name in ("k", "v"):
        x = torch.randn(shape, generator=gen, device=dev)
        if name == "k":
            x[..., :: max(1, case["head_dim"] // 4)] += 1.5
        if case["cache"] == "i8":
            s[name + "_cache"] = (x * 40).round_().clamp_(-127, 127).to(torch.int8)
            s[name + "_scale"] = torch.rand(shape[:-1], generator=gen, device=dev) * 0.03 + 0.01
        else:
            s[name + "_cache"] = x.to(_TYPES[case["cache"]])
            s[name + "_scale"] = None
        del x
    s["block_table"] = torch.randperm(pages, generator=gen, device=dev).to(torch.int32).view(case["batch"], -1)
    return s


class _Handle:
    """A context of the library, released with the state that holds it."""

    def __init__(self, ctx, release):
        self.ctx, self.release = ctx, release

    def __del__(self):
        self.release(self.ctx)


def _kv_handle(case, scores=False):
    import dynamic_quantized_gemm_amd as dq

    types = {"f32": dq.DQ_F32, "bf16": dq.DQ_BF16, "f16": dq.DQ_F16, "i8": dq.DQ_I8}
    per_seq = _pages_per_seq(case)
    return _Handle(dq.dq_kv_init(case["batch"], case.get("q_heads", case["kv_heads"]), case["kv_heads"],
                                 case["head_dim"], case["batch"] * per_seq, case["page_size"], per_seq,
                                 types[case.get("type", "bf16")], types[case["cache"]], scores), dq.dq_kv_release)


def _rope_handle(case):
    import dynamic_quantized_gemm_amd as dq

    return _Handle(dq.dq_rope_init(case["head_dim"], case.get("rotary_dim", case["head_dim"]), _axis_of_pair(case),
                                   _inv_freq(case), case.get("interleaved", False)), dq.dq_rope_release)


def _pages_per_seq(case):
    return case["pages_per_seq"] if "pages_per_seq" in case else -(-case["max_len"] // case["page_size"])


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    state = {"case": case}
    if case["op"] in ("rope", "append"):
        # what a program computes once for its model
        state["inv_freq"] = torch.tensor(_inv_freq(case), dtype=torch.float64, device=dev)
        state["axis"] = torch.tensor(_axis_of_pair(case), device=dev)
        if own:
            state["rope"] = _rope_handle(case)
    if case["op"] == "rope":
        t, h, d = case["tokens"], case["heads"], case["head_dim"]
        more = max(1, h // 4) if case["fused"] else 0  # the value heads of a fused projection
        state["x"] = _randn(gen, (t, h + more, d), _TYPES[case["type"]], dev)[:, :h]
        state["positions"] = _positions(gen, case["axes"], t, dev)
        state["y"] = torch.empty((t, h, d), dtype=_TYPES[case["type"]], device=dev)
        return state
    if case["op"] == "append":
        b, t, hq, hk, d = (case[n] for n in ("batch", "tokens", "q_heads", "kv_heads", "head_dim"))
        qkv = _randn(gen, (t, hq + 2 * hk, d), _TYPES[case["type"]], dev)
        state["q"], state["k"], state["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        state["positions"] = _positions(gen, case["axes"], t, dev)
        state.update(_cache(gen, case, b * case["pages_per_seq"], dev))
        # the tokens of a sequence follow one another, behind what it holds
        n = torch.arange(t, device=dev)
        each = -(-t // b)
        room = case["pages_per_seq"] * case["page_size"] - each
        held = torch.randint(0, room + 1, (b,), generator=gen, device=dev)
        state["seq_ids"] = (n // each).to(torch.int32)
        state["index"] = (held[n // each] + n % each).to(torch.int32)
        state["q_out"] = torch.empty((t, hq, d), dtype=_TYPES[case["type"]], device=dev)
        for name in ("k_out", "v_out"):
            state[name] = torch.empty((t, hk, d), dtype=_TYPES[case["type"]], device=dev)
        if own:
            state["kv"] = _kv_handle(case)
        return state
    b, hk, per_seq = case["batch"], case["kv_heads"], _pages_per_seq(case)
    cap = per_seq * case["page_size"]
    state.update(_cache(gen, case, b * per_seq, dev))
    order = torch.randperm(b, generator=gen, device=dev)
    state["lens"] = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)[order]
    if case["op"] == "attend":
        hq, d = case["q_heads"], case["head_dim"]
        state["q"] = _randn(gen, (b, hq, d), torch.float32, dev).mul_(1.5).to(_TYPES[case["type"]])
        state["out"] = torch.empty((b, hq, d), dtype=_TYPES[case["type"]], device=dev)
        state["lse"] = torch.empty((b, hq), dtype=torch.float32, device=dev)
        if case["scores"]:
            state["scores"] = torch.rand((b, hk, cap), generator=gen, device=dev)
            state["scores_out"] = torch.zeros((b, hk, cap), device=dev)
        if own:
            state["kv"] = _kv_handle(case, case["scores"])
        return state
    # a few tokens gather most of the attention; after earlier evictions the
    # running numbers of the slots are in no order and have gaps
    state["scores"] = torch.rand((b, hk, cap), generator=gen, device=dev).pow_(8).mul_(20)
    number = torch.rand((b, hk, cap), generator=gen, device=dev)
    number.masked_fill_(torch.arange(cap, device=dev) >= state["lens"][:, None, None], 2.0)
    state["order"] = number.argsort(-1).argsort(-1).to(torch.int32) * 2
    state["newest"] = (state["lens"] - 1) * 2
    state["scores_out"] = torch.zeros((b, hk, cap), device=dev)
    state["order_out"] = torch.zeros((b, hk, cap), dtype=torch.int32, device=dev)
    state["lens_out"] = torch.zeros((b,), dtype=torch.int32, device=dev)
    if own:
        state["kv"] = _kv_handle(case)
    return state


# ------------------------------------------------------------- plain forms

def _rotate(state, x, inverse=False):
    """x [tokens, heads, D] in fp32, angles in fp64."""
    case = state["case"]
    r = case.get("rotary_dim", case["head_dim"])
    angle = state["positions"].double()[state["axis"]].T * state["inv_freq"]
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    s = -s if inverse else s
    if case.get("interleaved"):
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., : r // 2], x[..., r // 2: r]
        turned = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((turned, x[..., r:]), -1)


def _plain_rope(state):
    x = state["x"]
    return _rotate(state, x.float(), state["case"]["inverse"]).to(x.dtype)


def _plain_append(state):
    case = state["case"]
    q, k, v = state["q"], state["k"], state["v"]
    q_out = _rotate(state, q.float()).to(q.dtype)
    index, size = state["index"].long(), case["page_size"]
    page, slot = state["block_table"][state["seq_ids"].long(), index // size].long(), index % size
    back = {"q": q_out}
    for name, rows in (("k", _rotate(state, k.float())), ("v", v.float())):
        cache, scale = state[name + "_cache"], state[name + "_scale"]
        if scale is None:
            cache[page, :, slot] = rows.to(cache.dtype)
            back[name + "_cache"] = cache
        else:
            step = rows.abs().amax(-1) / 127
            step = torch.where(step > 0, step, torch.ones_like(step))
            cache[page, :, slot] = (rows / step[..., None]).round().clamp(-127, 127).to(torch.int8)
            scale[page, :, slot] = step
            back[name + "_scale"] = scale
            back[name + "_rows"] = (cache[page, :, slot].float() * scale[page, :, slot][..., None]).to(q.dtype)
    return back


def _gathered(state, name):
    """The keys or values of every sequence, [B, Hk, capacity, D] in fp32."""
    case, table = state["case"], state["block_table"].long()
    shape = (case["batch"], case["kv_heads"], -1, case["head_dim"])
    x = state[name + "_cache"][table].permute(0, 2, 1, 3, 4).reshape(shape).float()
    if state[name + "_scale"] is not None:
        x *= state[name + "_scale"][table].permute(0, 2, 1, 3).reshape(shape[:3] + (1,))
    return x


def _plain_attend(state):
    case, q, lens = state["case"], state["q"], state["lens"]
    b, hq, hk, d = (case[n] for n in ("batch", "q_heads", "kv_heads", "head_dim"))
    s = torch.matmul(q.float().view(b, hk, hq // hk, d), _gathered(state, "k").transpose(-1, -2)) * d ** -0.5
    t = torch.arange(s.shape[-1], device=s.device)
    end = lens[:, None, None, None]
    seen = (t < end) & (t >= end - case["window"]) if case["window"] else t < end
    s = s.masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True).clamp_min(-3e38)
    e = (s - top).exp()
    total = e.sum(-1, keepdim=True)
    p = e / total.clamp_min(1e-30)
    out = torch.matmul(p, _gathered(state, "v")).view(b, hq, d).to(q.dtype)
    back = {"out": out, "lse": (total.log() + top).view(b, hq)}
    back["lse"] = torch.where(lens[:, None] > 0, back["lse"], -math.inf)
    if case["scores"]:
        gathered = state["scores"] * 0.95 + p.sum(2)
        back["scores"] = torch.where(t < lens[:, None, None], gathered, state["scores_out"])
    return back


def _plain_evict(state):
    case, lens = state["case"], state["lens"]
    budget, size = case["budget"], case["page_size"]
    scores, order = state["scores"], state["order"]
    slot = torch.arange(scores.shape[-1], device=scores.device)
    held = slot < lens[:, None, None]
    safe = (order < case["sinks"]) | (order > state["newest"][:, None, None] - case["recent"])
    key = torch.where(safe, math.inf, scores).masked_fill(~held, -math.inf)
    rank = key.argsort(dim=-1, descending=True, stable=True).argsort(dim=-1)
    kept = held & (rank < budget)
    n = min(budget, scores.shape[-1])
    movers = (~(kept & (slot >= budget))).byte().argsort(dim=-1, stable=True)
    hole = ~kept[..., :n] & held[..., :n]
    which = (hole.long().cumsum(-1) - 1).clamp_min(0)
    src = torch.where(hole, movers.gather(-1, which), slot[:n])
    new_lens = lens.clamp_max(budget)
    live = slot[:n] < new_lens[:, None, None]
    back = {"lens": new_lens}
    for name, x in (("scores", scores), ("order", order)):
        into = state[name + "_out"]
        into[..., :n] = torch.where(live, x.gather(-1, src), into[..., :n])
        back[name] = into
    table = state["block_table"].long()
    seq = torch.arange(case["batch"], device=slot.device)[:, None, None]
    head = torch.arange(case["kv_heads"], device=slot.device)[None, :, None]
    to = (table[seq, slot[:n] // size].expand(src.shape), head.expand(src.shape), (slot[:n] % size).expand(src.shape))
    at = (table[seq, src // size], head.expand(src.shape), src % size)
    for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
        if state[name] is not None:
            state[name][to] = state[name][at]
            back[name] = state[name]
    return back


# ----------------------------------------------------- the framework's form

def _own_rope(state):
    import dynamic_quantized_gemm_amd as dq

    dq.dq_rope_forward(state["rope"].ctx, state["x"], state["positions"], state["y"], inverse=state["case"]["inverse"])
    return state["y"]


def _own_append(state):
    import dynamic_quantized_gemm_amd as dq

    s = state
    cache = (s["block_table"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    dq.dq_kv_append(s["kv"].ctx, s["k"], s["v"], s["index"], *cache, seq_ids=s["seq_ids"], q=s["q"], q_out=s["q_out"],
                    rope=s["rope"].ctx, positions=s["positions"])
    back = {"q": s["q_out"]}
    if s["k_scale"] is None:
        return {**back, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    dq.dq_kv_read(s["kv"].ctx, s["index"], *cache, s["k_out"], s["v_out"], seq_ids=s["seq_ids"])
    return {**back, "k_scale": s["k_scale"], "v_scale": s["v_scale"], "k_rows": s["k_out"], "v_rows": s["v_out"]}


def _own_attend(state):
    import dynamic_quantized_gemm_amd as dq

    s, case = state, state["case"]
    more = dict(scores=s["scores"], scores_out=s["scores_out"], decay=0.95) if case["scores"] else {}
    dq.dq_kv_attend(s["kv"].ctx, s["q"], s["lens"], s["block_table"], s["k_cache"], s["v_cache"], s["k_scale"],
                    s["v_scale"], s["out"], case["head_dim"] ** -0.5, lse=s["lse"], window=case["window"], **more)
    back = {"out": s["out"], "lse": s["lse"]}
    return {**back, "scores": s["scores_out"]} if case["scores"] else back


def _own_evict(state):
    import dynamic_quantized_gemm_amd as dq

    s, case = state, state["case"]
    dq.dq_kv_evict(s["kv"].ctx, case["budget"], s["lens"], s["newest"], s["scores"], s["order"], s["block_table"],
                   s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["scores_out"], s["order_out"],
                   s["lens_out"], recent=case["recent"], sinks=case["sinks"])
    back = {"lens": s["lens_out"], "scores": s["scores_out"], "order": s["order_out"]}
    return {**back, **{n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale") if s[n] is not None}}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "append": _own_append, "attend": _own_attend, "evict": _own_evict}[op](state)
    return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend, "evict": _plain_evict}[op](state)


# -------------------------------------------------------------------- work

def work(case):
    op, d = case["op"], case["head_dim"]
    if op == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * d * _BYTES[case["type"]] + 4 * case["axes"] * case["tokens"],
                "flops": 3 * n * case["rotary_dim"]}
    row = d * _BYTES[case["cache"]] + (4 if case["cache"] == "i8" else 0)  # one key or value in the cache
    if op == "append":
        t, hq, hk = case["tokens"], case["q_heads"], case["kv_heads"]
        moved = t * (2 * hq + 2 * hk) * d * _BYTES[case["type"]] + t * 2 * hk * row + 4 * t * (case["axes"] + 2)
        if case["cache"] == "i8":  # the rows handed back as values
            moved += t * 2 * hk * (row + d * _BYTES[case["type"]])
        return {"bytes": moved, "flops": t * (3 * (hq + hk) * d + (4 * hk * d if case["cache"] == "i8" else 0))}
    if op == "attend":
        hq, hk = case["q_heads"], case["kv_heads"]
        lens = _lengths(case)
        seen = sum(min(n, case["window"]) if case["window"] else n for n in lens)
        moved = 2 * seen * hk * row + case["batch"] * hq * (2 * d * _BYTES[case["type"]] + 4)
        moved += 4 * case["batch"] * (1 + _pages_per_seq(case))
        if case["scores"]:
            moved += 8 * hk * sum(lens)
        return {"bytes": moved, "flops": 4 * seen * hq * d}
    hk, budget = case["kv_heads"], case["budget"]
    lens = _lengths(case)
    kept = sum(min(n, budget) for n in lens)
    # a token over the budget moves if it is kept: with the numbers in no order, budget of n are
    moves = sum((n - budget) * budget / n for n in lens if n > budget)
    return {"bytes": hk * (8 * sum(lens) + 8 * kept + 4 * row * moves), "flops": hk * sum(lens)}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    state = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attend": _exact_attend, "evict": _exact_evict}[case["op"]](
        case, state)


def _turned(case, state, x, sign):
    """Pairs as complex numbers times exp(i angle), in fp64, axis by axis."""
    x = x.double().clone()
    r = case.get("rotary_dim", case["head_dim"])
    angle = torch.zeros((x.shape[0], r // 2), dtype=torch.float64, device=x.device)
    for i, (axis, f) in enumerate(zip(_axis_of_pair(case), _inv_freq(case))):
        angle[:, i] = state["positions"][axis].double() * f
    unit = torch.polar(torch.ones_like(angle), sign * angle)[:, None]
    lo, hi = (slice(0, r, 2), slice(1, r, 2)) if case.get("interleaved") else (slice(0, r // 2), slice(r // 2, r))
    z = torch.complex(x[..., lo], x[..., hi]) * unit
    x[..., lo], x[..., hi] = z.real, z.imag
    return x


def _exact_rope(case, state):
    return _turned(case, state, state["x"], -1.0 if case["inverse"] else 1.0)


def _exact_append(case, state):
    back = {"q": _turned(case, state, state["q"], 1.0)}
    for name, rows in (("k", _turned(case, state, state["k"], 1.0)), ("v", state["v"].double())):
        held, scale = state[name + "_cache"], state[name + "_scale"]
        size, table = case["page_size"], state["block_table"].tolist()
        index = state["index"].tolist()
        at = torch.tensor([table[b][i // size] * size + i % size for b, i in zip(state["seq_ids"].tolist(), index)],
                          device=held.device)
        if scale is None:
            flat = held.double().transpose(1, 2).flatten(0, 1)  # [pages * page_size, Hk, D]
            flat[at] = rows
            back[name + "_cache"] = flat.unflatten(0, (-1, size)).transpose(1, 2)
            continue
        step = rows.abs().max(-1).values / 127.0
        step[step == 0] = 1.0
        flat = scale.double().transpose(1, 2).flatten(0, 1)
        flat[at] = step
        back[name + "_scale"] = flat.unflatten(0, (-1, size)).transpose(1, 2)
        back[name + "_rows"] = torch.round(rows / step[..., None]) * step[..., None]
    return back


def _exact_attend(case, state):
    hq, hk, d, size = case["q_heads"], case["kv_heads"], case["head_dim"], case["page_size"]
    out = torch.zeros((case["batch"], hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((case["batch"], hq), -math.inf, dtype=torch.float64, device="cuda")
    scores = state["scores_out"].double() if case["scores"] else None
    for b, n in enumerate(state["lens"].tolist()):
        if n == 0:
            continue
        pages = state["block_table"][b, : -(-n // size)].long()
        first = max(0, n - case["window"]) if case["window"] else 0
        rows = []
        for name in ("k", "v"):
            x = state[name + "_cache"][pages].double()
            if state[name + "_scale"] is not None:
                x = x * state[name + "_scale"][pages].double()[..., None]
            rows.append(x.transpose(0, 1).flatten(1, 2)[:, first:n])  # [Hk, tokens, D]
        for h in range(hk):
            q = state["q"][b, h * (hq // hk):(h + 1) * (hq // hk)].double()
            s = q @ rows[0][h].T.contiguous() / math.sqrt(d)
            at = slice(h * (hq // hk), (h + 1) * (hq // hk))
            lse[b, at] = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[b, at, None])
            out[b, at] = p @ rows[1][h].contiguous()
            if scores is not None:
                scores[b, h, :n] = 0.95 * state["scores"][b, h, :n].double()
                scores[b, h, first:n] += p.sum(0)
    return {"out": out, "lse": lse, "scores": scores} if case["scores"] else {"out": out, "lse": lse}


def _exact_evict(case, state):
    size, budget = case["page_size"], case["budget"]
    back = {n: state[n].clone() for n in ("k_cache", "v_cache", "k_scale", "v_scale") if state[n] is not None}
    for name in ("scores", "order"):
        back[name] = state[name + "_out"].clone()
    for b, n in enumerate(state["lens"].tolist()):
        pages = state["block_table"][b].long()
        for h in range(case["kv_heads"]):
            score, order = state["scores"][b, h, :n], state["order"][b, h, :n]
            if n > budget:
                safe = (order < case["sinks"]) | (order > int(state["newest"][b]) - case["recent"])
                weight = score.double().masked_fill(safe, math.inf)
                keep = torch.sort(weight, descending=True, stable=True).indices[:budget].sort().values
                stay, go = keep[keep < budget], keep[keep >= budget]
                free = torch.ones(budget, dtype=torch.bool, device=keep.device)
                free[stay] = False
                free = free.nonzero().view(-1)
                src = torch.arange(budget, device=keep.device)
                src[free] = go
                for x in ("k_cache", "v_cache", "k_scale", "v_scale"):
                    if x in back:
                        back[x][pages[free // size], h, free % size] = state[x][pages[go // size], h, go % size]
            else:
                src = torch.arange(n, device=score.device)
            back["scores"][b, h, : len(src)] = score[src]
            back["order"][b, h, : len(src)] = order[src]
    for x in ("scores", "k_cache", "v_cache", "k_scale", "v_scale"):
        if x in back and back[x].is_floating_point():
            back[x] = back[x].double()
    back["lens"] = state["lens"].clamp(max=budget)
    return back
