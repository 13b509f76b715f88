"""The operators of layers with 4-bit weights and of layers of experts, as they
are measured: products with 4-bit weights and group scales, the same grouped
by expert with any number of rows each, the router that sends tokens to
experts, and the sum of the experts' results.

Weights. Row n of an expert's W [rows, K] has a 4-bit code q for every k (two
in a byte, the even k in the low half) and, for every `group` values of k, a
scale s and a zero point z (4 bits, two in a byte; none: 8), so
W[n, k] = (q - z) s.

  product   y = x W^T + bias; gated: the rows of W are N of a gate and N of
            the values it gates, y = silu(x Wg^T + bg) (x Wu^T + bu),
            silu(v) = v / (1 + exp(-v))
  grouped   rows offsets[e] to offsets[e + 1] of y are products with expert
            e's weights; row r of y comes from row row_index[r] of x (or r)
  router    a token's top_k largest logits (ties: the lowest expert; an expert
            at -infinity is never chosen, its place holds -1 and weight 0),
            their weights by softmax over all experts or by sigmoid,
            normalised to sum to one or not; rows are the pairs (token,
            expert) in the order of the expert, then of the token:
            offsets[experts + 1], row_token[row], row_of[token, j]
  combine   out[t] = add[t] + sum_j weights[t, j] y[row_of[t, j]]
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one new token through a square projection: the launch itself counts
        dict(name="w4_token", op="w4", rows=1, n=4096, k=4096, group=128, type="bf16", scale="bf16", y="bf16",
             zeros=False, bias=False, gated=False),
        # one new token through a large layer in groups of 32 with zero points: the weights' way from memory
        dict(name="w4_token_large", op="w4", rows=1, n=16384, k=8192, group=32, type="f16", scale="f16", y="f16",
             zeros=True, bias=False, gated=False),
        # a few tokens of an fp32 program, sizes that fit no tile
        dict(name="w4_odd", op="w4", rows=7, n=1003, k=1111, group=64, type="f32", scale="f32", y="f32",
             zeros=True, bias=True, gated=False),
        # a serving batch through the first, gated half of a feed-forward layer
        dict(name="w4_batch_gated", op="w4", rows=48, n=8192, k=4096, group=128, type="bf16", scale="bf16", y="bf16",
             zeros=False, bias=False, gated=True),
        # a long prompt
        dict(name="w4_prompt", op="w4", rows=4096, n=4096, k=4096, group=128, type="bf16", scale="bf16", y="bf16",
             zeros=True, bias=False, gated=False),
        # one new token's eight experts of 64, gated
        dict(name="experts_token", op="grouped", tokens=1, top_k=8, experts=64, n=1024, k=2048, group=128, type="bf16",
             scale="bf16", y="bf16", zeros=False, bias=False, gated=True, gather=True),
        # a batch's second half of the experts' layers, fp32 for the sum that follows, a K that ends inside a block
        dict(name="experts_batch", op="grouped", tokens=64, top_k=4, experts=32, n=4096, k=1400, group=64, type="bf16",
             scale="f32", y="f32", zeros=True, bias=False, gated=False, gather=False),
        # a prompt's rows, shared out unevenly: the largest
        dict(name="experts_prompt", op="grouped", tokens=4096, top_k=4, experts=16, n=2048, k=4096, group=128,
             type="bf16", scale="bf16", y="bf16", zeros=False, bias=False, gated=True, gather=True),
        # the router of one step of a small batch
        dict(name="route_step", op="route", tokens=8, experts=64, top_k=6, type="f32", scoring="softmax",
             normalize=True, masked=False),
        # the router of a prompt over many experts, some switched off
        dict(name="route_prompt", op="route", tokens=16001, experts=256, top_k=8, type="bf16", scoring="sigmoid",
             normalize=True, masked=True),
        # the results of one step, added to the residual stream
        dict(name="combine_step", op="combine", tokens=8, experts=64, top_k=6, n=2048, y="bf16", out="bf16", add=True),
        # a prompt's
        dict(name="combine_prompt", op="combine", tokens=8101, experts=64, top_k=4, n=4096, y="f32", out="bf16",
             add=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _weights_kind(rng):
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    return dict(group=rng.choice([32, 64, 128, 256]), type=kind, scale=rng.choice([kind, "f32", "f16"]),
                y=rng.choice([kind, kind, "f32"]), zeros=rng.random() < 0.5, bias=rng.random() < 0.3,
                gated=rng.random() < 0.4)


def draw(rng):
    op = rng.choice(["w4", "w4", "grouped", "grouped", "route", "combine"])
    if op == "w4":
        kind = _weights_kind(rng)
        wide = 2 if kind["gated"] else 1
        k = _log(rng, 40, 16384)
        n = _log(rng, 24, min(16384, int(1.3e8 / (k * wide))))
        # at most the work of the largest; fp32 inputs cost three products
        most = 1.2e11 / (k * n * wide * (3 if kind["type"] == "f32" else 1))
        return dict(op=op, rows=_log(rng, 1, min(8192, most)), n=n, k=k, **kind)
    if op == "grouped":
        kind = _weights_kind(rng)
        wide = 2 if kind["gated"] else 1
        experts = _log(rng, 2, 128)
        k = _log(rng, 40, 4096)
        n = _log(rng, 24, min(4096, int(2.6e8 / (k * wide * experts))))
        top_k = rng.choice([t for t in (1, 2, 4, 6, 8) if t <= experts])
        most = 1.2e11 / (k * n * wide * top_k * (3 if kind["type"] == "f32" else 1))
        return dict(op=op, tokens=_log(rng, 1, min(8192 // top_k, most)), top_k=top_k, experts=experts, n=n, k=k,
                    gather=rng.random() < 0.6, **kind)
    experts = _log(rng, 2, 512)
    top_k = rng.randint(1, min(experts, 10))
    if op == "route":
        return dict(op=op, tokens=_log(rng, 1, min(16000, int(4e6 / experts))), experts=experts, top_k=top_k,
                    type=rng.choice(["f32", "f32", "bf16", "f16"]), scoring=rng.choice(["softmax", "softmax", "sigmoid"]),
                    normalize=rng.random() < 0.6, masked=rng.random() < 0.3)
    n = _log(rng, 24, 8192)
    return dict(op=op, tokens=_log(rng, 1, min(16000, int(1.3e8 / (n * top_k)))), experts=experts, top_k=top_k, n=n,
                y=rng.choice(["bf16", "f16", "f32"]), out=rng.choice(["bf16", "f16", "f32"]), add=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs

def _groups(case):
    return -(-case["k"] // case["group"])


def _w_rows(case):
    return case["n"] * (2 if case["gated"] else 1)


def _counts(case):
    """Rows of each expert, in some order: a few experts are in demand (up to
    about four times the mean), some get nothing; one expert has at most one
    row of a token."""
    rows, e = case["tokens"] * case["top_k"], case["experts"]
    share = [(0.15 + (i * 0.6180339887498949 % 1.0) ** 2) * (0.0 if e >= 8 and i % 8 == 5 else 1.0) for i in range(e)]
    total = sum(share)
    counts = [min(case["tokens"], int(rows * s / total)) for s in share]
    left, i = rows - sum(counts), 0
    while left > 0:
        if counts[i % e] < case["tokens"]:
            counts[i % e] += 1
            left -= 1
        i += 1
    return counts


def _randn(gen, shape, dev):
    return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)


def _weights(gen, case, dev):
    """Codes around the middle, scales that give results of about one, and
    zero points near the middle."""
    e, rows, k, g = case.get("experts", 1), _w_rows(case), case["k"], _groups(case)
    s = {"codes": torch.empty((e, rows, (k + 1) // 2), dtype=torch.uint8, device=dev)}
    for i in range(e):
        lo, hi = ((_randn(gen, (rows, (k + 1) // 2), dev) * 2.6 + 7.5).round_().clamp_(0, 15).to(torch.uint8)
                  for _ in range(2))
        if k % 2:
            hi[:, -1] = 0
        s["codes"][i] = lo | hi << 4
    scale = torch.rand((e, rows, g), generator=gen, device=dev) * 0.8 + 0.6
    s["scales"] = (scale * (0.35 / math.sqrt(k))).to(_TYPES[case["scale"]])
    s["zeros"] = s["bias"] = None
    if case["zeros"]:
        s["zeros"] = torch.randint(0x55, 0xbb, (e, rows, (g + 1) // 2), generator=gen, device=dev, dtype=torch.uint8)
    if case["bias"]:
        s["bias"] = _randn(gen, (e, rows), dev) * 0.1
    return s


def _tokens(gen, case, rows, dev):
    """Activations with a few strong channels."""
    x = _randn(gen, (rows, case["k"]), dev)
    x[:, :: max(1, case["k"] // 5)] *= 6
    return x.to(_TYPES[case["type"]])


class _Handle:
    """A context of the library, released with the state that holds it."""

    def __init__(self, ctx, release):
        self.ctx, self.release = ctx, release

    def __del__(self):
        self.release(self.ctx)


def _code(dq, name):
    return {"f32": dq.DQ_F32, "bf16": dq.DQ_BF16, "f16": dq.DQ_F16}[name]


def _w4_handle(case, state, rows):
    import dynamic_quantized_gemm_amd as dq

    h = dq.dq_w4_init(case.get("experts", 1), case["n"], case["k"], case["group"], _code(dq, case["type"]),
                      _code(dq, case["scale"]), _code(dq, case["y"]), case["gated"], rows)
    dq.dq_w4_set_w(h, state["codes"], state["scales"], state["zeros"], state["bias"])
    return _Handle(h, dq.dq_w4_release)


def _moe_handle(case):
    import dynamic_quantized_gemm_amd as dq

    scoring = {"softmax": dq.DQ_MOE_SOFTMAX, "sigmoid": dq.DQ_MOE_SIGMOID}[case.get("scoring", "softmax")]
    return _Handle(dq.dq_moe_init(case["tokens"], case["experts"], case["top_k"], _code(dq, case.get("type", "f32")),
                                  scoring, case.get("normalize", True), 1.0), dq.dq_moe_release)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    state = {"case": case}
    op = case["op"]
    if op == "w4":
        state.update(_weights(gen, case, dev))
        state["x"] = _tokens(gen, case, case["rows"], dev)
        state["out"] = torch.empty((case["rows"], case["n"]), dtype=_TYPES[case["y"]], device=dev)
        if own:
            state["w4"] = _w4_handle(case, state, case["rows"])
        return state
    if op == "grouped":
        rows, e = case["tokens"] * case["top_k"], case["experts"]
        state.update(_weights(gen, case, dev))
        state["x"] = _tokens(gen, case, case["tokens"] if case["gather"] else rows, dev)
        counts = torch.tensor(_counts(case), device=dev)[torch.randperm(e, generator=gen, device=dev)]
        state["offsets"] = torch.cat((counts.new_zeros(1), counts.cumsum(0))).to(torch.int32)
        state["row_index"] = None
        if case["gather"]:
            state["row_index"] = (torch.randperm(rows, generator=gen, device=dev) // case["top_k"]).to(torch.int32)
        state["out"] = torch.empty((rows, case["n"]), dtype=_TYPES[case["y"]], device=dev)
        if own:
            state["w4"] = _w4_handle(case, state, rows)
        return state
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    if op == "route":
        logits = _randn(gen, (t, e), dev) * 1.5 + _randn(gen, (e,), dev)
        if case["masked"]:
            # experts that are switched off, and tokens that may use few or none
            off = torch.rand((t, e), generator=gen, device=dev) < torch.rand((t, 1), generator=gen, device=dev).pow_(8)
            off |= torch.rand((e,), generator=gen, device=dev) < 0.1
            off[torch.rand((t,), generator=gen, device=dev) < 0.02] = True
            logits.masked_fill_(off, -math.inf)
        state["logits"] = logits.to(_TYPES[case["type"]])
        state["ids"] = torch.full((t, k), -7, dtype=torch.int32, device=dev)
        state["weights"] = torch.full((t, k), -7.0, device=dev)
        state["offsets"] = torch.full((e + 1,), -7, dtype=torch.int32, device=dev)
        state["row_token"] = torch.full((t * k,), -7, dtype=torch.int32, device=dev)
        state["row_of"] = torch.full((t, k), -7, dtype=torch.int32, device=dev)
        if own:
            state["moe"] = _moe_handle(case)
        return state
    state["y"] = _randn(gen, (t * k, case["n"]), dev).to(_TYPES[case["y"]])
    state["weights"] = torch.softmax(_randn(gen, (t, k), dev), -1)
    # the rows of a token lie far apart; a few tokens have less than top_k
    state["row_of"] = torch.randperm(t * k, generator=gen, device=dev).to(torch.int32).view(t, k)
    none = torch.rand((t, k), generator=gen, device=dev) < 0.01
    state["row_of"].masked_fill_(none, -1)
    state["weights"].masked_fill_(none, 0.0)
    state["add"] = _randn(gen, (t, case["n"]), dev).to(_TYPES[case["out"]]) if case["add"] else None
    state["out"] = torch.empty((t, case["n"]), dtype=_TYPES[case["out"]], device=dev)
    if own:
        state["moe"] = _moe_handle(case)
    return state


# ------------------------------------------------------------- plain forms

def _halves(packed, n):
    """The 4-bit values of the last dimension's bytes, n of them."""
    return torch.stack((packed & 15, packed >> 4), -1).flatten(-2)[..., :n]


def _dequantized(state):
    """W [experts, rows, K] in fp32."""
    case = state["case"]
    g = torch.arange(case["k"], device=state["codes"].device) // case["group"]
    zero = 8.0 if state["zeros"] is None else _halves(state["zeros"], _groups(case)).float()[..., g]
    return (_halves(state["codes"], case["k"]).float() - zero) * state["scales"].float()[..., g]


def _finished(case, v, bias):
    if bias is not None:
        v = v + bias
    if case["gated"]:
        gate, up = v[..., : case["n"]], v[..., case["n"]:]
        v = gate / (1 + (-gate).exp()) * up
    return v


def _plain_w4(state):
    case = state["case"]
    v = torch.matmul(state["x"].float(), _dequantized(state)[0].T)
    return _finished(case, v, state["bias"]).to(_TYPES[case["y"]])


def _plain_grouped(state):
    case, x, off = state["case"], state["x"], state["offsets"].long()
    rows, most = case["tokens"] * case["top_k"], max(_counts(case))
    # every expert's rows, filled up to the longest
    row = off[:-1, None] + torch.arange(most, device=x.device)
    live = row < off[1:, None]
    row = row.clamp_max(rows - 1)
    src = row if state["row_index"] is None else state["row_index"].long()[row]
    v = torch.matmul(x.float()[src], _dequantized(state).transpose(1, 2).contiguous())
    v = _finished(case, v, None if state["bias"] is None else state["bias"][:, None])
    state["out"][row[live]] = v[live].to(state["out"].dtype)
    return state["out"]


def _plain_route(state):
    case = state["case"]
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    logits = state["logits"].float()
    top, ids = torch.sort(logits, dim=-1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    chosen = top > -math.inf
    if case["scoring"] == "softmax":
        high = logits.amax(-1, keepdim=True)
        high = torch.where(high > -math.inf, high, 0.0)
        part = (top - high).exp()
        total = (logits - high).exp().sum(-1, keepdim=True)
    else:
        part = 1 / (1 + (-top).exp())
        total = torch.ones_like(part[:, :1])
    part = part * chosen
    if case["normalize"]:
        total = part.sum(-1, keepdim=True)
    weights = torch.where(chosen, part / total, 0.0)
    # pairs in the order of the expert, then of the token; those without an expert last
    key = torch.where(chosen, ids, e).flatten()
    order = key.argsort(stable=True)
    number = torch.empty_like(order)
    number[order] = torch.arange(t * k, device=order.device)
    offsets = (key[:, None] < torch.arange(e + 1, device=key.device)).sum(0)
    live = torch.arange(t * k, device=order.device) < offsets[-1]
    i32 = torch.int32
    return {"ids": torch.where(chosen, ids, -1).to(i32), "weights": weights, "offsets": offsets.to(i32),
            "row_token": torch.where(live, order // k, state["row_token"].long()).to(i32),
            "row_of": torch.where(chosen, number.view(t, k), -1).to(i32)}


def _plain_combine(state):
    row = state["row_of"].long()
    rows = state["y"][row.clamp_min(0)].float() * (state["weights"] * (row >= 0))[..., None]
    out = rows.sum(1)
    if state["add"] is not None:
        out = out + state["add"].float()
    return out.to(state["out"].dtype)


# ----------------------------------------------------- the framework's form

def _own_w4(state):
    import dynamic_quantized_gemm_amd as dq

    dq.dq_w4_forward(state["w4"].ctx, state["x"], state["out"])
    return state["out"]


def _own_grouped(state):
    import dynamic_quantized_gemm_amd as dq

    dq.dq_w4_forward_grouped(state["w4"].ctx, state["x"], state["offsets"], state["out"],
                             row_index=state["row_index"])
    return state["out"]


def _own_route(state):
    import dynamic_quantized_gemm_amd as dq

    s = state
    dq.dq_moe_route(s["moe"].ctx, s["logits"], s["ids"], s["weights"], s["offsets"], s["row_token"], s["row_of"])
    return {n: s[n] for n in ("ids", "weights", "offsets", "row_token", "row_of")}


def _own_combine(state):
    import dynamic_quantized_gemm_amd as dq

    s = state
    dq.dq_moe_combine(s["moe"].ctx, s["y"], s["weights"], s["row_of"], s["out"], add=s["add"])
    return s["out"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"w4": _own_w4, "grouped": _own_grouped, "route": _own_route, "combine": _own_combine}[op](state)
    return {"w4": _plain_w4, "grouped": _plain_grouped, "route": _plain_route, "combine": _plain_combine}[op](state)


# -------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op in ("w4", "grouped"):
        wr, k = _w_rows(case), case["k"]
        one = wr * ((k + 1) // 2 + _groups(case) * _BYTES[case["scale"]])
        one += wr * ((_groups(case) + 1) // 2) if case["zeros"] else 0
        one += 4 * wr if case["bias"] else 0
        if op == "w4":
            rows, moved = case["rows"], one + case["rows"] * k * _BYTES[case["type"]]
        else:
            rows = case["tokens"] * case["top_k"]
            moved = one * sum(c > 0 for c in _counts(case)) + 4 * (case["experts"] + 1)
            moved += (case["tokens"] if case["gather"] else rows) * k * _BYTES[case["type"]]
            moved += 4 * rows if case["gather"] else 0
        return {"bytes": moved + rows * case["n"] * _BYTES[case["y"]], "flops": 2 * rows * wr * k}
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    if op == "route":
        return {"bytes": t * e * _BYTES[case["type"]] + 16 * t * k + 4 * (e + 1), "flops": 3 * t * e}
    moved = t * k * (case["n"] * _BYTES[case["y"]] + 8) + t * case["n"] * _BYTES[case["out"]] * (2 if case["add"] else 1)
    return {"bytes": moved, "flops": 2 * t * k * case["n"]}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    state = prepare(case, seed)
    return {"w4": _exact_w4, "grouped": _exact_grouped, "route": _exact_route, "combine": _exact_combine}[case["op"]](
        case, state)


def _exact_rows(case, state, expert, x):
    """x [rows, K] through one expert, group by group: the sum over a group
    is s (sum of x q - z sum of x), in fp64."""
    wr, k, group = _w_rows(case), case["k"], case["group"]
    packed = state["codes"][expert].to(torch.int32)
    q = torch.zeros((wr, 2 * packed.shape[1]), dtype=torch.float64, device=x.device)
    q[:, 0::2], q[:, 1::2] = packed % 16, packed // 16
    x, v = x.double(), torch.zeros((x.shape[0], wr), dtype=torch.float64, device=x.device)
    for g in range(_groups(case)):
        at = slice(g * group, min(k, (g + 1) * group))
        z = 8
        if state["zeros"] is not None:
            z = (state["zeros"][expert][:, g // 2].int() // (16 if g % 2 else 1) % 16).double()
        v += (x[:, at] @ q[:, at].T - x[:, at].sum(1, keepdim=True) * z) * state["scales"][expert][:, g].double()
    if state["bias"] is not None:
        v += state["bias"][expert].double()
    if not case["gated"]:
        return v
    return v[:, : case["n"]] * torch.sigmoid(v[:, : case["n"]]) * v[:, case["n"]:]


def _exact_w4(case, state):
    return _exact_rows(case, state, 0, state["x"])


def _exact_grouped(case, state):
    out = torch.zeros(state["out"].shape, dtype=torch.float64, device="cuda")
    off = state["offsets"].tolist()
    for e in range(case["experts"]):
        a, b = off[e], off[e + 1]
        if a < b:
            x = state["x"][a:b] if state["row_index"] is None else state["x"][state["row_index"][a:b].long()]
            out[a:b] = _exact_rows(case, state, e, x)
    return out


def _exact_route(case, state):
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    logits = state["logits"].double()
    left = logits.clone()
    ids = torch.full((t, k), -1, dtype=torch.int64, device="cuda")
    weights = torch.zeros((t, k), dtype=torch.float64, device="cuda")
    score = torch.softmax(logits, -1) if case["scoring"] == "softmax" else torch.sigmoid(logits)
    each = torch.arange(e, device="cuda")
    for j in range(k):
        best = left.amax(-1, keepdim=True)
        pick = torch.where(left == best, each, e).amin(-1)  # the lowest of the largest
        some = best[:, 0] > -math.inf
        ids[some, j] = pick[some]
        weights[some, j] = score[some, pick[some]]
        left[some, pick[some]] = -math.inf
    if case["normalize"]:
        weights /= weights.sum(-1, keepdim=True).clamp_min(1e-300)
    row_token, row_of = state["row_token"].clone(), torch.full((t, k), -1, dtype=torch.int32, device="cuda")
    offsets, at = [0], 0
    for x in range(e):
        token, j = (ids == x).nonzero(as_tuple=True)
        row = torch.arange(at, at + len(token), dtype=torch.int32, device="cuda")
        row_token[at:at + len(token)] = token.to(torch.int32)
        row_of[token, j] = row
        at += len(token)
        offsets.append(at)
    return {"ids": ids.to(torch.int32), "weights": weights,
            "offsets": torch.tensor(offsets, dtype=torch.int32, device="cuda"), "row_token": row_token, "row_of": row_of}


def _exact_combine(case, state):
    out = torch.zeros((case["tokens"], case["n"]), dtype=torch.float64, device="cuda")
    if state["add"] is not None:
        out += state["add"].double()
    for j in range(case["top_k"]):
        t = (state["row_of"][:, j] >= 0).nonzero()[:, 0]
        out[t] += state["y"][state["row_of"][t, j].long()].double() * state["weights"][t, j, None].double()
    return out
