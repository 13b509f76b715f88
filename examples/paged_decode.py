#!/usr/bin/env python3
"""One attention layer decoding a batch of sequences over a paged int8 cache.

    python examples/paged_decode.py [--steps 64] [--budget 256]

The projections are the library's dynamic quantized inner products (weights
int8, activations quantized per row on every call), and around them run
rotary positions and the append to the cache, the attention of the new token
with its weights gathered, and the eviction that keeps every sequence at its
budget. Weights and inputs are random: what is shown is how the calls fit
together, and that from the budget on a step's buffers no longer grow.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import dynamic_quantized_gemm_amd as dq


class Projection:
    """x [rows, k] bf16 -> [rows, n] bf16 by a constant int8 weight."""

    def __init__(self, k, n, gen):
        self.k, self.n, self.ctx = k, n, {}
        self.w = torch.randint(-127, 128, (k, n), generator=gen, device="cuda", dtype=torch.int8)
        self.scale = torch.full((n,), 1.0 / (73.0 * k ** 0.5), device="cuda")

    def __call__(self, x):
        rows = x.shape[0]
        if rows not in self.ctx:
            self.ctx[rows] = dq.dqip_init(rows, self.n, self.k, dq.DQ_BF16, dq.DQ_I8, dq.DQ_BF16, True, False,
                                          dq.DQ_ACT_IDENTITY, False)
            dq.dqip_set_params(self.ctx[rows], self.w, self.scale)
        y = torch.empty((rows, self.n), dtype=torch.bfloat16, device="cuda")
        dq.dqip_forward(self.ctx[rows], x, None, None, y)
        return y

    def release(self):
        for h in self.ctx.values():
            dq.dqip_release(h)


class Layer:
    def __init__(self, batch, width, q_heads, kv_heads, head_dim, budget, page_size=16, sinks=4, recent=32, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.batch, self.hq, self.hk, self.dim, self.budget = batch, q_heads, kv_heads, head_dim, budget
        self.sinks, self.recent = sinks, recent
        self.qkv = Projection(width, (q_heads + 2 * kv_heads) * head_dim, gen)
        self.out = Projection(q_heads * head_dim, width, gen)
        # a page more than the budget: the new token is attended to before anything leaves
        self.per_seq = -(-(budget + 1) // page_size)
        self.cap, pages = self.per_seq * page_size, self.per_seq * batch
        shape = (pages, kv_heads, page_size, head_dim)
        self.k, self.v = (torch.empty(shape, dtype=torch.int8, device="cuda") for _ in range(2))
        self.ks, self.vs = (torch.empty(shape[:3], device="cuda") for _ in range(2))
        self.table = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).view(batch, self.per_seq)
        self.scores = torch.zeros((batch, kv_heads, self.cap), device="cuda")
        self.order = torch.zeros((batch, kv_heads, self.cap), dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.number = torch.zeros(batch, dtype=torch.int32, device="cuda")  # of the next token
        half = head_dim // 2
        self.rope = dq.dq_rope_init(head_dim, head_dim, [0] * half, [10000.0 ** (-i / half) for i in range(half)])
        self.kv = dq.dq_kv_init(batch, q_heads, kv_heads, head_dim, pages, page_size, self.per_seq, dq.DQ_BF16,
                                dq.DQ_I8, gather_scores=True)

    def cache(self):
        return self.table, self.k, self.v, self.ks, self.vs

    def _split(self, x):
        y = self.qkv(x).view(x.shape[0], self.hq + 2 * self.hk, self.dim)
        return y[:, :self.hq], y[:, self.hq:self.hq + self.hk], y[:, self.hq + self.hk:]

    def prompt(self, x):
        """x [batch, tokens, width]: stores the prompt's keys and values (at
        most `budget` tokens; nothing is attended to)."""
        b, t = x.shape[:2]
        _, k, v = self._split(x.reshape(b * t, -1))
        index = torch.arange(t, dtype=torch.int32, device="cuda").repeat(b)
        seq = torch.arange(b, dtype=torch.int32, device="cuda").repeat_interleave(t)
        dq.dq_kv_append(self.kv, k, v, index, *self.cache(), seq_ids=seq, rope=self.rope, positions=index.view(1, -1))
        self.order[:, :, :t] = torch.arange(t, device="cuda", dtype=torch.int32)
        self.lens.fill_(t)
        self.number.fill_(t)

    def step(self, x):
        """x [batch, width], one token of every sequence -> [batch, width]."""
        q, k, v = self._split(x)
        index = self.lens.clone()
        at = index.long().view(-1, 1, 1).expand(-1, self.hk, 1)
        self.order.scatter_(2, at, self.number.view(-1, 1, 1).expand(-1, self.hk, 1))
        self.scores.scatter_(2, at, 0.0)  # the slot may have been another token's
        turned = torch.empty((self.batch, self.hq, self.dim), dtype=torch.bfloat16, device="cuda")
        dq.dq_kv_append(self.kv, k, v, index, *self.cache(), q=q, q_out=turned, rope=self.rope,
                        positions=self.number.view(1, -1))
        self.lens += 1
        y = torch.empty_like(turned)
        dq.dq_kv_attend(self.kv, turned, self.lens, *self.cache(), y, self.dim ** -0.5, scores=self.scores,
                        scores_out=self.scores, decay=0.99)
        self.seen = turned, y, self.lens.clone()  # what this step's attention took and gave
        dq.dq_kv_evict(self.kv, self.budget, self.lens, self.number, self.scores, self.order, *self.cache(),
                       self.scores, self.order, self.lens, recent=self.recent, sinks=self.sinks)
        self.number += 1
        return self.out(y.view(self.batch, -1))

    def release(self):
        dq.dq_kv_release(self.kv)
        dq.dq_rope_release(self.rope)
        self.qkv.release()
        self.out.release()


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=64)
    p.add_argument("--batch", type=int, default=16)
    p.add_argument("--prompt", type=int, default=240)
    p.add_argument("--budget", type=int, default=256)
    a = p.parse_args()
    width = 1024
    layer = Layer(a.batch, width, 16, 4, 64, a.budget)
    gen = torch.Generator(device="cuda").manual_seed(1)
    layer.prompt(torch.randn((a.batch, min(a.prompt, a.budget), width), generator=gen, device="cuda").bfloat16())
    x = torch.randn((a.batch, width), generator=gen, device="cuda").bfloat16()
    x = layer.step(x)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        x = layer.step(x)
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    lost = dq.dq_kv_take_errors(layer.kv)
    print(f"{a.steps} steps of {a.batch} sequences: {t / a.steps * 1e6:.0f} us a step, lengths "
          f"{int(layer.lens.min())}..{int(layer.lens.max())}, {lost} bad places, "
          f"|x| {float(x.float().abs().mean()):.3g}")
    layer.release()


if __name__ == "__main__":
    main()
