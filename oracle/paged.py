"""Reference decoding over a paged key-value cache (CPU oracle, fp64).

TEST INFRASTRUCTURE: only the test suite may use it.

Everything is computed from the definitions in numpy's fp64 (angles in
extended precision), token by token where that is the plainest, on the
values that the inputs stand for; nothing is rounded to the library's types.
The cache is [pages, kv_heads, page_size, head_dim]; slot t of sequence b lies
in page table[b, t // page_size] at t % page_size.
"""
from __future__ import annotations

import numpy as np


def rotate(x, positions, axis, inv_freq, interleaved=False, inverse=False):
    """x [tokens, heads, dim]; pair i turns by positions[axis[i]] * inv_freq[i]."""
    out = np.array(x, np.float64)
    half = len(axis)
    for i in range(half):
        turns = positions[axis[i]].astype(np.longdouble) * np.longdouble(inv_freq[i])
        angle = turns * (-1 if inverse else 1)
        c = np.cos(angle).astype(np.float64)[:, None]
        s = np.sin(angle).astype(np.float64)[:, None]
        j, k = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a, b = np.array(x[..., j], np.float64), np.array(x[..., k], np.float64)
        out[..., j], out[..., k] = a * c - b * s, b * c + a * s
    return out


def place(table, b, t, page_size):
    """(page, slot) of slot t of sequence b."""
    return int(table[b, t // page_size]), t % page_size


def quantize_rows(rows):
    """(codes, scales) of the symmetric int8 quantization of rows [..., dim]
    in the arithmetic of rows' type."""
    top = np.abs(rows).max(-1)
    scale = (top / rows.dtype.type(127)).astype(rows.dtype)
    scale = np.where(scale > 0, scale, rows.dtype.type(1))
    return np.clip(np.rint(rows / scale[..., None]), -127, 127).astype(np.int8), scale


def sequence(cache, scale, table, b, n, page_size, first=0):
    """Rows [first, n) of sequence b, [kv_heads, n - first, dim] fp64."""
    heads, dim = cache.shape[1], cache.shape[3]
    out = np.zeros((heads, n - first, dim))
    for t in range(first, n):
        p, s = place(table, b, t, page_size)
        out[:, t - first] = cache[p, :, s].astype(np.float64)
        if scale is not None:
            out[:, t - first] *= scale[p, :, s].astype(np.float64)[:, None]
    return out


def attend(q, lens, table, k, v, k_scale, v_scale, sm_scale, page_size, window=0):
    """Returns out [batch, q_heads, dim], lse [batch, q_heads], gathered
    [batch, kv_heads, cap] (sum of p over the query heads) and, for the error
    bounds, the sum of p |v| and the largest sum of |q k| of a token."""
    batch, hq, dim = q.shape
    hk = k.shape[1]
    g = hq // hk
    out, lse = np.zeros((batch, hq, dim)), np.full((batch, hq), -np.inf)
    gathered = np.zeros((batch, hk, table.shape[1] * page_size))
    mass, reach = np.zeros((batch, hq, dim)), np.zeros((batch, hq))
    for b in range(batch):
        n = int(lens[b])
        first = max(0, n - window) if window else 0
        if n == first:
            continue
        ks = sequence(k, k_scale, table, b, n, page_size, first)
        vs = sequence(v, v_scale, table, b, n, page_size, first)
        for h in range(hq):
            x = q[b, h].astype(np.float64)
            s = sm_scale * (ks[h // g] @ x)
            reach[b, h] = abs(sm_scale) * (np.abs(ks[h // g]) @ np.abs(x)).max()
            top = s.max()
            e = np.exp(s - top)
            lse[b, h] = top + np.log(e.sum())
            p = e / e.sum()
            out[b, h] = p @ vs[h // g]
            mass[b, h] = p @ np.abs(vs[h // g])
            gathered[b, h // g, first:n] += p
    return out, lse, gathered, mass, reach


def evict_source(scores, order, n, budget, newest, recent, sinks):
    """For a head of n tokens: src[j], the slot whose token is at slot j
    afterwards."""
    if n <= budget:
        return list(range(n))
    safe = [order[i] < sinks or int(order[i]) > int(newest) - recent for i in range(n)]

    def key(i):
        w = float(scores[i])
        return (0, 0.0, i) if safe[i] else (1, 0.0, i) if w != w else (2, -w, i)  # a NaN above every other weight

    kept = set(sorted(range(n), key=key)[:budget])
    movers = [i for i in sorted(kept) if i >= budget]
    src = list(range(budget))
    for hole in [i for i in range(budget) if i not in kept]:
        src[hole] = movers.pop(0)
    assert not movers
    return src
