"""Reference products with 4-bit weights and layers of experts (CPU oracle, fp64).

TEST INFRASTRUCTURE: only the test suite may use it.

Everything is computed from the definitions in numpy's fp64 on the values that
the inputs stand for; nothing is rounded to the library's types. Codes are
packed two in a byte, the even index in the low half.
"""
from __future__ import annotations

import numpy as np


def halves(packed, n):
    """The n 4-bit values of the last dimension's bytes."""
    packed = np.asarray(packed)
    out = np.zeros(packed.shape[:-1] + (n,), np.int64)
    for i in range(n):
        out[..., i] = packed[..., i // 2] >> (4 if i % 2 else 0) & 15
    return out


def weights(codes, scales, zeros, K, group):
    """W [rows, K] = (q - z) s of one expert; zeros None: every z is 8."""
    q = halves(codes, K)
    groups = -(-K // group)
    z = np.full(q.shape[:-1] + (groups,), 8) if zeros is None else halves(zeros, groups)
    W = np.zeros(q.shape)
    for k in range(K):
        W[..., k] = (q[..., k] - z[..., k // group]) * np.asarray(scales, np.float64)[..., k // group]
    return W


def product(x, W, bias=None, gated=False):
    v = np.asarray(x, np.float64) @ W.T
    if bias is not None:
        v = v + np.asarray(bias, np.float64)
    if not gated:
        return v
    n = W.shape[0] // 2
    with np.errstate(over="ignore"):
        return v[:, :n] / (1 + np.exp(-v[:, :n])) * v[:, n:]


def product_bound(x, codes, scales, zeros, K, group, pieces, bias=None, gated=False):
    """How far fp32 sums may be from `product`, before y is rounded.

    A group's sums (of x q and of x) take `pieces` products a k, one rounding
    each (relative to a partial sum, none of which exceeds the sum of the
    magnitudes); they are joined, scaled and added to the groups before with
    three more roundings a group, and the partial sums of at most 16 parts of
    K with one each, the bias with one: with B the sum over all k of
    |s| (q + z) |x| + |bias|, (pieces min(group, K) + 3 G + 17) 2^-24 B.
    """
    q = halves(codes, K)
    groups = -(-K // group)
    z = np.full(q.shape[:-1] + (groups,), 8) if zeros is None else halves(zeros, groups)
    g = np.arange(K) // group
    B = np.abs(np.asarray(x, np.float64)) @ ((q + z[..., g]) * np.abs(np.asarray(scales, np.float64)[..., g])).T
    if bias is not None:
        B = B + np.abs(np.asarray(bias, np.float64))
    d = (pieces * min(group, K) + 3 * groups + 17) * 2.0 ** -24 * B
    if not gated:
        return d
    # silu has a slope of at most 1.1; its exp, sum and quotient and the product
    # with u are within 8 roundings
    v = product(x, weights(codes, scales, zeros, K, group), bias)
    n = d.shape[1] // 2
    with np.errstate(over="ignore"):
        s = v[:, :n] / (1 + np.exp(-v[:, :n]))
    return (1.1 * d[:, :n] * (np.abs(v[:, n:]) + d[:, n:]) + np.abs(s) * d[:, n:]
            + 8 * 2.0 ** -24 * np.abs(s * v[:, n:]))


def route(logits, top_k, sigmoid=False, normalize=True, scale=1.0):
    """ids, weights [tokens, top_k], offsets, row_token, row_of."""
    logits = np.asarray(logits, np.float64)
    tokens, experts = logits.shape
    ids = np.full((tokens, top_k), -1, np.int64)
    weights = np.zeros((tokens, top_k))
    for t in range(tokens):
        l = logits[t]
        order = sorted((e for e in range(experts) if l[e] > -np.inf), key=lambda e: (-l[e], e))[:top_k]
        ids[t, :len(order)] = order
        with np.errstate(over="ignore", invalid="ignore"):
            if sigmoid:
                w = 1 / (1 + np.exp(-l[order]))
                total = w.sum() if normalize else 1.0
            else:
                high = max((v for v in l if v > -np.inf), default=0.0)
                e = np.exp(l - high)
                w = e[order]
                total = w.sum() + 0 * e.sum() if normalize else e.sum()
            weights[t, :len(order)] = w / total * scale
    offsets, row_token, row_of = [0], [], np.full((tokens, top_k), -1, np.int64)
    for e in range(experts):
        for t in range(tokens):
            for j in range(top_k):
                if ids[t, j] == e:
                    row_of[t, j] = len(row_token)
                    row_token.append(t)
        offsets.append(len(row_token))
    return ids, weights, np.array(offsets), np.array(row_token, np.int64), row_of


def combine(y, weights, row_of, add=None):
    y = np.asarray(y, np.float64)
    out = np.zeros((len(row_of), y.shape[1])) if add is None else np.array(add, np.float64)
    for t in range(len(row_of)):
        for j, r in enumerate(row_of[t]):
            if r >= len(y):
                out[t] = np.nan
            elif r >= 0:
                out[t] += float(weights[t, j]) * y[r]
    return out
