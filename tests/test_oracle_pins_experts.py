"""Pins of the fp64 oracle of 4-bit weights and layers of experts: values
worked out by hand."""
import numpy as np

from oracle import experts as X


def test_halves_low_first():
    assert X.halves(np.array([[0x21, 0x43, 0xF5]], np.uint8), 5).tolist() == [[1, 2, 3, 4, 5]]


def test_weights_by_groups_of_two():
    # codes 1 2 3 4 5, groups of 2 with scales 1, 10, 100 and zero points 0, 3, 15
    W = X.weights(np.array([[0x21, 0x43, 0x05]], np.uint8), np.array([[1.0, 10.0, 100.0]]),
                  np.array([[0x30, 0x0F]], np.uint8), 5, 2)
    assert W.tolist() == [[1.0, 2.0, 0.0, 10.0, -1000.0]]
    W = X.weights(np.array([[0x21, 0x43, 0x05]], np.uint8), np.array([[1.0, 10.0, 100.0]]), None, 5, 2)
    assert W.tolist() == [[-7.0, -6.0, -50.0, -40.0, -300.0]]


def test_product_and_gate():
    W = np.array([[1.0, 2.0], [3.0, -1.0]])
    x = np.array([[2.0, 1.0], [0.0, 0.0]])
    assert X.product(x, W).tolist() == [[4.0, 5.0], [0.0, 0.0]]
    assert X.product(x, W, bias=[1.0, -1.0]).tolist() == [[5.0, 4.0], [1.0, -1.0]]
    got = X.product(x, W, gated=True)
    assert np.allclose(got, [[4 / (1 + np.exp(-4.0)) * 5], [0.0]], rtol=1e-15)


def test_route_ties_masks_and_rows():
    inf = np.inf
    logits = np.array([[0.0, 1.0, 1.0, -inf],      # a tie: expert 1 before 2
                       [-inf, -inf, 5.0, -inf],    # one expert left
                       [-inf] * 4,                 # none
                       [3.0, np.nan, 2.0, 1.0]])
    ids, w, off, tok, row = X.route(logits, 2)
    assert ids.tolist() == [[1, 2], [2, -1], [-1, -1], [0, 2]]
    assert w[0].tolist() == [0.5, 0.5] and w[1].tolist() == [1.0, 0.0] and w[2].tolist() == [0.0, 0.0]
    assert np.isnan(w[3]).all()
    assert off.tolist() == [0, 1, 2, 5, 5]
    assert tok.tolist() == [3, 0, 0, 1, 3]
    assert row.tolist() == [[1, 2], [3, -1], [-1, -1], [0, 4]]
    _, w, _, _, _ = X.route(logits, 2, normalize=False, scale=2.0)
    assert np.allclose(w[0], 2 * np.e / (1 + 2 * np.e), rtol=1e-15)
    _, w, _, _, _ = X.route(logits, 2, sigmoid=True, normalize=False)
    assert np.allclose(w[3], [1 / (1 + np.exp(-3.0)), 1 / (1 + np.exp(-2.0))], rtol=1e-15)


def test_combine():
    y = np.array([[1.0, 2.0], [10.0, 20.0]])
    out = X.combine(y, np.array([[0.5, 2.0], [1.0, 9.0], [1.0, 1.0]]), np.array([[0, 1], [1, -1], [0, 2]]),
                    np.array([[100.0, 100.0]] * 3))
    assert out[:2].tolist() == [[120.5, 141.0], [110.0, 120.0]]
    assert np.isnan(out[2]).all()


def test_product_bound_covers_fp32_sums():
    r = np.random.default_rng(1)
    K, n, group = 300, 6, 32
    codes = r.integers(0, 256, (n, 150), dtype=np.uint8)
    scales = r.uniform(0.01, 0.03, (n, 10))
    x = r.normal(0, 1, (5, K)).astype(np.float32)
    for gated in (False, True):
        want = X.product(x, X.weights(codes, scales, None, K, group), gated=gated)
        d = X.product_bound(x, codes, scales, None, K, group, 1, gated=gated)
        v = np.zeros((5, n), np.float32)
        q = X.halves(codes, K).astype(np.float32)
        for g in range(10):
            sl = slice(g * group, min(K, g * group + group))
            s = np.zeros((5, n), np.float32)
            for k in range(sl.start, sl.stop):
                s += x[:, k, None] * (q[None, :, k] - np.float32(8))
            v += s * scales[:, g].astype(np.float32)
        if gated:
            v = v[:, :3] / (1 + np.exp(-v[:, :3])) * v[:, 3:]
        err = np.abs(v - want)
        assert (err <= d + 2.0 ** -23 * np.abs(want)).all()
        # and says something: a code off by one in one place is outside it
        assert (d < np.abs(x[:, 7, None]) * 0.01 + 0.01).mean() > 0.5
