"""Pins of the paged-cache oracle: worked values, invariants and finite
differences, none of which uses the library."""
import numpy as np
import pytest

from oracle import paged as O


def test_rotation_by_a_quarter_turn_and_pass_through():
    x = np.arange(1.0, 7.0).reshape(1, 1, 6)
    pos = np.array([[1]], np.int32)
    y = O.rotate(x, pos, [0, 0], [np.pi / 2, np.pi])
    # pairs (1, 3) and (2, 4): a quarter and a half turn; 5, 6 pass through
    assert np.allclose(y[0, 0], [-3, -2, 1, -4, 5, 6], atol=1e-12)
    y = O.rotate(x, pos, [0, 0], [np.pi / 2, np.pi], interleaved=True)
    assert np.allclose(y[0, 0], [-2, 1, -3, -4, 5, 6], atol=1e-12)


def test_each_pair_takes_its_axis():
    r = np.random.default_rng(1)
    x = r.normal(size=(3, 2, 8))
    pos = np.array([[5, 6, 7], [1, 1, 1], [0, 9, 2]], np.int32)
    axis, freq = [0, 1, 2, 0], [1.0, 0.5, 0.25, 0.125]
    y = O.rotate(x, pos, axis, freq)
    for t in range(3):
        for i in range(4):
            z = (x[t, :, i] + 1j * x[t, :, i + 4]) * np.exp(1j * pos[axis[i], t] * freq[i])
            assert np.allclose(y[t, :, i], z.real) and np.allclose(y[t, :, i + 4], z.imag)


@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse_undoes_and_is_the_gradient(interleaved):
    r = np.random.default_rng(2)
    x, g = r.normal(size=(2, 1, 10)), r.normal(size=(2, 1, 10))
    pos = np.array([[3, 40000]], np.int32)
    axis, freq = [0] * 4, [1.0, 0.1, 0.01, 0.001]
    y = O.rotate(x, pos, axis, freq, interleaved)
    assert np.allclose(O.rotate(y, pos, axis, freq, interleaved, inverse=True), x)
    dx = O.rotate(g, pos, axis, freq, interleaved, inverse=True)
    for d in range(10):
        e = np.zeros_like(x)
        e[..., d] = 1e-6
        diff = (O.rotate(x + e, pos, axis, freq, interleaved) - O.rotate(x - e, pos, axis, freq, interleaved)) / 2e-6
        assert np.allclose((diff * g).sum(-1), dx[..., d], atol=1e-8)


def test_quantized_rows():
    codes, scale = O.quantize_rows(np.array([[127.0, -63.5, 0.5, 1.5], [0, 0, 0, 0]], np.float32))
    assert scale.tolist() == [1.0, 1.0]
    assert codes.tolist() == [[127, -64, 0, 2], [0, 0, 0, 0]]


def _cache(r, pages, heads, size, dim):
    return r.normal(size=(pages, heads, size, dim)), r.normal(size=(pages, heads, size, dim))


def test_attention_of_one_and_of_equal_tokens():
    r = np.random.default_rng(3)
    k, v = _cache(r, 4, 1, 2, 4)
    table = np.array([[2, 0, 3], [1, 1, 1]], np.int32)
    q = r.normal(size=(2, 2, 4))
    out, lse, got, _, _ = O.attend(q, [1, 0], table, k, v, None, None, 0.5, 2)
    assert np.allclose(out[0], v[2, 0, 0]) and np.allclose(lse[0], 0.5 * q[0] @ k[2, 0, 0])
    assert np.all(out[1] == 0) and np.all(np.isneginf(lse[1]))
    assert got[0, 0].tolist() == [2.0, 0, 0, 0, 0, 0]
    # equal scores: the mean of the values, lse = s + log n
    out, lse, got, _, _ = O.attend(np.zeros((2, 2, 4)), [5, 0], table, k, v, None, None, 0.5, 2)
    rows = np.stack([v[2, 0, 0], v[2, 0, 1], v[0, 0, 0], v[0, 0, 1], v[3, 0, 0]])
    assert np.allclose(out[0], rows.mean(0)) and np.allclose(lse[0], np.log(5))
    # the last two tokens only
    out, lse, got, _, _ = O.attend(np.zeros((2, 2, 4)), [5, 0], table, k, v, None, None, 0.5, 2, window=2)
    assert np.allclose(out[0], rows[3:].mean(0)) and np.allclose(got[0, 0], [0, 0, 0, 1, 1, 0])


def test_log_sum_is_the_derivative_of_the_scale():
    # d lse / d sm_scale = sum p (q . k), by central differences
    r = np.random.default_rng(4)
    k, v = _cache(r, 3, 1, 4, 4)
    table = np.array([[1, 0, 2]], np.int32)
    q = r.normal(size=(1, 1, 4))
    def lse(c):
        return O.attend(q, [11], table, k, v, None, None, c, 4)[1][0, 0]
    kk = O.sequence(k, None, table, 0, 11, 4)[0]
    s = kk @ q[0, 0]
    p = np.exp(0.3 * s) / np.exp(0.3 * s).sum()
    assert np.isclose((lse(0.3 + 1e-6) - lse(0.3 - 1e-6)) / 2e-6, p @ s)


def test_eviction_keeps_what_it_should():
    #        slot  0    1    2    3    4    5
    scores = [5.0, 1.0, 3.0, 3.0, 9.0, 3.0]
    order = [7, 0, 2, 3, 4, 6]
    # the first (order 0) and the last (order 7 > 7 - 1) stay, then 9.0, then the lowest 3.0
    assert O.evict_source(scores, order, 6, 4, 7, 1, 1) == [0, 1, 2, 4]
    assert O.evict_source(scores, order, 6, 3, 7, 1, 1) == [0, 1, 4]
    assert O.evict_source(scores, order, 6, 2, 7, 0, 0) == [0, 4]
    # nothing to do, more protected than fit, a NaN above everything
    assert O.evict_source(scores, order, 4, 4, 7, 1, 1) == [0, 1, 2, 3]
    assert O.evict_source(scores, order, 6, 2, 7, 8, 0) == [0, 1]
    assert O.evict_source([1.0, 2.0, np.nan], [0, 1, 2], 3, 1, 2, 0, 0) == [2]
