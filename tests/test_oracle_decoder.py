"""The f64 oracles of the decoder calls against closed forms, brute force and
differences (no GPU needed)."""
import numpy as np
import pytest

from oracle import decoder as od


def test_norm_then_rotation_of_one_pair():
    x = np.array([3.0, 4.0]).reshape(1, 1, 1, 2)
    out, _ = od.qk_norm_rope(x, [2.0, 1.0], np.array([[1]]), 2, eps=0.0)
    r = 1 / np.sqrt(12.5)
    a, b = 6 * r, 4 * r
    c, s = np.cos(1.0), np.sin(1.0)
    np.testing.assert_allclose(out.ravel(), [a * c - b * s, a * s + b * c], rtol=1e-14)


@pytest.mark.parametrize("D,rope", [(8, 8), (9, 5), (6, 0)])
def test_qk_gradient_against_differences(D, rope):
    rng = np.random.default_rng(D)
    x, w, g = rng.normal(size=(2, 3, 4, D)), rng.normal(size=D), rng.normal(size=(2, 3, 4, D))
    pos = rng.integers(0, 50, (2, 4))
    f = rng.uniform(0.5, 2.0, rope // 2)
    dx, dw, _, _ = od.qk_norm_rope_backward(g, x, w, pos, rope, factors=f)

    def loss(x, w):
        return float((od.qk_norm_rope(x, w, pos, rope, factors=f)[0] * g).sum())

    h = 1e-5
    for _ in range(12):
        i = tuple(rng.integers(0, n) for n in x.shape)
        e = np.zeros_like(x)
        e[i] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[i]) < 1e-7
    for d in range(D):
        e = np.zeros(D)
        e[d] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[d]) < 1e-7


@pytest.mark.parametrize("window,sinks,kv_len,start", [(3, 1, None, None), (None, 0, 7, 0), (2, 2, 9, -2), (4, 0, 5, None)])
def test_window_gradients_against_differences(window, sinks, kv_len, start):
    rng = np.random.default_rng(1)
    B, H, K, M, N, D = 1, 4, 2, 6, 9, 5
    q, k, v, g = (rng.normal(size=s) for s in ((B, H, M, D), (B, K, N, D), (B, K, N, D), (B, H, M, D)))
    seen = od.window_visible(M, N, window, sinks, kv_len, start)[None]

    def forward(q, k, v):
        return od.attention(q, k, v, seen, 0.7, 0.0)

    out, _, w, ob, sc, _ = forward(q, k, v)
    grads, _ = od.attention_backward(g, q, k, v, out, w, seen, 0.7, 0.0, ob, sc)
    h = 1e-5
    for n, x in enumerate((q, k, v)):
        for _ in range(15):
            i = tuple(rng.integers(0, m) for m in x.shape)
            up, down = [q, k, v], [q, k, v]
            e = np.zeros_like(x)
            e[i] = h
            up[n], down[n] = x + e, x - e
            slope = float(((forward(*up)[0] - forward(*down)[0]) * g).sum()) / (2 * h)
            assert abs(slope - grads[n][i]) < 1e-7


def test_visible_by_hand():
    # queries end the sequence: row 0 is at position 4 of 6
    seen = od.window_visible(2, 8, 2, 1, 6, None)
    np.testing.assert_array_equal(seen.astype(int), [[1, 0, 0, 1, 1, 0, 0, 0], [1, 0, 0, 0, 1, 1, 0, 0]])
    # rows before the sequence and behind it see nothing
    assert not od.window_visible(3, 4, None, 0, 2, -1)[[0]].any() and not od.window_visible(3, 4, None, 0, 2, 2).any()
    # a chain of new tokens is the causal mask
    np.testing.assert_array_equal(od.cached_visible(3, 9, 4, 1, 8, None), od.window_visible(3, 9, 4, 1, 8, None))
    # two branches from one root: neither sees the other
    seen = od.cached_visible(3, 6, None, 0, 5, [0b001, 0b011, 0b101])
    np.testing.assert_array_equal(seen.astype(int), [[1, 1, 1, 0, 0, 0], [1, 1, 1, 1, 0, 0], [1, 1, 1, 0, 1, 0]])
