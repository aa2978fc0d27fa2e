"""The tests' float64 windowed attention: a window over everything is the causal
one's, the gradient is that of differences (no GPU)."""
import numpy as np
import pytest

import attention_ref
import window_ref as ref


def draw(T, heads, dim, seed):
    return np.random.default_rng(seed).standard_normal((T, heads, dim))


def test_a_window_over_everything():
    lens = [5, 0, 9]
    q, k, v, do = draw(14, 4, 8, 0), draw(14, 2, 8, 1), draw(14, 2, 8, 2), draw(14, 4, 8, 3)
    for window, sinks in ((9, 0), (100, 3), (1, 9), (4, 6)):
        a, b = attention_ref.forward(q, k, v, lens, 0.4), ref.forward(q, k, v, lens, 0.4, window, sinks)
        for x, y in zip(a, b):
            np.testing.assert_allclose(x, y, rtol=1e-12, atol=1e-300)
        a = attention_ref.backward(do, q, k, v, a[0], a[1], lens, 0.4)
        b = ref.backward(do, q, k, v, b[0], b[1], lens, 0.4, window, sinks)
        for x, y in zip(a[:3], b[:3]):
            np.testing.assert_allclose(x, y, rtol=1e-9, atol=1e-12)


def test_who_sees_whom():
    m = ref.seen(6, 2, 1)
    assert m.astype(int).tolist() == [[1, 0, 0, 0, 0, 0], [1, 1, 0, 0, 0, 0], [1, 1, 1, 0, 0, 0], [1, 0, 1, 1, 0, 0],
                                      [1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1]]


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 2), (3, 0), (3, 1), (4, 5)])
def test_gradient_against_differences(window, sinks):
    lens, scale, h = [7, 1, 4], 0.5, 1e-6
    x = [draw(12, 2, 4, 0), draw(12, 1, 4, 1), draw(12, 1, 4, 2)]
    do = draw(12, 2, 4, 3)

    def loss(x):
        return (ref.forward(*x, lens, scale, window, sinks)[0] * do).sum()

    o, lse = ref.forward(*x, lens, scale, window, sinks)[:2]
    grads = ref.backward(do, *x, o, lse, lens, scale, window, sinks)[:3]
    for i in range(3):
        for t, a, d in ((0, 0, 0), (3, 0, 2), (6, -1, 3), (7, 0, 1), (11, -1, 0)):
            up, down = [y.copy() for y in x], [y.copy() for y in x]
            up[i][t, a, d] += h
            down[i][t, a, d] -= h
            assert abs((loss(up) - loss(down)) / (2 * h) - grads[i][t, a, d]) < 1e-7
