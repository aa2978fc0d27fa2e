"""The float64 attention of the tests, checked on the CPU: against sums written
out, and its gradients against differences."""
import numpy as np
import pytest

import attention_ref as ref

LENGTHS = [3, 0, 1, 5]


def draw(seed, heads=4, kv=2, dim=3):
    rng = np.random.default_rng([21, seed])
    T = sum(LENGTHS)
    return tuple(rng.standard_normal((T, h, dim)) for h in (heads, kv, kv, heads))


def test_forward_by_hand():
    q, k, v, _ = draw(0)
    o, lse, top, eo, el, et = ref.forward(q, k, v, LENGTHS, 0.7)
    start = np.repeat(np.concatenate([[0], np.cumsum(LENGTHS)[:-1]]), LENGTHS)
    for h in range(4):
        most = -np.inf
        for i in range(len(start)):
            w = [np.exp(0.7 * float(q[i, h] @ k[j, h // 2])) for j in range(start[i], i + 1)]
            most = max(most, np.log(max(w)))
            np.testing.assert_allclose(lse[h, i], np.log(sum(w)), rtol=1e-12)
            np.testing.assert_allclose(o[i, h], sum(x * v[j, h // 2] for x, j in zip(w, range(start[i], i + 1))) / sum(w),
                                       rtol=1e-11, atol=1e-13)
        np.testing.assert_allclose(top[h], most, rtol=1e-11)
    assert (eo > 0).all() and (el > 0).all() and (et > 0).all()


@pytest.mark.parametrize("which", [0, 1, 2])
def test_gradients_by_differences(which):
    x = list(draw(1))
    do = x[3]
    o, lse, *_ = ref.forward(*x[:3], LENGTHS, 0.7)
    grads = ref.backward(do, *x[:3], o, lse, LENGTHS, 0.7)
    step = 1e-6
    rng = np.random.default_rng(22)
    for _ in range(12):
        at = tuple(rng.integers(0, n) for n in x[which].shape)
        value = []
        for sign in (1, -1):
            y = [a.copy() for a in x[:3]]
            y[which][at] += sign * step
            value.append((ref.forward(*y, LENGTHS, 0.7)[0] * do).sum())
        # central difference: error step^2 / 6 of third derivatives plus 1e-16 / step of rounding
        np.testing.assert_allclose(grads[which][at], (value[0] - value[1]) / (2 * step), rtol=1e-6, atol=1e-8)
