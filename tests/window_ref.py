"""Plain float64 attention with a window and first tokens that stay visible, for
the tests: the formulas alone, with numpy, one sequence and head at a time, and
the errors that a kernel may make (as in attention_ref, over visible pairs)."""
import numpy as np

from attention_ref import BF, F32, PROB


def seen(n, window, sinks):
    i, j = np.arange(n)[:, None], np.arange(n)[None, :]
    return (j <= i) & ((i - j < window) | (j < sinks))


def spans(lengths):
    a = 0
    for n in lengths:
        if n:
            yield slice(a, a + n), n
        a += n


def logits(q, k, scale, mask):
    s = scale * (q @ k.T)
    s[~mask] = -np.inf
    return s


def product_error(q, k, scale, mask):
    """Each row's largest error of a logit: D + 2 half steps of sum |q||k|."""
    sums = scale * (q.shape[1] + 2) * F32 * (np.abs(q) @ np.abs(k).T)
    return np.where(mask, sums, 0).max(axis=1)


def forward(q, k, v, lengths, scale, window, sinks):
    """o, lse, each head's largest logit, and their errors."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    H, K = q.shape[1], k.shape[1]
    T = sum(lengths)
    o, eo = np.zeros(q.shape), np.zeros(q.shape)
    lse, es = np.zeros((H, T)), np.zeros((H, T))
    top = np.full(H, -np.inf)
    for r, n in spans(lengths):
        mask = seen(n, window, sinks)
        for h in range(H):
            g = h // (H // K)
            s = logits(q[r, h], k[r, g], scale, mask)
            m = s.max(axis=1)
            lse[h, r] = m + np.log(np.exp(s - m[:, None]).sum(axis=1))
            p = np.exp(s - lse[h, r, None])
            o[r, h] = p @ v[r, g]
            top[h] = max(top[h], m.max())
            es[h, r] = product_error(q[r, h], k[r, g], scale, mask)
            prob = np.expm1(2 * es[h, r])[:, None] + PROB + BF * (1 + PROB)
            eo[r, h] = prob * (p @ np.abs(v[r, g])) + BF * (1 + 2 * BF) * np.abs(o[r, h])
    e_top = np.array([es[h].max() if T else 0.0 for h in range(H)]) + 4 * F32 * np.abs(np.where(np.isfinite(top), top, 0))
    return o, lse, top, eo, es + 4 * F32 * (np.abs(lse) + 1) + 2.0 ** -20, e_top


def backward(do, q, k, v, o, lse, lengths, scale, window, sinks):
    """dq, dk, dv with o and lse as given, and their errors."""
    do, q, k, v, o, lse = (np.asarray(x, dtype=np.float64) for x in (do, q, k, v, o, lse))
    H, K, D = q.shape[1], k.shape[1], q.shape[2]
    out = [np.zeros(x.shape) for x in (q, k, v)]
    err = [np.zeros(x.shape) for x in (q, k, v)]
    for r, n in spans(lengths):
        mask = seen(n, window, sinks)
        for h in range(H):
            g = h // (H // K)
            p = np.exp(logits(q[r, h], k[r, g], scale, mask) - lse[h, r, None])
            ds = p * (do[r, h] @ v[r, g].T - (do[r, h] * o[r, h]).sum(axis=1)[:, None])
            out[0][r, h] = scale * ds @ k[r, g]
            out[1][r, g] += scale * ds.T @ q[r, h]
            out[2][r, g] += p.T @ do[r, h]
            prob = np.expm1(2 * product_error(q[r, h], k[r, g], scale, mask))[:, None] + PROB
            part = (D + 2) * F32 * (np.abs(do[r, h]) @ np.abs(v[r, g]).T
                                    + (np.abs(do[r, h]) * np.abs(o[r, h])).sum(axis=1)[:, None])
            es = (prob + BF * (1 + PROB)) * np.abs(ds) + (1 + BF) * p * part
            run = (n + 16) * F32   # sums over rows in float32
            err[0][r, h] = scale * (es + run * np.abs(ds)) @ np.abs(k[r, g])
            err[1][r, g] += scale * (es + run * np.abs(ds)).T @ np.abs(q[r, h])
            err[2][r, g] += ((prob + BF * (1 + PROB) + run) * p).T @ np.abs(do[r, h])
    return tuple(out) + tuple(e + BF * (1 + 2 * BF) * np.abs(x) + 1e-30 for e, x in zip(err, out))
