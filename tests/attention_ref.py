"""Plain float64 attention over packed sequences, for the tests: the formulas
alone, with numpy, one sequence and head at a time."""
import numpy as np

BF = 2.0 ** -8     # half a step of bfloat16, relative
F32 = 2.0 ** -24   # half a step of float32, relative
# Relative error of a float32 probability: exp2's argument is off by half a
# step of the logit and of the reference each (|.| < 2^7 in base 2 for the
# tests' inputs) and the function by a few steps: below 2^7 * 4 * 2^-24 + 2^-21.
PROB = 2.0 ** -14


def forward(q, k, v, lengths, scale):
    """o (T, H, D), lse (H, T), each head's largest logit, and the errors that a
    kernel may make in o, in lse and in the logit: products in float32 (an
    absolute logit error of (D + 2) half steps of sum |q||k|), probabilities
    off by PROB and rounded to bfloat16, o rounded once to bfloat16."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    H, K, D = q.shape[1], k.shape[1], q.shape[2]
    T = sum(lengths)
    o, lse, top = np.zeros((T, H, D)), np.zeros((H, T)), np.full(H, -np.inf)
    eo, es = np.zeros((T, H, D)), np.zeros((H, T))
    a = 0
    for n in lengths:
        for h in range(H if n else 0):
            g = h // (H // K)
            s = scale * (q[a:a + n, h] @ k[a:a + n, g].T)
            s[np.triu_indices(n, 1)] = -np.inf
            m = s.max(axis=1)
            lse[h, a:a + n] = m + np.log(np.exp(s - m[:, None]).sum(axis=1))
            p = np.exp(s - lse[h, a:a + n, None])
            o[a:a + n, h] = p @ v[a:a + n, g]
            top[h] = max(top[h], m.max())
            sums = scale * (D + 2) * F32 * np.tril(np.abs(q[a:a + n, h]) @ np.abs(k[a:a + n, g]).T)
            es[h, a:a + n] = sums.max(axis=1)
            # the same error in every logit of a row cancels; the spread counts, at most twice the largest
            prob = np.expm1(2 * sums.max(axis=1))[:, None] + PROB + BF * (1 + PROB)
            eo[a:a + n, h] = prob * (p @ np.abs(v[a:a + n, g])) + BF * (1 + 2 * BF) * np.abs(o[a:a + n, h])
        a += n
    e_lse = es + 4 * F32 * (np.abs(lse) + 1) + 2.0 ** -20
    e_top = np.array([es[h].max() if T else 0.0 for h in range(H)]) + 4 * F32 * np.abs(np.where(np.isfinite(top), top, 0))
    return o, lse, top, eo, e_lse, e_top


def backward(do, q, k, v, o, lse, lengths, scale):
    """dq, dk, dv with o and lse as given (the forward's rounded ones, or exact
    ones), and the errors that a kernel may make in each: p and ds off as in
    the forward pass and by the float32 sums of dO.v and delta, both rounded
    to bfloat16 as operands, the results rounded once to bfloat16."""
    do, q, k, v, o, lse = (np.asarray(x, dtype=np.float64) for x in (do, q, k, v, o, lse))
    H, K = q.shape[1], k.shape[1]
    T = sum(lengths)
    D = q.shape[2]
    dq, dk, dv = (np.zeros((T,) + x.shape[1:]) for x in (q, k, v))
    eq, ek, ev = (np.zeros((T,) + x.shape[1:]) for x in (q, k, v))
    a = 0
    for n in lengths:
        r = slice(a, a + n)
        for h in range(H if n else 0):
            g = h // (H // K)
            s = scale * (q[r, h] @ k[r, g].T)
            s[np.triu_indices(n, 1)] = -np.inf
            p = np.exp(s - lse[h, r, None])
            ds = p * (do[r, h] @ v[r, g].T - (do[r, h] * o[r, h]).sum(axis=1)[:, None])
            dq[r, h] = scale * ds @ k[r, g]
            dk[r, g] += scale * ds.T @ q[r, h]
            dv[r, g] += p.T @ do[r, h]
            sums = scale * (D + 2) * F32 * np.tril(np.abs(q[r, h]) @ np.abs(k[r, g]).T)
            prob = np.expm1(2 * sums.max(axis=1))[:, None] + PROB
            part = (D + 2) * F32 * (np.abs(do[r, h]) @ np.abs(v[r, g]).T
                                    + (np.abs(do[r, h]) * np.abs(o[r, h])).sum(axis=1)[:, None])
            es = (prob + BF * (1 + PROB)) * np.abs(ds) + (1 + BF) * p * part
            # sums over rows in float32: one half step per 16 products and per row block, all positive
            run = (n + 16) * F32
            eq[r, h] = scale * (es + run * np.abs(ds)) @ np.abs(k[r, g])
            ek[r, g] += scale * (es + run * np.abs(ds)).T @ np.abs(q[r, h])
            ev[r, g] += ((prob + BF * (1 + PROB) + run) * p).T @ np.abs(do[r, h])
        a += n
    return (dq, dk, dv) + tuple(e + BF * (1 + 2 * BF) * np.abs(x) + 1e-30 for e, x in ((eq, dq), (ek, dk), (ev, dv)))
