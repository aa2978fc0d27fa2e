"""Norms of queries and keys with rotary positions in float64, for the tests:
the formulas alone, with numpy, and the errors that a kernel may make."""
from fractions import Fraction

import numpy as np

BF = 2.0 ** -8     # half a step of bfloat16, relative
F32 = 2.0 ** -24   # half a step of float32, relative
TWO_PI = Fraction("6.283185307179586476925286766559005768394338798750211641949889184615632812572417997256")


def places(lengths, axes=1):
    """Each token's index in its sequence, on every axis."""
    p = np.concatenate([np.arange(n) for n in lengths]) if sum(lengths) else np.zeros(0)
    return np.broadcast_to(p.astype(np.int64), (axes, p.size))


def angles(positions, rotary):
    """(tokens, pairs) angles within one turn of position times frequency, from whole numbers."""
    axes, T = positions.shape
    out = np.zeros((T, len(rotary.frequencies)))
    seen = {}
    for i, (f, a) in enumerate(zip(rotary.frequencies, rotary.pair_axes)):
        for t in range(T):
            key = (i, int(positions[a, t]))
            if key not in seen:
                turns = Fraction(f) * key[1] / TWO_PI
                seen[key] = float((turns - round(turns)) * TWO_PI)
            out[t, i] = seen[key]
    return out


def pairs_of(rotary):
    R = rotary.rotary_dim
    if rotary.interleaved:
        return np.arange(0, R, 2), np.arange(1, R, 2)
    return np.arange(R // 2), np.arange(R // 2, R)


def turn(x, u, rotary, back=False):
    lo, hi = pairs_of(rotary)
    c, s = np.cos(u)[:, None], np.sin(u)[:, None] * (-1 if back else 1)
    z = x.copy()
    z[..., lo] = x[..., lo] * c - x[..., hi] * s
    z[..., hi] = x[..., hi] * c + x[..., lo] * s
    return z


def both(x, rotary):
    """|x| of an element and of its pair's other one."""
    lo, hi = pairs_of(rotary)
    e = np.abs(x)
    z = e.copy()
    z[..., lo] = z[..., hi] = e[..., lo] + e[..., hi]
    return z


def inverse(x, eps):
    return 1 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)


def forward(x, u, rotary, norm, weight, eps):
    """z and its error: the sum of D squares (half of its error counts in the
    root), the root, two products and the rotation in float32, cos and sin off
    by up to 4 half steps, z rounded once to bfloat16."""
    x = np.asarray(x, dtype=np.float64)
    D = x.shape[-1]
    y = x * inverse(x, eps) if norm else x
    if weight is not None:
        y = y * weight
    z = turn(y, u, rotary)
    return z, (D + 20) * F32 * both(y, rotary) + BF * (1 + 2 * BF) * np.abs(z) + 2.0 ** -133


def backward(dz, x, u, rotary, norm, weight, eps):
    """dx, dw and their errors."""
    dz = np.asarray(dz, dtype=np.float64)
    D = dz.shape[-1]
    g = turn(dz, u, rotary, back=True)
    eg = 10 * F32 * both(dz, rotary)
    if not norm:
        return g, None, eg + BF * (1 + 2 * BF) * np.abs(g) + 2.0 ** -133, None
    x = np.asarray(x, dtype=np.float64)
    r = inverse(x, eps)
    n = x * r
    w = np.ones(D) if weight is None else np.asarray(weight, dtype=np.float64)
    along = (w * g * n).mean(axis=-1, keepdims=True)
    size = (np.abs(w * n) * both(dz, rotary)).mean(axis=-1, keepdims=True)
    dx = r * (w * g - n * along)
    rel = (D + 20) * F32
    ex = r * (np.abs(w) * (eg + rel * np.abs(g)) + np.abs(n) * (2 * rel + 10 * F32) * size)
    dw = (g * n).sum(axis=(0, 1))
    # sums in float32 over at most 64 terms of a lane and its work-group, then in float64
    ew = ((eg + (rel + 64 * F32) * np.abs(g)) * np.abs(n)).sum(axis=(0, 1)) + 2 * F32 * np.abs(dw) + 1e-30
    return dx, dw, ex + BF * (1 + 2 * BF) * np.abs(dx) + 2.0 ** -133, ew
