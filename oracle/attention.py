"""Rotary positions and attention over cached keys and values, fp64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

Rotary positions: the pair (a, b) at position p turns by p * f, (a cos - b sin, b cos + a sin),
and is scaled by a gain. Attention: softmax of scaled products over the tokens a query sees.
Both are written per pair and per query, to be checked by eye.
"""

import numpy as np


def rope(x, positions, inv_freq, rot, interleaved=False, gain=1.0, transposed=False):
    """x [tokens][heads][D] -> the same shape, fp64."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        # the angle in extended precision, reduced there
        t = np.asarray(positions, dtype=np.longdouble) * np.longdouble(inv_freq[i])
        t = np.fmod(t, 2 * np.arccos(np.longdouble(-1.0))).astype(np.float64)[:, None]
        c, s = np.cos(t) * gain, np.sin(t) * gain * (-1.0 if transposed else 1.0)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def seen(length, count, i, tree_row=None):
    """Mask over the `length` tokens that query i of `count` sees: its own token is
    length - count + i; with tree_row (0/1 per own token) those bits replace the causal rule
    among the last `count` tokens."""
    j = np.arange(length)
    before = length - count
    if tree_row is None:
        return j <= before + i
    own = j - before
    bits = np.zeros(length, dtype=bool)
    inside = (own >= 0) & (own < len(tree_row))
    bits[inside] = np.asarray(tree_row, dtype=bool)[own[inside]]
    return (j < before) | bits


def attend(q, k, v, scale, mask):
    """One query head: q [D], k and v [n][D], mask [n] -> (out [D], p [n]); zeros where the
    mask leaves nothing."""
    p = np.zeros(len(k))
    if mask.any():
        s = scale * (k[mask] @ q)
        e = np.exp(s - s.max())
        p[mask] = e / e.sum()
    return p @ v, p
