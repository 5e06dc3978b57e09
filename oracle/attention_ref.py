"""Float64 oracle of rotary tables, norms of queries and keys with the rotation,
and attention, in plain numpy; test infrastructure, nothing shared with the
library."""

from __future__ import annotations

import numpy as np


def angles(positions, dims, theta, shared=False):
    """Angle of every token and pair, [tokens, sum(dims) / 2]."""
    positions = np.asarray(positions, np.float64).reshape(len(positions), len(dims))
    cols, before, total = [], 0, sum(dims)
    for a, n in enumerate(dims):
        for j in range(n // 2):
            power = 2 * (before + j) / total if shared else 2 * j / n
            cols.append(positions[:, a] * theta ** -power)
        before += n // 2
    return np.stack(cols, 1)


def rotate(v, table, halves):
    """Turn the first 2 pairs elements of v [tokens, heads, d] by table [tokens, pairs, 2]."""
    v, p = v.copy(), table.shape[1]
    c, s = table[:, None, :, 0], table[:, None, :, 1]
    i = np.arange(p)
    x, y = (i, i + p) if halves else (2 * i, 2 * i + 1)
    a, b = v[..., x], v[..., y]
    v[..., x], v[..., y] = a * c - b * s, b * c + a * s
    return v


def attention(q, k, v, scale, causal=False):
    """One sequence: q [n, hq, d], k, v [l, hk, d] -> out [n, hq, d], lse [hq, n], and
    the mean of |v| under the softmax weights [n, hq, d]. Keys that a query does not
    see are left out of its sums, whatever they hold."""
    n, hq, d = q.shape
    length, hk, _ = k.shape
    out = np.zeros((n, hq, d))
    lse = np.full((hq, n), -np.inf)
    spread = np.zeros((n, hq, d))
    if length == 0:
        return out, lse, spread
    for h in range(hq):
        kh, vh = k[:, h // (hq // hk)], v[:, h // (hq // hk)]
        x = q[:, h] @ kh.T * scale
        if causal:
            seen = np.arange(length)[None] <= np.arange(n)[:, None] + length - n
            x = np.where(seen, x, -np.inf)
        top = x.max(1)
        some = top > -np.inf
        p = np.exp(x - np.where(some, top, 0)[:, None])
        total = p.sum(1)
        p = p / np.where(some, total, 1)[:, None]
        out[:, h], spread[:, h] = p @ vh, p @ np.abs(vh)
        with np.errstate(divide="ignore"):
            lse[h] = np.where(some, top + np.log(total), -np.inf)
    return out, lse, spread
