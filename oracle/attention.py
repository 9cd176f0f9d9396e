"""The attention layers' operators, straight from their definitions, in float64.

prep    every head's norm and the rotation by position
attend  softmax attention of every new row over the places that it sees
commit  the accepted path's places moved together

A paged cache is (pages [P, HKV, page_size, d], table [B, max_pages]); ``place``
reads one stream's place.
"""

from __future__ import annotations

import numpy as np

from .tree import depths, root_path


def prep(x, norm="rms", weight=None, eps=1e-6, freqs=None, positions=None, axis=None, pairs="half"):
    """x [N, H, d] normed and rotated; positions [axes, N] (integers), freqs [R/2], axis [R/2] or None."""
    x = np.array(x, np.float64)
    if norm != "none":
        ss = (x ** 2).sum(-1, keepdims=True)
        x = x / np.sqrt((ss / x.shape[-1] if norm == "rms" else ss) + eps)
        if weight is not None:
            x = x * np.asarray(weight, np.float64)
    for j in range(0 if freqs is None else len(freqs)):
        a, b = (j, j + len(freqs)) if pairs == "half" else (2 * j, 2 * j + 1)
        row = positions[0 if axis is None else min(max(int(axis[j]), 0), len(positions) - 1)]
        angle = (np.asarray(row, np.float64) * float(freqs[j]))[:, None]
        xa, xb = x[..., a].copy(), x[..., b].copy()
        x[..., a] = xa * np.cos(angle) - xb * np.sin(angle)
        x[..., b] = xb * np.cos(angle) + xa * np.sin(angle)
    return x


def place(cache, table, b, i):
    """Place i of stream b: [HKV, d]."""
    ps = cache.shape[2]
    return cache[table[b, i // ps], :, i % ps]


def attend(q, k_cache, v_cache, table, context, rows, parent=None, window=0, sinks=0, scale=1.0):
    """(o, weight) float64, o [N, HQ, d] and weight [N, HQ, d] = sum_j p_ij |v_j| (what errors are measured by), for
    rows[b] = the rows of q that stream b's new tokens are, in order.  Rows of no stream stay NaN."""
    q = np.asarray(q, np.float64)
    N, HQ, d = q.shape
    HKV = k_cache.shape[1]
    o, weight = np.full((N, HQ, d), np.nan), np.full((N, HQ, d), np.nan)
    for b, mine in enumerate(rows):
        c = int(context[b])
        deep = list(range(len(mine))) if parent is None else depths(parent[b][:len(mine)])
        for i, row in enumerate(mine):
            path = range(i + 1) if parent is None else root_path(parent[b][:len(mine)], i)
            seen = [(c + i2, c + deep[i2]) for i2 in path] + [(j, j) for j in range(c)]
            if window:
                seen = [(j, t) for j, t in seen if c + deep[i] - t < window or t < sinks]
            K = np.stack([place(k_cache, table, b, j) for j, _ in seen]).astype(np.float64)
            V = np.stack([place(v_cache, table, b, j) for j, _ in seen]).astype(np.float64)
            for h in range(HQ):
                hk = h // (HQ // HKV)
                s = scale * (K[:, hk] @ q[row, h])
                p = np.exp(s - s.max())
                p /= p.sum()
                o[row, h] = p @ V[:, hk]
                weight[row, h] = p @ np.abs(V[:, hk])
    return o, weight


def commit(accepted, parent, k_cache, v_cache, table, context):
    """(k_cache, v_cache, context) after the accepted paths' moves; every place is read from the caches before."""
    k_new, v_new, ctx = k_cache.copy(), v_cache.copy(), np.array(context)
    ps = k_cache.shape[2]
    for b, node in enumerate(accepted):
        path = [] if node < 0 else root_path(parent[b], int(node))
        for at, i in enumerate(sorted(path)):
            for new, old in ((k_new, k_cache), (v_new, v_cache)):
                to = context[b] + at
                new[table[b, to // ps], :, to % ps] = place(old, table, b, context[b] + i)
        ctx[b] += len(path)
    return k_new, v_new, ctx
