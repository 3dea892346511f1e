"""fp64 oracle of trees of drafted tokens and of a cache of bounded length.

Plain statements of what ``mla_tree_attention``, ``mla_key_weights``,
``mla_cache_select`` and ``mla_cache_compact`` compute: explicit loops and
numpy float64, nothing of the library.  Only tests import it.
"""
from __future__ import annotations

import numpy as np


def paths(parent):
    """Per node the nodes it sees of its own block (its path from the context,
    itself last), or None when the node is not in the tree."""
    out = []
    for i, p in enumerate(parent):
        if p == -1:
            out.append([i])
        elif p < -1 or p >= i or out[p] is None:
            out.append(None)
        else:
            out.append(out[p] + [i])
    return out


def visible(kv_len, positions, window=0, q_visible=None, parent=None):
    """vis[i, j]: query i of the block sees logical key j."""
    T = len(positions)
    vis = np.zeros((T, kv_len), dtype=bool)
    if window < 0 or (parent is not None and kv_len < T):
        return vis
    path = None if parent is None else paths(parent)
    ctx = kv_len if parent is None else kv_len - T
    for i in range(T):
        if q_visible is not None and not q_visible[i]:
            continue
        if path is not None and path[i] is None:
            continue
        for j in range(ctx):
            vis[i, j] = window == 0 or positions[i] - j < window
        for k in (path[i] if path is not None else ()):
            vis[i, ctx + k] = window == 0 or positions[i] - positions[k] < window
    return vis


def attention(q, entries, vis, rank, scale):
    """o [T, H, rank], lse [T, H] of q [T, H, L] over entries [n, L]; unseen
    entries take no part whatever they hold."""
    T, H, _ = q.shape
    o, lse = np.zeros((T, H, rank)), np.full((T, H), -np.inf)
    for i in range(T):
        e = np.asarray(entries[vis[i]], dtype=np.float64)
        if len(e) == 0:
            continue
        s = scale * (np.asarray(q[i], dtype=np.float64) @ e.T)
        m = s.max(axis=1, keepdims=True)
        p = np.exp(s - m)
        lse[i] = (m + np.log(p.sum(axis=1, keepdims=True)))[:, 0]
        o[i] = (p / p.sum(axis=1, keepdims=True)) @ e[:, :rank]
    return o, lse


def weight_mass(q, entries, vis, rank, scale):
    """sum_j p_j |v_j| of every row and dim: what a relative rounding of the
    weights can move the output by."""
    T, H, _ = q.shape
    o = np.zeros((T, H, rank))
    for i in range(T):
        e = np.asarray(entries[vis[i]], dtype=np.float64)
        if len(e):
            s = scale * (np.asarray(q[i], dtype=np.float64) @ e.T)
            p = np.exp(s - s.max(axis=1, keepdims=True))
            o[i] = (p / p.sum(axis=1, keepdims=True)) @ np.abs(e[:, :rank])
    return o


def key_weights(q, entries, vis, lse, scale):
    """(sums [n], terms): per key the sum over its rows of exp(s - lse), and per
    key the sum of those terms times (1 + |s| + |lse|), for error bounds."""
    n = vis.shape[1]
    total, size = np.zeros(n), np.zeros(n)
    for i in range(vis.shape[0]):
        cols = np.flatnonzero(vis[i])
        if not len(cols):
            continue
        s = scale * (np.asarray(q[i], dtype=np.float64) @ np.asarray(entries[cols], dtype=np.float64).T)
        for h in range(q.shape[1]):
            if np.isneginf(lse[i, h]):
                continue
            p = np.exp(s[h] - lse[i, h])
            total[cols] += p
            size[cols] += p * (1 + np.abs(s[h]) + abs(lse[i, h]))
    return total, size


def select(weights, n, budget, sink, recent):
    """Ascending indices of the keys that stay."""
    if n <= budget:
        return list(range(n))
    rank = [(bool(np.isnan(w)), 0.0 if np.isnan(w) else -float(w), j)       # NaN below -inf
            for j, w in enumerate(weights[:n]) if sink <= j < n - recent]
    best = sorted(rank)[:budget - sink - recent]
    return sorted([j for *_, j in best] + list(range(sink)) + list(range(n - recent, n)))


def compact(rows, first, keep):
    """The sequence's rows after the kept ones moved together behind `first`."""
    out = list(rows)
    for d, s in enumerate(keep):
        out[first + d] = rows[s]
    return out
