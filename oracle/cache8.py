"""fp64 oracle of the 8-bit latent cache and of the verification of drafted tokens.

Plain statements of what ``mla_cache8_store``, ``mla_cache8_load`` and
``mla_verify_drafts`` compute: numpy and loops, nothing of the library.  Only
tests import it.
"""
from __future__ import annotations

import math

import numpy as np


def e4m3_values():
    """The number of every e4m3 code 0 .. 255: a sign, 4 bits of exponent (bias 7) and 3
    of fraction; no infinities, 0x7f and 0xff NaN."""
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out[c] = math.nan if (c & 127) == 127 else -v if c & 128 else v
    return out


E4M3 = e4m3_values()


def to_e4m3(x):
    """Codes of the nearest e4m3 numbers (ties to the even code), |x| <= 448."""
    x = np.asarray(x, dtype=np.float64)
    grid, a = E4M3[:127], np.abs(x)
    up = np.clip(np.searchsorted(grid, a), 0, 126)
    down = np.maximum(up - 1, 0)
    du, dd = grid[up] - a, a - grid[down]
    code = np.where((du < dd) | ((du == dd) & (up % 2 == 0)), up, down)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def scale_of(latent):
    """The least power of two that brings the largest magnitude to 448 or below."""
    k, top = -64, float(np.max(np.abs(latent)))
    while top > 448.0 * 2.0 ** k:
        k += 1
    return 2.0 ** k


def quantise(entries, rank=512):
    """(codes [n, rank], rope [n, rest], scale [n]) of float64 entries holding bf16 numbers."""
    codes, scales = np.zeros((len(entries), rank), dtype=np.uint8), np.empty(len(entries))
    for i, e in enumerate(entries):
        if not np.isfinite(e).all() or np.abs(e[:rank]).max() >= 2.0 ** 127:
            scales[i] = math.nan
            continue
        scales[i] = scale_of(e[:rank])
        codes[i] = to_e4m3(e[:rank] / scales[i])
    return codes, entries[:, rank:], scales


def dequantise(codes, rope, scale):
    return np.concatenate([E4M3[codes] * scale[:, None], rope], axis=1)


def _clean(row):
    row = np.asarray(row, dtype=np.float64)
    return np.where(np.isfinite(row) & (row > 0), row, 0.0)


def pick(w, u):
    """The least x with sum_{y <= x} w(y) > u sum w, -1 without mass."""
    total = math.fsum(w)
    if not total > 0:
        return -1
    c = np.cumsum(np.asarray(w, dtype=np.longdouble))
    over = np.flatnonzero((c > np.longdouble(u) * c[-1]) & (w > 0))
    return int(over[0]) if len(over) else int(np.flatnonzero(w > 0)[-1])


def verify(target, draft, tokens, uniforms, parent=None, first=0):
    """(accepted nodes + first, next token) of one sequence: target [T + 1, V], draft
    [T, V] or None, tokens [T], uniforms [T + 1]."""
    T, V = len(tokens), target.shape[1]
    parent = [i - 1 for i in range(T)] if parent is None else parent
    node, path = -1, []
    w, s = _clean(target[0]), 1.0
    for i in range(T):
        x = tokens[i]
        if parent[i] >= i or parent[i] != node or not 0 <= x < V:
            continue
        q = _clean(draft[node + 1]) if draft is not None else None
        qx = 1.0 if q is None else q[x]
        if uniforms[i] * s * qx < w[x]:
            path.append(i)
            node = i
            w, s = _clean(target[i + 1]), 1.0
        elif q is None:
            s -= w[x]
            w[x] = 0.0
        else:
            w = np.maximum(w - s * q, 0.0)
            s = math.fsum(w)
    if not math.fsum(w) > 0:
        w = _clean(target[node + 1])
    return [p + first for p in path], pick(w, float(uniforms[T]))
