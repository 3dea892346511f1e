"""The oracle of trees and eviction against closed forms and a scalar restatement (CPU)."""
import math

import numpy as np
import pytest

from oracle import mla, tree


def _softmax_rows(q, e, cols, rank, scale):
    s = [scale * math.fsum(float(a) * float(b) for a, b in zip(q, e[j])) for j in cols]
    m = max(s)
    z = math.fsum(math.exp(x - m) for x in s)
    o = [math.fsum(math.exp(x - m) * float(e[j][d]) for x, j in zip(s, cols)) / z for d in range(rank)]
    return o, m + math.log(z)


def test_attention_against_scalar_loops():
    rng = np.random.default_rng(3)
    T, H, L, r, n = 5, 2, 6, 4, 11
    q, e = rng.normal(size=(T, H, L)), rng.normal(size=(n, L))
    parent = [-1, 0, 0, 1, -2]
    ctx = n - T
    pos = [ctx, ctx + 1, ctx + 1, ctx + 2, ctx]
    vis = tree.visible(n, pos, 0, None, parent)
    key_sets = {0: [0], 1: [0, 1], 2: [0, 2], 3: [0, 1, 3]}
    o, lse = tree.attention(q, e, vis, r, 0.5)
    for i in range(T):
        if i == 4:
            assert (o[i] == 0).all() and np.isneginf(lse[i]).all()
            continue
        cols = list(range(ctx)) + [ctx + k for k in key_sets[i]]
        for h in range(H):
            ref, l = _softmax_rows(q[i, h], e, cols, r, 0.5)
            np.testing.assert_allclose(o[i, h], ref, rtol=1e-13)
            assert abs(lse[i, h] - l) < 1e-13


def test_a_chain_is_causal_and_a_star_is_alone():
    n, T = 20, 8
    pos = list(range(12, 20))
    chain = tree.visible(n, pos, 0, None, [-1, 0, 1, 2, 3, 4, 5, 6])
    assert (chain == (np.arange(n)[None] <= np.asarray(pos)[:, None])).all()
    star = tree.visible(n, [12] * T, 0, None, [-1] * T)
    assert (star[:, 12:] == np.eye(T, dtype=bool)).all() and star[:, :12].all()


@pytest.mark.parametrize("window", [1, 3, 13, 50])
def test_windows_count_token_positions(window):
    n, T = 16, 6
    parent, pos = [-1, 0, 0, 1, 2, 4], [10, 11, 11, 12, 12, 13]
    vis = tree.visible(n, pos, window, None, parent)
    key_pos = list(range(10)) + pos
    full = tree.visible(n, pos, 0, None, parent)
    for i in range(T):
        for j in range(n):
            assert vis[i, j] == (full[i, j] and pos[i] - key_pos[j] < window)


def test_block_rule_is_the_layer_oracles():
    pos, qv = [9, 10, 11], [1, 0, 1]
    for w in (0, 2, 4):
        ref = mla.visibility(pos, 12, w, qv, 12)
        assert (tree.visible(12, pos, w, qv, None) == ref).all()


def test_weights_of_a_rows_keys_sum_to_its_heads():
    rng = np.random.default_rng(4)
    q, e = rng.normal(size=(3, 4, 5)), rng.normal(size=(9, 5))
    vis = tree.visible(9, [6, 7, 8], 0, [1, 1, 0], [-1, 0, 1])
    _, lse = tree.attention(q, e, vis, 5, 0.3)
    w, _ = tree.key_weights(q, e, vis, lse, 0.3)
    assert abs(w.sum() - 2 * 4) < 1e-12 and w[8] == 0


def test_selection_and_compaction_by_hand():
    w = [5.0, 0.0, 2.0, 2.0, 9.0, float("nan"), 2.0, 1.0]
    assert tree.select(w, 8, 8, 0, 0) == list(range(8))
    assert tree.select(w, 8, 3, 0, 0) == [0, 2, 4]           # the tie at 2.0 to the lowest index
    assert tree.select(w, 8, 4, 1, 1) == [0, 2, 4, 7]
    assert tree.select(w, 8, 2, 1, 1) == [0, 7]
    assert tree.compact("abcdefgh", 2, [3, 6]) == list("abdgefgh")
