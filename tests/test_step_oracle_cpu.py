"""Pins of oracle/stepref.py: cases worked by hand, and its agreement with attnref where they meet; tree_mask (CPU)."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import attnref, stepref


def test_norm_by_hand():
    x = np.array([[[3.0, 4.0]]])  # mean square 12.5
    assert np.allclose(stepref.norm(x, None, 0.0), np.array([3.0, 4.0]) / 12.5 ** 0.5, rtol=1e-15)
    assert np.allclose(stepref.norm(x, [2.0, -1.0], 3.5), [6.0 / 4.0, -1.0], rtol=1e-15)
    assert (stepref.norm(np.zeros((1, 1, 8)), np.ones(8), 1e-6) == 0).all()


def test_plan_by_hand():
    # pages of 4.  0: 7 + 1 tokens stay in 2 pages; 1: 8 + 1 need a third; 2: cut back from 3 pages to 1; 3: ended;
    # 4: 0 + 6 need 2
    table = [[10, 11, -1, -1], [12, 13, -1, -1], [14, 15, 16, -1], [17, -1, -1, -1], [-1, -1, -1, -1]]
    r = stepref.plan([7, 8, 2, 0, 0], [1, 1, 2, 0, 6], table, [2, 2, 3, 1, 0], list(range(20, 40)), 3, 4, 12)
    # given back in order: 15, 16, 17 on top of 20, 21, 22; taken from the top: 17 by 1, 16 and 15 by 4
    assert r["table"] == [[10, 11, -1, -1], [12, 13, 17, -1], [14, -1, -1, -1], [-1, -1, -1, -1], [16, 15, -1, -1]]
    assert r["owned"] == [2, 3, 1, 0, 2] and r["count"] == 3 and r["status"] == [0] * 5
    assert r["free"][:6] == [20, 21, 22, 15, 16, 17]
    assert r["q_start"] == [0, 1, 2, 4, 4, 10] and r["kv_total"] == [8, 9, 4, 0, 6]
    assert r["pos"] == [7, 8, 2, 3, 0, 1, 2, 3, 4, 5, 0, 0]
    # pages 14 .. 17 are slots 56 ..; 20 pages is the stack's size, so 20 and on would be no pages
    assert r["slot"] == [11 * 4 + 3, 17 * 4, 14 * 4 + 2, 14 * 4 + 3, 64, 65, 66, 67, 60, 61, -1, -1]


def test_plan_refusals_by_hand():
    # two free pages: 0 takes one, 1 lacks two and gets none, 2 (one) is behind it, 3 needs none; 4 does not fit the table,
    # 5 has a negative length, 6's rows end past the step's
    r = stepref.plan([4, 4, 4, 1, 16, -1, 0], [1, 5, 1, 1, 1, 1, 9], [[0, -1, -1, -1], [1, -1, -1, -1], [2, -1, -1, -1],
                                                                   [3, -1, -1, -1], [4, 5, 6, 7], [-1] * 4, [-1] * 4],
                     [1, 1, 1, 1, 4, 0, 0], [8, 9], 2, 4, 12)
    assert r["status"] == [0, 2, 1, 0, -1, -1, -1] and r["count"] == 1
    assert r["owned"] == [2, 1, 1, 1, 4, 0, 0] and r["table"][0] == [0, 9, -1, -1]
    assert r["q_start"] == [0, 1, 6, 7, 8, 9, 10, 12] and r["kv_total"] == [5, 4, 4, 2, 16, -1, 0]
    assert r["pos"][:8] == [4, 4, 5, 6, 7, 8, 4, 1] and r["slot"][1:7] == [-1] * 6


def test_seen_keys_by_hand():
    assert stepref.seen_keys({0, 2}, 10, 4) == [0, 1, 2, 3, 4, 5, 6, 8]
    assert stepref.seen_keys({0, 2}, 10, 4, window=4) == [4, 5, 6, 8]  # depth 1: position 7
    assert stepref.seen_keys(set(), 10, 4, window=4) == [3, 4, 5]
    assert stepref.seen_keys({0, 1, 3}, 2, 4) == [1]  # two of the four tokens are cached
    assert stepref.seen_keys({5}, 10, 4) == [0, 1, 2, 3, 4, 5]


@pytest.mark.parametrize("window", [0, 9])
def test_tree_attention_of_a_chain_is_causal_attention(window):
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((2, 6, 2, 4, 8))
    table = np.array([[3, 1, 5, -1], [0, 2, 4, -1]])
    q = rng.standard_normal((9, 4, 8))
    starts, lens = [0, 5, 9], [11, 12]
    sees = [set(range(i + 1)) for i in range(5)] + [set(range(i + 1)) for i in range(4)]
    a = stepref.attention(q, k, v, table, lens, starts, sees, scale=0.3, window=window)
    b = attnref.attention(q, k, v, table, lens, starts, scale=0.3, window=window)
    for x, y in zip(a, b):
        assert np.allclose(x, y, rtol=1e-13)


def test_adjust_by_hand():
    x = np.array([[2.0, -2.0, 1.0, 0.0, 5.0]])
    tokens = np.array([[0, 1, 1, 2, 9, -1]])
    y, _ = stepref.adjust(x, None, tokens, [5], [2], [2.0], [0.5], [0.25], [[(3, 1.0), (3, 4.0), (7, 1.0)]], [{0, 1, 3}])
    # 0: prompt only, 2 / 2; 1: twice in the prompt's 2 and once behind, -4 - 0.5 - 0.25; 2 and 4 are masked
    assert y[0].tolist() == [1.0, -4.75, -np.inf, 4.0, -np.inf]


def test_tree_mask():
    from int4_weight_only_group_amd import tree_mask
    mask, depth = tree_mask([-1, 0, 0, 2, -1])
    assert mask.tolist() == [[1], [3], [5], [13], [16]] and depth.tolist() == [0, 1, 1, 2, 0]
    mask, depth = tree_mask(range(-1, 69))  # a chain of 70
    assert mask.shape == (70, 2) and mask[63].tolist() == [-1, 0] and mask[69].tolist() == [-1, 63]
    assert depth.tolist() == list(range(70))
    assert tree_mask([])[0].shape == (0, 0)
    for bad in ([0], [-1, 1], [-1, -2], [-1, 5]):
        with pytest.raises(ValueError):
            tree_mask(bad)
