"""Pins of the paged-cache oracle: hand-worked plans and closed forms."""
import math

import numpy as np

from oracle import paged_oracle as PO


def test_plan_by_hand():
    # pages of 4 rows; request 0 holds 5 tokens in pages 9, 2 and brings 4; request 1 is finished
    # and returns page 7; request 2 is new with 6 tokens; request 3 asks for more than is left
    table = np.array([[9, 2, -1, -1], [7, -1, -1, -1], [-1, -1, -1, -1], [-1, -1, -1, -1]])
    free = np.array([4, 5, -1, -1])
    p = PO.page_plan(4, [4, -1, 6, 1], [5, 3, 0, 0], table, free, 2, 11)
    # stack 4, 5, 7: request 0 needs one page (9 tokens in 3), request 2 two
    assert p["block_table"].tolist() == [[9, 2, 7, -1], [7, -1, -1, -1], [5, 4, -1, -1], [-1] * 4]
    assert p["kv_lens"].tolist() == [9, 0, 6, 0]
    assert p["status"].tolist() == [0, 0, 0, PO.PLAN_NO_PAGES]
    assert p["q_start"].tolist() == [0, 4, 4, 10, 11]
    assert p["slots"].tolist() == [9, 10, 11, 28, 20, 21, 22, 23, 16, 17, -1]
    assert p["positions"].tolist() == [5, 6, 7, 8, 0, 1, 2, 3, 4, 5, -1]
    assert p["n_free"] == 0 and p["free_pages"].tolist() == [4, 5, -1, -1]


def test_plan_returns_pages():
    p = PO.page_plan(4, [-1, 2], [8, 1], np.array([[3, 1], [0, -1]]), np.array([2, -1, -1, -1]), 1, 2)
    assert p["n_free"] == 3 and p["free_pages"].tolist() == [2, 3, 1, -1]
    assert p["slots"].tolist() == [1, 2]


def test_attention_closed_forms():
    d, B = 4, 2
    K = np.zeros((3, 1, 1, B, d))
    V = np.arange(3 * B * d, dtype=float).reshape(3, 1, 1, B, d)
    q = np.ones((2, 2, d))
    table = np.array([[2, 0]])
    # equal scores: the mean of the rows in sight, in the order of the table
    o, z, _, _ = PO.paged_attention(q, K, V, table, [0, 2], [3], 1.0)
    rows = np.concatenate([V[2, 0, 0], V[0, 0, 0]])
    assert np.allclose(o[0, 0], rows[:2].mean(0)) and np.allclose(o[1, 1], rows[:3].mean(0))
    assert np.allclose(z, [[math.log(2)] * 2, [math.log(3)] * 2])
    o, z, _, _ = PO.paged_attention(q, K, V, table, [0, 2], [3], 1.0, window=1)
    assert np.allclose(o[:, 0], rows[1:3]) and np.allclose(z, 0)
    o, z, _, _ = PO.paged_attention(q, K, V, table, [0, 2], [1], 1.0)      # the first row sees nothing
    assert (o[0] == 0).all() and np.isneginf(z[0]).all() and np.allclose(o[1, 0], rows[0])
    # one key of a much larger score
    K[0, 0, 0, 0] = 50.0
    o, z, _, E = PO.paged_attention(q, K, V, table, [0, 2], [3], 1.0)
    assert np.allclose(o[1, 0], rows[2]) and np.allclose(z[1], 200.0) and np.allclose(E[1], 200.0)


def test_write_by_hand():
    src = np.arange(1, 13, dtype=float).reshape(1, 1, 2, 3, 2)
    out = PO.page_write(src, np.array([[5, -1, 0]]), np.zeros((3, 2, 2, 2, 2)), layer=1)
    assert out[2, 1, 0, 1].tolist() == [1, 2] and out[2, 1, 1, 1].tolist() == [7, 8]
    assert out[0, 1, 0, 0].tolist() == [5, 6] and out.sum() == 1 + 2 + 7 + 8 + 5 + 6 + 11 + 12
