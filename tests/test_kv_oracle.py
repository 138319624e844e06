"""Hand-worked cases that pin the oracle of the cache-feeding calls (CPU)."""
import numpy as np

from oracle import gqa_kv


def test_tables_hand_worked():
    # Blocks of 4. Request 0 holds 3 rows and brings 2 (one new block), request 1
    # starts empty with 5 (two), request 2 brings nothing, request 3 fills its block.
    table = np.array([[7, 0, 0], [0, 0, 0], [1, 0, 0], [2, 0, 0]])
    out, lens, start, slots, pos, left = gqa_kv.tables(
        [3, 0, 4, 2], [2, 5, 0, 2], [9, 8, 6, 5, 3], 4, table, 10, 4, 10, [100, 0, 0, 50])
    assert out.tolist() == [[7, 5, 0], [6, 8, 0], [1, 0, 0], [2, 0, 0]]
    assert lens.tolist() == [5, 5, 4, 4] and start.tolist() == [0, 2, 7, 7, 9] and left == 1
    assert slots.tolist() == [31, 20, 24, 25, 26, 27, 32, 10, 11, -1]
    assert pos.tolist() == [103, 104, 0, 1, 2, 3, 4, 52, 53, 0]


def test_tables_refuse_in_request_order():
    # Two free blocks: request 0 needs 1, request 1 needs 2 (not served), request 2
    # needs 1 (the running sum is past the list), request 3 needs none.
    out, lens, _, slots, _, left = gqa_kv.tables(
        [0, 0, 0, 1], [1, 5, 1, 1], [4, 6], 2, np.zeros((4, 2)), 8, 4, 8)
    assert lens.tolist() == [1, 0, 0, 2] and left == 1
    assert slots.tolist() == [24, -1, -1, -1, -1, -1, -1, 1]


def test_quarter_turns():
    # A pair turned by a quarter of a turn goes (a, b) -> (-b, a).
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    y, _ = gqa_kv.norm_rotate(x, None, 0, 0, [[1]], [np.pi / 2, 0.0], [2], False)
    assert np.allclose(y, [[[-3, 2, 1, 4]]])
    y, _ = gqa_kv.norm_rotate(x, None, 0, 0, [[1], [2]], [np.pi / 2, np.pi / 2], [1, 1], True)
    assert np.allclose(y, [[[-2, 1, -3, -4]]])


def test_norm_has_unit_mean_square():
    x = np.random.default_rng(0).standard_normal((2, 3, 16))
    y, _ = gqa_kv.norm_rotate(x, np.zeros(16), 0.0, 1.0, [[5, 9]], [0.3] * 8, [8], False)
    assert np.allclose((y * y).mean(-1), 1)
