"""The oracle of forks, accepted drafts and released blocks on cases worked by hand (CPU only)."""
import numpy as np

from oracle import gqa_pages


def test_fork_by_hand():
    pool = np.arange(6 * 4).reshape(6, 4, 1)
    out = gqa_pages.fork([pool], [0, 0, 1], [2, 3, 4], [[3, 1], [2, 0], [9, 9], [9, 9], [9, 9]],
                         [6, 4, 0, 0, 0], [0] * 6, [4, 5], 2)
    pools, table, lens, shares, block, left = out
    assert table.tolist() == [[3, 1], [2, 0], [3, 5], [3, 4], [2, 9]]
    assert lens.tolist() == [6, 4, 6, 6, 4]
    assert shares.tolist() == [0, 0, 1, 2, 0, 0]
    assert block.tolist() == [5, 4, -1] and left == 0
    # Rows 4 and 5 of the parent are the first two of block 1.
    assert pools[0][5, :, 0].tolist() == [4, 5, 22, 23] and pools[0][4, :, 0].tolist() == [4, 5, 18, 19]


def test_fork_without_blocks_or_with_a_row_twice():
    pool = np.zeros((4, 4, 1))
    out = gqa_pages.fork([pool], [0, 0, 1], [2, 2, 0], [[1], [2], [3]], [3, 4, 7], [0] * 4, [3], 1)
    assert out[4].tolist() == [3, -2, -2] and out[5] == 0
    out = gqa_pages.fork([pool], [0], [2], [[1], [2], [3]], [3, 4, 7], [0] * 4, [3], 0)
    assert out[4].tolist() == [-2] and out[2].tolist() == [3, 4, 7]


def test_keep_by_hand():
    pool = np.arange(4 * 4).reshape(4, 4, 1)
    pools, kept = gqa_pages.keep([pool], [3], [[0, 2, 4, 3]], [4], [[2, 0]], [8])
    assert kept.tolist() == [6]
    # Rows 3, 5, 7 of the request become 3, 4, 5: block 2 holds rows 0-3, block 0 rows 4-7.
    assert pools[0][2, :, 0].tolist() == [8, 9, 10, 11] and pools[0][0, :, 0].tolist() == [1, 3, 2, 3]


def test_release_by_hand():
    shares, free, left = gqa_pages.release([[0, 1, 2], [0, 1, 3], [4, 5, 5]], [12, 9, 4], [0, 4, 0],
                                           [1, 1, 0, 0, 0, 0], [7, 8, 9, 9, 9, 9], 1, 6, 4)
    assert shares.tolist() == [0, 0, 0, 0, 0, 0]
    assert free.tolist() == [7, 1, 2, 3, 4, 9] and left == 5
    # A block that one owner keeps stays.
    shares, free, left = gqa_pages.release([[0], [0]], [4, 4], [0, 4], [1, 0], [], 0, 2, 4)
    assert shares.tolist() == [0, 0] and left == 0
