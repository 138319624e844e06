"""Requests that go back behind the fork they came from, and on from there: a fork of the row
from itself at the length to keep, then the release of the row. The others' rows stay as they are."""
import numpy as np
import pytest
import torch

from oracle import gqa_pages

BS, MB = 8, 6
# Rows 0-2 share the first 21 rows (two full blocks and a copied one each) and have grown to LENS;
# rows 1 and 2 go back to KEEP: inside a block that all share, and to the end of one. Rows 3 and 4
# are unused.
LENS, KEEP = [29, 33, 21, 0, 0], [None, 13, 16]


def owners(table, lens):
    n = {}
    for b, m in enumerate(lens):
        for x in table[b][:-(-int(m) // BS)]:
            n[int(x)] = n.get(int(x), 0) + 1
    return n


def state():
    table = np.full((5, MB), 99)
    table[0, :4], table[1, :5], table[2, :3] = [3, 7, 1, 9], [3, 7, 4, 2, 11], [3, 7, 8]
    shares = np.zeros(16, dtype=np.int64)
    shares[[3, 7]] = 2
    free = [0, 5, 6, 10, 12, 13, 14, 15] + [77] * 8
    return table, shares, free, 8


def test_rollback_by_the_oracle():
    table, shares, free, count = state()
    pool = np.random.default_rng(0).integers(0, 1000, (16, BS, 1))
    at_fork = [m if k is None else k for m, k in zip(LENS, KEEP + [None] * 2)]
    pools, tab, lens, sh, block, left = gqa_pages.fork([pool], [1, 2], [3, 4], table, at_fork, shares,
                                                       free, count)
    assert block.tolist() == [15, -1] and left == 7 and lens.tolist()[3:] == [13, 16]
    sh, free, left = gqa_pages.release(tab, LENS, [29, 0, 0, 0, 0], sh, free, left, 16, BS)
    now = [29, 0, 0, 13, 16]
    n = owners(tab, now)
    assert [sh[x] for x in n] == [k - 1 for k in n.values()]
    assert sorted([*n, *free[:left].tolist()]) == list(range(16))
    # The last block of each row that goes on is its own, or full.
    assert n[int(tab[3, 1])] == 1 and tab[3, 0] == 3 and n[3] == 3 and tab[4, 1] == 7
    assert (pools[0][15, :5] == pool[7, :5]).all()


@pytest.mark.gpu
def test_rollback_and_new_rows_leave_the_others_alone():
    from gqa_attention_weighted_gb300 import build
    build.build()
    import gqa_attention_weighted_gb300 as gq
    Hkv, D = 2, 64
    g = torch.Generator(device="cuda").manual_seed(1)

    def i32(x):
        return torch.tensor(np.array(x), dtype=torch.int32, device="cuda")

    def rows(pool, row, n):   # what a request reads
        return pool[tab[row].long().clamp(0, 15)].flatten(0, 1)[:n].clone()

    def draw(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    pools = [draw(16, BS, Hkv, D) for _ in "kv"]
    table, shares, free, count = state()
    tab, sh, fl, fc, left = i32(table), i32(shares), i32(free), i32([count]), i32([0])
    at_fork = i32([m if k is None else k for m, k in zip(LENS, KEEP + [None] * 2)])
    first = [rows(p, 0, 29) for p in pools]
    back = {row: [rows(p, row, KEEP[row]) for p in pools] for row in (1, 2)}
    gq.gqa_kv_fork(pools, i32([1, 2]), i32([3, 4]), tab, at_fork, sh, fl, fc, i32([0, 0]), left)
    gq.gqa_kv_release(tab, i32(LENS), i32([29, 0, 0, 0, 0]), sh, fl, left, fc, block_size=BS)
    # Seven new tokens for rows 3 and 4, one for row 0.
    cached, new = i32([29, 0, 0, 13, 16]), i32([1, 0, 0, 7, 7])
    lens, start, slots, pos = i32([0] * 5), i32([0] * 6), i32([0] * 15), i32([0] * 15)
    gq.gqa_kv_tables(cached, new, fl, fc, tab, lens, start, slots, pos, left, block_size=BS,
                     num_blocks=16)
    assert lens.tolist() == [30, 0, 0, 20, 23]
    q, k, v = draw(15, Hkv, D), draw(15, Hkv, D), draw(15, Hkv, D)
    gq.gqa_kv_norm_rope_append(q, k, v, pos, slots, torch.zeros(0, device="cuda"), torch.empty_like(q),
                               *pools)
    for i, (p, x, old) in enumerate(zip(pools, (k, v), first)):
        assert torch.equal(rows(p, 0, 29), old) and torch.equal(rows(p, 0, 30)[29], x[0])
        for row, kept, t0 in ((3, 1, 1), (4, 2, 8)):
            n = KEEP[kept]
            assert torch.equal(rows(p, row, n), back[kept][i])
            assert torch.equal(rows(p, row, n + 7)[n:], x[t0:t0 + 7])
    n = owners(tab.tolist(), lens.tolist())
    assert [sh[x].item() for x in n] == [m - 1 for m in n.values()]
    gq.gqa_kv_release(tab, lens, i32([0] * 5), sh, fl, left, fc, block_size=BS)
    assert fc.item() == 16 and sorted(fl.tolist()) == list(range(16)) and sh.sum().item() == 0
