"""gqa_kv_fork, gqa_kv_keep and gqa_kv_release against their oracle: tables, counts and
lists exactly, pools bit for bit (CUDA GPU)."""
import numpy as np
import pytest
import torch

from oracle import gqa_pages

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    from gqa_attention_weighted_gb300 import build
    build.build()
    import gqa_attention_weighted_gb300 as pkg
    return pkg


def i32(x):
    return torch.tensor(np.array(x).astype(np.int32), device="cuda")


def pools_of(rng, n, nb, bs, shape, dtype=torch.bfloat16):
    """Distinct 16-bit (or 8-bit) patterns, NaNs among them, as a server's pools may hold."""
    raw = rng.integers(0, 256, size=(n, nb, bs, *shape, torch.empty(0, dtype=dtype).element_size()),
                       dtype=np.uint8)
    return [torch.tensor(x).view(dtype).squeeze(-1).cuda() for x in raw]


def raw(t):
    return t.cpu().contiguous().view(torch.uint8).numpy()


def shuffled_table(rng, lens, bs, nb, spare=0):
    need = [-(-max(0, n) // bs) for n in lens]
    perm = rng.permutation(nb)
    tab = rng.integers(-5, nb + 5, size=(len(lens), max(need + [1]) + 1))
    at = 0
    for b, r in enumerate(need):
        tab[b, :r] = perm[at:at + r]
        at += r
    return tab, perm[at:]


def same(got, want):
    return np.array_equal(got.cpu().numpy().reshape(-1), np.asarray(want).reshape(-1))


# ---------------------------------------------------------------- fork
def run_fork(gq, pools, parent, child, tab, lens, shares, free, count, handle=False):
    ref = gqa_pages.fork([raw(p) for p in pools], parent, child, tab, lens, shares, free, count)
    t, s, sh, fl = i32(tab), i32(lens), i32(shares), i32(free)
    N = len(parent)
    block, left = i32([77] * N), i32([77])
    gq.gqa_kv_fork(gq.KvPools(pools) if handle else pools, i32(parent), i32(child), t, s, sh, fl,
                   i32([count]), block, left)
    for got, want in zip((t, s, sh, block, left), ref[1:]):
        assert same(got, want), (got.cpu().numpy(), want)
    for got, want in zip(pools, ref[0]):
        assert np.array_equal(raw(got), want)
    assert same(fl, free)
    return ref


# block size, row shape, pools, parents' lengths, children a parent
FORKS = [(16, (2, 64), 2, [33], 4), (8, (1, 8), 1, [0, 8, 7, 1], 2), (32, (8, 128), 5, [500, 64, 31], 3),
         (48, (3, 40), 3, [47, 49, 200], 1), (256, (1, 16), 2, [255, 700], 2)]


@pytest.mark.parametrize("case", FORKS, ids=[f"bs{c[0]}-{c[1]}-n{len(c[3]) * c[4]}" for c in FORKS])
def test_forks_match_the_oracle(gq, case):
    bs, shape, n_pools, parents, copies = case
    rng = np.random.default_rng(bs)
    lens, parent, child = [], [], []
    for n in parents:
        parent += [len(lens)] * copies
        child += range(len(lens) + 1, len(lens) + 1 + copies)
        lens += [n] + [3] * copies
    held = [n if b in parent else 0 for b, n in enumerate(lens)]
    nb = sum(-(-n // bs) for n in held) + len(parent) + 2
    tab, free = shuffled_table(rng, held, bs, nb)
    for handle in (False, True):
        run_fork(gq, pools_of(rng, n_pools, nb, bs, shape), parent, child, tab, lens,
                 rng.integers(0, 3, nb), free, len(free), handle)


def test_forks_that_are_not_served(gq):
    # A child twice, a child that is a parent, itself, rows outside the table, blocks that run
    # out, lengths past the table's row, entries and list entries outside the pool.
    rng = np.random.default_rng(1)
    bs, nb = 8, 40
    lens = [20, 5, 16, 100, -3, 0, 0, 0, 0, 0, 0, 0]
    tab = rng.integers(0, 30, size=(12, 4))
    tab[0, 2], tab[2, 1] = 50, -2
    parent = [0, 1, 0, 2, 5, 12, -1, 3, 4, 1, 0, 1, 2]
    child = [6, 6, 1, 7, 5, 8, 8, 9, 10, -1, 12, 11, 8]
    for free, count in (([30, 31, -7, 45], 4), ([30, 31, 32], 1), ([30], 0), ([], 5), ([30, 31], -1)):
        ref = run_fork(gq, pools_of(rng, 2, nb, bs, (1, 16)), parent, child, tab, lens, [0] * nb, free,
                       count)
        assert -2 in ref[4]


def test_many_forks_of_many_rows(gq):
    rng = np.random.default_rng(2)
    B, bs = 8192, 8
    lens = rng.integers(0, 40, B)
    lens[4000:] = 0
    nb = sum(-(-int(n) // bs) for n in lens) + 3000
    tab, free = shuffled_table(rng, lens, bs, nb)
    parent = rng.integers(0, 4000, 4192)
    child = 4000 + rng.permutation(4192)
    run_fork(gq, pools_of(rng, 2, nb, bs, (1, 8)), parent, child, tab, lens, [0] * nb, free, len(free))


def test_no_forks_and_no_rows(gq):
    rng = np.random.default_rng(3)
    pools = pools_of(rng, 1, 4, 8, (1, 8))
    run_fork(gq, pools, [], [], np.zeros((3, 2)), [9, 0, 0], [0] * 4, [1, 2], 2)
    run_fork(gq, pools, [1], [2], np.zeros((3, 2)), [9, 0, 5], [0] * 4, [], 0)


# ---------------------------------------------------------------- keep
def run_keep(gq, pools, cached, acc, count, tab, lens):
    ref, kept = gqa_pages.keep([raw(p) for p in pools], cached, acc, count, tab, lens)
    out = i32([77] * len(cached))
    W = len(acc[0]) if len(acc) else 0
    gq.gqa_kv_keep(pools, i32(cached), i32(acc).reshape(len(cached), W), i32(count), i32(tab),
                   i32(lens), out)
    assert same(out, kept), (out.tolist(), kept)
    for got, want in zip(pools, ref):
        assert np.array_equal(raw(got), want)
    return kept


# block size, row shape, type, pools, widths W
KEEPS = [(16, (2, 64), torch.bfloat16, 2, 7), (8, (1, 8), torch.float16, 1, 1),
         (32, (8, 128), torch.bfloat16, 5, 70), (48, (1, 40), torch.bfloat16, 3, 9),
         (16, (4, 256), torch.float32, 2, 33), (16, (1, 48), torch.uint8, 2, 12)]


@pytest.mark.parametrize("case", KEEPS, ids=[f"bs{c[0]}-{c[1]}-W{c[4]}" for c in KEEPS])
def test_accepted_rows_match_the_oracle(gq, case):
    bs, shape, dtype, n_pools, W = case
    rng = np.random.default_rng(bs + W)
    B = 9
    cached = rng.integers(0, 4 * bs, B)
    new = rng.integers(1, 3 * W + 2, B)
    lens = cached + new
    nb = sum(-(-int(n) // bs) for n in lens) + 2
    tab, _ = shuffled_table(rng, lens, bs, nb)
    acc, count = np.full((B, W), 10 ** 6), []
    for b in range(B):
        n = int(min(W, rng.integers(0, new[b] + 1)))
        acc[b, :n] = np.sort(rng.choice(new[b], n, replace=False))
        count.append(n)
    run_keep(gq, pools_of(rng, n_pools, nb, bs, shape, dtype), cached, acc, count, tab, lens)


def test_accepted_numbers_that_do_not_count(gq):
    # Not ascending, twice the same, negative, at and past the length, more than W, a negative
    # count, a negative cache, a length past the table's row, entries outside the pool.
    rng = np.random.default_rng(5)
    bs, nb = 8, 64
    cached = [5, 3, 0, 9, 30, -4, 7, 20, 2, 1]
    lens = [25, 23, 20, 19, 50, 6, 27, 25, 22, 21]
    acc = [[0, 3, 2, 9], [1, 4, 4, 9], [-1, 2, 3, 4], [2, 9, 10, 11], [1, 2, 3, 9], [1, 3, 6, 7],
           [2, 3, 9, 11], [3, 4, 5, 6], [0, 1, 2, 3], [1, 5, 9, 13]]
    count = [4, 4, 4, 4, 4, 4, 9, -2, 4, 4]
    tab = rng.permutation(nb)[:40].reshape(10, 4)
    tab[9, 0], tab[9, 1] = nb, -1
    kept = run_keep(gq, pools_of(rng, 3, nb, bs, (2, 8)), cached, acc, count, tab, lens)
    assert kept.tolist() == [7, 5, 0, 11, 31, 2, 11, 20, 6, 5]
    run_keep(gq, pools_of(rng, 1, nb, bs, (2, 8)), cached, [[]] * 10, count, tab, lens)


def test_pools_whose_offsets_pass_32_bits(gq):
    # 2.1 GB of 2 KB rows: rows of the last blocks lie past 2^31 bytes.
    bs, nb = 64, 16500
    pool = torch.zeros((nb, bs, 8, 128), dtype=torch.bfloat16, device="cuda")
    pool[nb - 1, 10:20] = torch.arange(10, device="cuda").view(10, 1, 1).bfloat16() + 1
    kept, out = i32([0]), i32([77])
    gq.gqa_kv_keep([pool], i32([10]), i32([[1, 4, 9]]), i32([3]), i32([[nb - 1]]), i32([20]), kept)
    assert kept.item() == 13
    assert pool[nb - 1, 10:14, 3, 5].tolist() == [2.0, 5.0, 10.0, 4.0]
    gq.gqa_kv_fork([pool], i32([0]), i32([1]), i32([[nb - 1], [0]]), i32([13, 0]),
                   torch.zeros(nb, dtype=torch.int32, device="cuda"), i32([nb - 2]), i32([1]), out,
                   i32([0]))
    assert out.item() == nb - 2
    assert pool[nb - 2, 9:14, 7, 127].tolist() == [0.0, 2.0, 5.0, 10.0, 0.0]


# ------------------------------------------------------------- release
def run_release(gq, tab, old, new, shares, free, count, nb, bs):
    ref = gqa_pages.release(tab, old, new, shares, free, count, nb, bs)
    sh, fl, left = None if shares is None else i32(shares), i32(free), i32([77])
    t = i32(tab)
    gq.gqa_kv_release(t, i32(old), i32(new), sh, fl, i32([count]), left, block_size=bs, num_blocks=nb)
    assert same(left, ref[2]), (left.item(), ref[2])
    assert same(fl, ref[1])
    assert shares is None or same(sh, ref[0])
    assert same(t, tab)
    return ref


def release_case(rng, B, longest, bs, copies):
    old = rng.integers(0, longest + 1, B)
    new = np.where(rng.random(B) < 0.5, 0, np.maximum(0, old - rng.integers(0, 3 * bs, B)))
    nb = sum(-(-int(n) // bs) for n in old) + 3
    tab, _ = shuffled_table(rng, old, bs, nb)
    shares = np.zeros(nb, dtype=np.int64)
    for b in range(0, B - copies + 1, copies):
        n = int(min(old[b:b + copies])) // bs
        tab[b + 1:b + copies, :n] = tab[b, :n]
        shares[tab[b, :n]] = copies - 1
    return tab, old, new, shares, nb


@pytest.mark.parametrize("B,longest,bs,copies", [(1, 1, 8, 1), (3, 700, 16, 1), (40, 300, 8, 4),
                                                 (256, 4000, 16, 3), (8192, 60, 8, 2),
                                                 (20, 160000, 8, 5)])
def test_releases_match_the_oracle(gq, B, longest, bs, copies):
    rng = np.random.default_rng(B + longest)
    tab, old, new, shares, nb = release_case(rng, B, longest, bs, copies)
    ref = run_release(gq, tab, old, new, shares, rng.permutation(nb), 2, nb, bs)
    for _ in range(2):
        assert ref[2] == run_release(gq, tab, old, new, shares, rng.permutation(nb), 2, nb, bs)[2]
    if copies == 1:
        run_release(gq, tab, old, new, None, rng.permutation(nb), 0, nb, bs)


def test_releases_with_odd_arguments(gq):
    # Counts that stay above 0, one block many times, more owners than the count allows, entries
    # outside the pool, lengths past the row, negative ones, a new length above the old, a list
    # that is full, counts outside it.
    bs, nb = 8, 12
    tab = [[1, 2, 3, 4], [1, 2, 3, 12], [1, 2, -1, 5], [6, 6, 6, 7], [8, 9, 10, 11]]
    old, new = [32, 32, 200, 25, 16], [0, 8, -5, 0, 30]
    shares = [0, 4, 1, 2, 0, 0, 0, 3, 0, 0, 0, 0]
    for size, count in ((12, 0), (12, 5), (3, 1), (2, 9), (0, 0), (4, -3)):
        ref = run_release(gq, tab, old, new, shares, list(range(100, 100 + size)), count, nb, bs)
    assert ref[2] == 4 and ref[1].tolist()[:2] == [2, 4]
    run_release(gq, tab, [0] * 5, [0] * 5, shares, [0] * 3, 1, nb, bs)


def test_calls_are_captured_and_replayed(gq):
    # One graph of fork, keep and release on its own stream; lengths change between replays.
    rng = np.random.default_rng(9)
    bs, nb = 8, 64
    pools = pools_of(rng, 4, nb, bs, (2, 8))
    tab = np.zeros((4, 8), dtype=np.int64)
    tab[0], tab[1] = rng.permutation(40)[:16].reshape(2, 8)
    t, lens, shares = i32(tab), i32([20, 37, 0, 0]), i32([0] * nb)
    free, count, left, after = i32(list(range(40, 64))), i32([24]), i32([0]), i32([0])
    parent, child, block = i32([0, 0]), i32([2, 3]), i32([0, 0])
    acc, n_acc, cached, kept = i32([[0, 2, 3]] * 4), i32([3, 3, 3, 3]), i32([15, 30, 0, 0]), i32([0] * 4)
    handle = gq.KvPools(pools)

    def step():
        gq.gqa_kv_fork(handle, parent, child, t, lens, shares, free, count, block, left)
        gq.gqa_kv_keep(handle, cached, acc, n_acc, t, lens, kept)
        gq.gqa_kv_release(t, lens, kept, shares, free, left, after, block_size=bs)

    state = (t, lens, shares, free, *pools)
    before = [x.clone() for x in state]
    step()
    for x, y in zip(state, before):
        x.copy_(y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for n0 in (20, 28, 31):   # drafted rows that move lie in the partial block
        for x, y in zip(state, before):
            x.copy_(y)
        lens[0], cached[0] = n0, n0 - 5
        cached[2:] = n0 - 5
        want_pools, want_t, want_l, want_s, want_b, want_left = gqa_pages.fork(
            [raw(p) for p in pools], [0, 0], [2, 3], t.cpu().numpy(), lens.cpu().numpy(), [0] * nb,
            free.cpu().numpy(), 24)
        # The oracle's pools are bytes: rows are the same.
        want_pools, want_kept = gqa_pages.keep(want_pools, cached.cpu().numpy(), [[0, 2, 3]] * 4,
                                               [3] * 4, want_t, want_l)
        want = gqa_pages.release(want_t, want_l, want_kept, want_s, free.cpu().numpy(), want_left, nb, bs)
        g.replay()
        torch.cuda.synchronize()
        assert same(block, want_b) and same(kept, want_kept) and same(after, want[2])
        assert same(t, want_t) and same(shares, want[0]) and same(free, want[1])
        for got, ref in zip(pools, want_pools):
            assert np.array_equal(raw(got), ref)
