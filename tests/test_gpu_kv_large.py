"""gqa_kv_tables for batches whose requests take more shared memory than a
kernel has by default, up to the largest batch."""
import numpy as np
import pytest

from test_gpu_kv import gq, run_tables  # noqa: F401  (gq: the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [3413, 3414, 8191, 8192])
def test_tables_of_large_batches(gq, B):  # noqa: F811
    rng = np.random.default_rng(B)
    bs = 16
    cached, new = rng.integers(0, 40, size=B), rng.integers(0, 4, size=B)
    held, want = -(-cached // bs), -(-(cached + new) // bs)
    need = int((want - held).sum())
    nb = int(held.sum()) + need + 5
    perm = rng.permutation(nb)
    table = rng.integers(-3, nb + 3, size=(B, int(want.max()) + 1))
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    run_tables(gq, cached, new, perm[at:], need - 7, table, int(new.sum()) + 33, bs, nb,
               rng.integers(0, 10000, size=B))


def test_lengths_near_the_largest(gq):  # noqa: F811
    # Far past what the table holds: not served, nothing written, the others as usual.
    big = 2 ** 31 - 1
    run_tables(gq, [big, 5, big - 16, big - 5], [0, 2, 1, 3], [1, 2, 3], 3,
               [[0, 0], [1, 2], [3, 4], [5, 6]], 6, 16, 8)
