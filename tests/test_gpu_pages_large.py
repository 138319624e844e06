"""gqa_kv_release of more entries than its CTAs keep in shared memory (CUDA GPU)."""
import numpy as np
import pytest

from test_gpu_pages import run_release

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    from gqa_attention_weighted_gb300 import build
    build.build()
    import gqa_attention_weighted_gb300 as pkg
    return pkg


@pytest.mark.parametrize("shared", [False, True])
def test_releases_of_half_a_million_entries(gq, shared):
    # 8192 rows of 64 blocks, 32768 entries a CTA of 16: all but every 50th row ended, the rows in
    # groups of three that share their first 20 blocks.
    rng = np.random.default_rng(11)
    B, MB, bs = 8192, 64, 8
    nb = B * MB + 7
    tab = rng.permutation(nb)[:B * MB].reshape(B, MB)
    shares = np.zeros(nb, dtype=np.int64)
    if shared:
        for b in range(0, B - 2, 3):
            tab[b + 1:b + 3, :20] = tab[b, :20]
            shares[tab[b, :20]] = 2
    old = rng.integers(MB * bs - 100, MB * bs + 1, B)
    new = np.where(np.arange(B) % 50 == 0, old // 3, 0)
    ref = run_release(gq, tab, old, new, shares if shared else None, rng.permutation(nb), 1, nb, bs)
    assert ref[2] > 16 * 16384
