"""The calls of include/gqa_prompt.h: exported, bad arguments rejected on the
host before any CUDA call, and the oracle on hand-worked cases (CPU only)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from oracle import gqa_prefix, gqa_prompt

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gqa_prompt.h")
FAKE = 1 << 20  # a non-NULL 16-byte-aligned address that no rejected call touches
OUT = 1 << 40   # out lies elsewhere than the inputs


@pytest.fixture(scope="module")
def native():
    from gqa_attention_weighted_gb300 import build
    build.build()
    from gqa_attention_weighted_gb300 import _native
    return _native


def test_library_exports_every_declared_symbol(native):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"(gqa_\w+)\s*\(", text))
    assert {"gqa_prompt_attn", "gqa_tree_attn", "gqa_prompt_device_status"} <= names
    lib = ctypes.CDLL(native.LIBRARY)
    assert [n for n in sorted(names) if not hasattr(lib, n)] == []


PROMPT = dict(q=FAKE, qs=512, k=FAKE, v=FAKE, ts=FAKE, cached=FAKE, tab=FAKE, lens=FAKE, out=OUT,
              B=2, T=9, Hq=8, Hkv=2, D=64, dt=0, bs=16, nb=8, mb=4, scale=0.125)
TREE = dict(q=FAKE, qs=512, k=FAKE, v=FAKE, ts=FAKE, cached=FAKE, mask=FAKE, words=1, tab=FAKE,
            lens=FAKE, out=OUT, B=2, T=9, Hq=8, Hkv=2, D=64, dt=0, bs=16, nb=8, mb=4, scale=0.125)
BAD = [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(Hq=0), 1), (dict(Hkv=-2), 1), (dict(D=0), 1),
    (dict(bs=0), 1), (dict(nb=0), 1), (dict(mb=0), 1), (dict(Hkv=3), 1), (dict(dt=2), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(q=None), 1),
    (dict(k=None), 1), (dict(v=None), 1), (dict(ts=None), 1), (dict(tab=None), 1),
    (dict(out=None), 1), (dict(tab=FAKE + 2), 1), (dict(lens=FAKE + 1), 1), (dict(ts=FAKE + 2), 1),
    (dict(cached=FAKE + 2), 1), (dict(qs=504), 1), (dict(D=96), 2), (dict(D=512), 2),
    (dict(Hq=258, qs=258 * 64), 2), (dict(bs=12), 2), (dict(bs=4), 2), (dict(B=8193), 2),
    (dict(T=(1 << 20) + 1), 2), (dict(Hkv=1025, Hq=1025, qs=1025 * 64), 2), (dict(nb=1 << 27), 2),
    (dict(mb=(1 << 22) + 1), 2), (dict(q=FAKE + 8), 2), (dict(v=FAKE + 2), 2), (dict(out=FAKE + 2), 2),
    (dict(qs=516), 2), (dict(qs=1 << 38), 2),
    # out in the last query row, over the first and the last bytes of the pools, and of tables
    (dict(q=OUT - 8 * 512 * 2 - 1008), 1), (dict(out=FAKE + 16 * 8 * 2 * 64 * 2 - 16), 1),
    (dict(k=OUT + 9 * 512 * 2 - 16), 1), (dict(v=OUT - 16 * 8 * 2 * 64 * 2 + 16), 1),
    (dict(tab=OUT + 9 * 512 * 2 - 4), 1), (dict(ts=OUT - 8), 1), (dict(lens=OUT - 4), 1),
    (dict(cached=OUT), 1),
]


@pytest.mark.parametrize("change,status", BAD)
def test_prompt_host_checks(native, change, status):
    rc = native.lib.gqa_prompt_attn(*dict(PROMPT, **change).values(), None)
    assert rc == status, native.lib.gqa_prompt_last_error()
    assert native.lib.gqa_prompt_last_error() != b""


@pytest.mark.parametrize("change,status", BAD + [
    (dict(cached=None), 1), (dict(mask=None), 1), (dict(mask=FAKE + 2), 1), (dict(words=0), 1),
    (dict(words=(1 << 15) + 1), 2), (dict(mask=OUT - 32), 1)])
def test_tree_host_checks(native, change, status):
    rc = native.lib.gqa_tree_attn(*dict(TREE, **change).values(), None)
    assert rc == status, native.lib.gqa_prompt_last_error()
    assert native.lib.gqa_prompt_last_error() != b""


def test_no_tokens_need_no_tensors(native):
    none = dict(T=0, q=None, out=None, cached=None, lens=None)
    assert native.lib.gqa_prompt_attn(*dict(PROMPT, **none).values(), None) == 0
    none = dict(T=0, q=None, out=None, mask=None, lens=None)
    assert native.lib.gqa_tree_attn(*dict(TREE, **none).values(), None) == 0


@pytest.mark.parametrize("wait_ns,withhold", [(99999, 0), (2000000001, 0), (-1, 0), (200000, -1)])
def test_selftest_host_checks(native, wait_ns, withhold):
    rc = native.lib.gqa_prompt_selftest_wait_timeout(*PROMPT.values(), wait_ns, withhold, None)
    assert rc == 1 and b"wait_ns" in native.lib.gqa_prompt_last_error()
    rc = native.lib.gqa_prompt_selftest_wait_timeout(*dict(PROMPT, D=96).values(), 200000, 0, None)
    assert rc == 2


def test_binding_rejects_tensors_that_do_not_fit(native):
    pool = torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16)  # on the CPU
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="k_pool"):
        native.gqa_prompt_attn(q, pool, pool, i, None, i.view(1, 2), None, q)
    with pytest.raises(ValueError, match="cached_lens"):
        native.gqa_tree_attn(q, pool, pool, i, None, i.view(1, 2), i.view(1, 2), None, q)


# ------------------------------------------------------------------ oracle
def pool_of(rows):
    return np.asarray(rows, dtype=np.float64).reshape(2, 2, 1, 1)


def test_oracle_by_hand():
    # Rows 0..3 of the sequence have values 1, 2, 4, 8 (blocks swapped); equal scores: means.
    v, q = pool_of([4, 8, 1, 2]), np.zeros((5, 1, 1))
    out, size = gqa_prompt.attention(q, v * 0, v, [0, 3], [1], None, np.array([[1, 0]]), None, 1.0,
                                     np.full(q.shape, 7.0))
    assert np.allclose(out[:, 0, 0], [1.5, 7 / 3, 15 / 4, 7, 7]) and size[3, 0, 0] == 0
    # A token below the length sees less; nothing at all: 0.
    out, _ = gqa_prompt.attention(q, v * 0, v, [0, 3], [1], None, np.array([[1, 0]]), [2], 1.0, q)
    assert np.allclose(out[:3, 0, 0], [1.5, 1.5, 1.5])
    out, _ = gqa_prompt.attention(q, v * 0, v, [0, 3], [1], None, np.array([[1, 0]]), [0], 1.0, q + 7)
    assert np.allclose(out[:, 0, 0], [0, 0, 0, 7, 7])
    # A tree: the second and third token are both behind the first.
    mask = np.array([[1], [3], [5], [0], [0]])
    out, _ = gqa_prompt.attention(q, v * 0, v, [0, 3], [1], mask, np.array([[1, 0]]), None, 1.0, q)
    assert np.allclose(out[:3, 0, 0], [1.5, 7 / 3, 11 / 3])


def test_oracle_of_one_token_is_decode():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((2, 4, 64)), *rng.standard_normal((2, 6, 8, 2, 64))
    tab = rng.permutation(6).reshape(2, 3)
    ref, size = gqa_prefix.attention(q, k, v, None, None, None, tab, [20, 7], 0.3)
    got, size2 = gqa_prompt.attention(q, k, v, [0, 1, 2], [19, 6], None, tab, [20, 7], 0.3, q)
    assert np.allclose(ref, got) and np.allclose(size, size2)
    got, _ = gqa_prompt.attention(q, k, v, [0, 1, 2], [19, 6], [[1], [1]], tab, [20, 7], 0.3, q)
    assert np.allclose(ref, got)
    # Its own bit not set: only what is cached.
    ref, _ = gqa_prefix.attention(q, k, v, None, None, None, tab, [19, 6], 0.3)
    got, _ = gqa_prompt.attention(q, k, v, [0, 1, 2], [19, 6], [[0], [2]], tab, [20, 7], 0.3, q)
    assert np.allclose(ref, got)
