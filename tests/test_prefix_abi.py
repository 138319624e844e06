"""The calls of include/gqa_prefix.h: exported, bad arguments rejected on the
host before any CUDA call, and the oracle on hand-worked cases (CPU only)."""
import ctypes
import os
import re

import numpy as np
import pytest

from oracle import gqa_prefix

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gqa_prefix.h")
FAKE = 1 << 20  # a non-NULL 16-byte-aligned address that no rejected call touches


@pytest.fixture(scope="module")
def native():
    from gqa_attention_weighted_gb300 import build
    build.build()
    from gqa_attention_weighted_gb300 import _native
    return _native


def test_library_exports_every_declared_symbol(native):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"(gqa_prefix_\w+)\s*\(", text))
    assert {"gqa_prefix_attn_decode", "gqa_prefix_device_status"} <= names
    lib = ctypes.CDLL(native.LIBRARY)
    assert [n for n in sorted(names) if not hasattr(lib, n)] == []


CALL = dict(q=FAKE, k=FAKE, v=FAKE, ptab=FAKE, plen=FAKE, gs=FAKE, tab=FAKE, lens=FAKE, out=FAKE,
            B=2, P=1, Hq=8, Hkv=2, D=64, dt=0, bs=16, nb=8, mpb=4, mb=4, scale=0.125)


@pytest.mark.parametrize("change,status", [
    (dict(B=0), 1), (dict(P=-1), 1), (dict(Hq=0), 1), (dict(Hkv=-2), 1), (dict(D=0), 1),
    (dict(bs=0), 1), (dict(nb=0), 1), (dict(Hkv=3), 1), (dict(dt=2), 1), (dict(mb=-1), 1),
    (dict(mpb=0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(q=None), 1), (dict(k=None), 1), (dict(out=None), 1), (dict(ptab=None), 1),
    (dict(plen=None), 1), (dict(tab=None), 1), (dict(P=2, gs=None), 1), (dict(tab=FAKE + 2), 1),
    (dict(lens=FAKE + 1), 1), (dict(D=96), 2), (dict(D=512), 2), (dict(Hq=258), 2),
    (dict(bs=12), 2), (dict(bs=4), 2), (dict(B=4097), 2), (dict(P=129), 2), (dict(P=33), 2),
    (dict(B=4096, Hq=512, Hkv=512), 2),
    (dict(nb=1 << 27), 2), (dict(mb=1 << 27), 2),
    (dict(mb=(1 << 22) + 1), 2), (dict(mpb=(1 << 22) + 1), 2), (dict(q=FAKE + 8), 2), (dict(v=FAKE + 2), 2),
])
def test_host_checks(native, change, status):
    a = dict(CALL, **change)
    rc = native.lib.gqa_prefix_attn_decode(*a.values(), None)
    assert rc == status, native.lib.gqa_prefix_last_error()
    assert native.lib.gqa_prefix_last_error() != b""


def test_binding_rejects_tensors_that_do_not_fit(native):
    import torch
    pool = torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16)  # on the CPU
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k_pool"):
        native.gqa_prefix_attn_decode(q, pool, pool, None, None, None, None, None, q)


def test_oracle_is_one_softmax_over_prefix_and_own_rows():
    # Equal scores: the mean of the prefix's and the sequence's own values.
    pool = np.arange(2 * 8 * 1 * 2, dtype=np.float64).reshape(2, 8, 1, 2)
    q = np.zeros((2, 1, 2))
    out, _ = gqa_prefix.attention(q, pool, pool, np.array([[1]]), [2], [0, 1], np.array([[0], [0]]),
                                  [1, 3], 1.0)
    assert np.allclose(out[0, 0], (pool[1, 0, 0] + pool[1, 1, 0] + pool[0, 0, 0]) / 3)
    assert np.allclose(out[1, 0], pool[0, :3, 0].mean(0))   # in no group


def test_oracle_agrees_with_the_contiguous_one():
    from oracle import gqa_attn
    rng = np.random.default_rng(3)
    B, C, Hq, Hkv, D, bs = 2, 24, 4, 2, 64, 8
    k, v = (rng.standard_normal((B, C, Hkv, D)).astype(np.float16) for _ in "kv")
    q = rng.standard_normal((B, Hq, D)).astype(np.float32)
    lens = np.array([24, 10])
    ref = gqa_attn.gqa_attention(q, k.view(np.uint16), v.view(np.uint16), "fp16", lens, 0.3)
    pools = [x.astype(np.float64).reshape(B * C // bs, bs, Hkv, D) for x in (k, v)]
    table = np.arange(B * C // bs).reshape(B, -1)
    got, _ = gqa_prefix.attention(q.astype(np.float64), *pools, None, None, None, table, lens, 0.3)
    assert np.allclose(got, ref, atol=1e-12)
    # The same rows cut into a shared prefix of 8 and the rest.
    pools = [np.concatenate([x[:1, :8], x[:1, 8:16], x[:1, 16:]]).astype(np.float64)
             for x in (k, v)]
    one, _ = gqa_prefix.attention(q[:1].astype(np.float64), *pools, np.array([[0]]), [8], None,
                                  np.array([[1, 2]]), [16], 0.3)
    assert np.allclose(one[0], ref[0], atol=1e-12)


@pytest.mark.parametrize("wait_ns,withhold", [(99999, 0), (2000000001, 0), (-1, 0), (200000, -1)])
def test_selftest_host_checks(native, wait_ns, withhold):
    rc = native.lib.gqa_prefix_selftest_wait_timeout(*CALL.values(), wait_ns, withhold, None)
    assert rc == 1 and b"wait_ns" in native.lib.gqa_prefix_last_error()
    rc = native.lib.gqa_prefix_selftest_wait_timeout(*dict(CALL, D=96).values(), 200000, 0, None)
    assert rc == 2
