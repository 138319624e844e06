"""The calls of include/gqa_kv.h: exported, and bad arguments rejected on the
host before any CUDA call (CPU only)."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gqa_kv.h")
FAKE = 1 << 20  # a non-NULL 16-byte-aligned address that no rejected call touches


@pytest.fixture(scope="module")
def native():
    from gqa_attention_weighted_gb300 import build
    build.build()
    from gqa_attention_weighted_gb300 import _native
    return _native


def test_library_exports_every_declared_symbol(native):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"(gqa_kv_\w+)\s*\(", text))
    assert {"gqa_kv_tables", "gqa_kv_norm_rope_append", "gqa_kv_last_error"} <= names
    lib = ctypes.CDLL(native.LIBRARY)
    assert [n for n in sorted(names) if not hasattr(lib, n)] == []


TABLES = dict(cached=FAKE, new=FAKE, base=None, free=FAKE, count=FAKE, table=FAKE, seq=FAKE + 64,
              start=FAKE, slots=FAKE, pos=FAKE, left=FAKE + 128, B=4, T=8, max_blocks=4, n_free=4,
              bs=16, nb=8)


@pytest.mark.parametrize("change,status", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(max_blocks=0), 1), (dict(n_free=-1), 1),
    (dict(bs=0), 1), (dict(nb=0), 1), (dict(cached=None), 1), (dict(count=None), 1),
    (dict(free=None), 1), (dict(slots=None), 1), (dict(left=None), 1),
    (dict(table=FAKE + 2), 1), (dict(base=FAKE + 1), 1),
    (dict(seq=FAKE), 1),                      # seq_lens is cached_lens
    (dict(left=FAKE), 1),                     # free_left is free_count
    (dict(bs=1 << 16, nb=1 << 16), 2), (dict(B=8193), 2),
])
def test_tables_host_checks(native, change, status):
    a = dict(TABLES, **change)
    rc = native.lib.gqa_kv_tables(*a.values(), None)
    assert rc == status, native.lib.gqa_kv_last_error()
    assert native.lib.gqa_kv_last_error() != b""


ROPE = dict(q=FAKE, k=FAKE, v=FAKE, qs=512, ks=128, vs=128, pos=FAKE, sec=None, axes=1, inv=FAKE,
            qw=FAKE, kw=FAKE, eps=1e-6, off=0.0, inter=0, slots=FAKE, q_out=FAKE, od=0, kp=FAKE,
            vp=FAKE, T=4, Hq=8, Hkv=2, D=64, rot=64, dt=0, bs=16, nb=8)
SEC = ctypes.c_int * 3


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(D=0), 1), (dict(dt=2), 1),
    (dict(od=1), 1), (dict(od=3), 1), (dict(bs=0), 1), (dict(nb=-1), 1),
    (dict(D=60), 2), (dict(D=264), 2), (dict(rot=-16), 1), (dict(rot=80), 1), (dict(rot=24), 2),
    (dict(rot=20, inter=1), 2), (dict(axes=0), 1), (dict(axes=5), 1), (dict(axes=3), 1),
    (dict(axes=3, sec=SEC(8, 8, 8)), 1), (dict(axes=3, sec=SEC(-8, 20, 20)), 1),
    (dict(eps=float("nan")), 1), (dict(eps=-1.0), 1), (dict(off=float("inf")), 1),
    (dict(q=None), 1), (dict(slots=None), 1), (dict(inv=None), 1), (dict(pos=None), 1),
    (dict(vp=None), 1), (dict(slots=FAKE + 2), 1), (dict(q=FAKE + 8), 2), (dict(kw=FAKE + 2), 2),
    (dict(qs=516), 2), (dict(qs=504), 1), (dict(vs=0), 1), (dict(bs=1 << 16, nb=1 << 15), 2),
])
def test_norm_rope_host_checks(native, change, status):
    a = dict(ROPE, **change)
    rc = native.lib.gqa_kv_norm_rope_append(*a.values(), None)
    assert rc == status, native.lib.gqa_kv_last_error()
    assert native.lib.gqa_kv_last_error() != b""


def test_no_tokens_is_not_an_error(native):
    a = dict(ROPE, T=0, q=None, k=None, v=None, slots=None)
    assert native.lib.gqa_kv_norm_rope_append(*a.values(), None) == 0


def test_binding_rejects_tensors_that_do_not_fit(native):
    import torch
    t = torch.zeros((2, 4), dtype=torch.int32)  # on the CPU
    with pytest.raises(ValueError, match="block_table"):
        native.gqa_kv_tables(t[0], t[0], t[0], t[0], t, t[0], t[0], t[0], t[0], t[0], 16, 8)
    pool = torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16)
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k_pool"):
        native.gqa_kv_norm_rope_append(x, x, x, t[0], t[0], t[0], x, pool, pool)


INS = dict(cached=4, new=4, base=4, free=4, count=1)        # entries of each
OUTS = dict(table=16, seq=4, start=5, slots=8, pos=8, left=1)


def apart():
    """The call's arrays behind one another: nothing overlaps."""
    a, at = dict(TABLES), FAKE
    for name, n in (INS | OUTS).items():
        a[name], at = at, at + 4 * n
    return a


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("inp", INS)
def test_tables_outputs_must_not_overlap_inputs(native, inp, out):
    for shift in (0, 4 * (INS[inp] - 1), 4 - 4 * OUTS[out]):   # the same, and by one entry
        a = apart()
        a[out] = a[inp] + shift
        assert native.lib.gqa_kv_tables(*a.values(), None) == 1
        assert b"overlaps" in native.lib.gqa_kv_last_error(), native.lib.gqa_kv_last_error()
