"""gqa_kv_fork, gqa_kv_keep and gqa_kv_release: bad arguments rejected on the host
before any CUDA call (CPU only)."""
import ctypes

import pytest
import torch

AT = [(1 << 20) * (i + 1) for i in range(16)]   # distinct addresses that no rejected call touches


@pytest.fixture(scope="module")
def native():
    from gqa_attention_weighted_gb300 import build
    build.build()
    from gqa_attention_weighted_gb300 import _native
    return _native


FORK = dict(pools=(1 << 30, 1 << 31), row=64, parent=AT[0], child=AT[1], tab=AT[2], lens=AT[3],
            shares=AT[4], free=AT[5], count=AT[6], block=AT[7], left=AT[8], N=3, B=5, mb=4, nf=6,
            bs=16, nb=8)
KEEP = dict(pools=(1 << 30, 1 << 31), row=64, cached=AT[0], acc=AT[1], n=AT[2], tab=AT[3],
            lens=AT[4], kept=AT[5], B=5, W=3, mb=4, bs=16, nb=8)
RELEASE = dict(tab=AT[0], old=AT[1], new=AT[2], shares=AT[3], free=AT[4], count=AT[5], left=AT[6],
               B=5, mb=4, nf=6, bs=16, nb=8)


def call(native, fn, args):
    args = dict(args)
    if "pools" in args:
        pools = args.pop("pools")
        n = args.pop("np", len(pools) if pools is not None else 1)
        array = None if pools is None else (ctypes.c_void_p * max(1, len(pools)))(*pools)
        return getattr(native.lib, fn)(array, n, *args.values(), None)
    return getattr(native.lib, fn)(*args.values(), None)


POOLS = [
    (dict(pools=(1 << 30, None)), 1), (dict(pools=None), 1), (dict(row=0), 1), (dict(np=-1), 1),
    (dict(bs=0), 1), (dict(nb=-1), 1), (dict(B=0), 1), (dict(mb=0), 1),
    (dict(pools=(1 << 30, 1 << 30)), 1),                             # one pool twice
    (dict(pools=(1 << 30, (1 << 30) + 64 * 16 * 8 - 16)), 1),        # the last row of one in the other
    (dict(pools=((1 << 30) + 8,)), 2), (dict(row=24), 2), (dict(row=(1 << 20) + 16), 2),
    (dict(pools=(1 << 30,) * 257), 2), (dict(nb=1 << 27), 2), (dict(B=8193), 2), (dict(mb=1 << 27), 2),
]


@pytest.mark.parametrize("change,status", POOLS + [
    (dict(N=-1), 1), (dict(nf=-1), 1), (dict(N=8193), 2), *[(dict([(n, None)]), 1) for n in
     ("parent", "child", "tab", "lens", "shares", "free", "count", "block", "left")],
    *[(dict([(n, AT[9] + 2)]), 1) for n in ("parent", "tab", "shares", "block")],
    (dict(lens=AT[2] + 76), 1), (dict(left=AT[6]), 1), (dict(block=AT[0] + 8), 1),
    (dict(tab=AT[5] - 76), 1), (dict(left=AT[4] + 28), 1)])
def test_fork_host_checks(native, change, status):
    rc = call(native, "gqa_kv_fork", dict(FORK, **change))
    assert rc == status and native.lib.gqa_kv_last_error() != b"", native.lib.gqa_kv_last_error()


@pytest.mark.parametrize("change,status", POOLS + [
    (dict(pools=(), np=0), 1), (dict(W=-1), 1), (dict(W=(1 << 20) + 1), 2),
    *[(dict([(n, None)]), 1) for n in ("cached", "acc", "n", "tab", "lens", "kept")],
    *[(dict([(n, AT[9] + 2)]), 1) for n in ("cached", "acc", "n", "tab", "lens", "kept")],
    (dict(kept=AT[4]), 1), (dict(kept=AT[0] + 16), 1), (dict(kept=AT[1] + 56), 1)])
def test_keep_host_checks(native, change, status):
    rc = call(native, "gqa_kv_keep", dict(KEEP, **change))
    assert rc == status and native.lib.gqa_kv_last_error() != b"", native.lib.gqa_kv_last_error()


@pytest.mark.parametrize("change,status", [
    (dict(B=0), 1), (dict(mb=0), 1), (dict(nf=-1), 1), (dict(bs=0), 1), (dict(nb=0), 1),
    (dict(B=8193), 2), (dict(B=8192, mb=1 << 17, bs=1), 2), (dict(mb=1 << 27), 2), (dict(nb=1 << 27), 2),
    *[(dict([(n, None)]), 1) for n in ("tab", "old", "new", "free", "count", "left")],
    *[(dict([(n, AT[9] + 2)]), 1) for n in ("tab", "old", "new", "shares", "free", "count", "left")],
    (dict(left=AT[5]), 1), (dict(shares=AT[0] + 76), 1), (dict(free=AT[1] - 20), 1),
    (dict(free=AT[3] + 28), 1)])
def test_release_host_checks(native, change, status):
    rc = call(native, "gqa_kv_release", dict(RELEASE, **change))
    assert rc == status and native.lib.gqa_kv_last_error() != b"", native.lib.gqa_kv_last_error()


def test_bindings_refuse_what_does_not_fit(native):
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="pools"):
        native.KvPools([])
    with pytest.raises(ValueError, match=r"pools\[0\]"):
        native.KvPools([torch.zeros((2, 16, 64))])             # on the CPU
    with pytest.raises(ValueError, match="block_table"):
        native.gqa_kv_release(i.view(1, 2), i, i, None, i, i, i, block_size=16, num_blocks=4)
    with pytest.raises(ValueError, match="num_blocks"):
        native.gqa_kv_release(i.view(1, 2), i, i, None, i, i, i, block_size=16)
