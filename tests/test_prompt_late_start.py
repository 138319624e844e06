"""Calls of gqa_prompt_attn and gqa_tree_attn whose CTAs are not all placed at once: none waits
for one that has not started, so late ones delay nothing but themselves, and calls on streams of
different priority, which take SMs from each other, all end with the bits of a call alone."""
import ctypes

import numpy as np
import pytest
import torch

from test_gpu_prompt import check, i32, make
from test_gpu_prompt_overlap import Job
from test_prompt_abi import PROMPT


@pytest.fixture(scope="module")
def gq():
    from gqa_attention_weighted_gb300 import build
    build.build()
    import gqa_attention_weighted_gb300 as pkg
    yield pkg
    if torch.cuda.is_available():
        pkg.gqa_prompt_device_status()


@pytest.mark.parametrize("wait_ns,late_from,late_ns", [(99999, 0, 0), (2000000001, 0, 0),
                                                       (200000, -1, 0), (200000, 0, -1),
                                                       (200000, 0, 2000000001)])
def test_host_checks(gq, wait_ns, late_from, late_ns):
    from gqa_attention_weighted_gb300 import _native
    rc = _native.lib.gqa_prompt_selftest_late_start(*PROMPT.values(), wait_ns, late_from, late_ns, None)
    assert rc == 1 and b"late_ns" in _native.lib.gqa_prompt_last_error()
    rc = _native.lib.gqa_prompt_selftest_late_start(*dict(PROMPT, D=96).values(), 200000, 0, 0, None)
    assert rc == 2


def late(x, out, wait_ns, late_from, late_ns):
    from gqa_attention_weighted_gb300 import _native
    t = {n: x[n].cuda() for n in "qkv"}
    t.update({n: i32(x[n]) for n in ("start", "cached", "tab", "lens")})
    T, Hq, D = t["q"].shape
    nb, bs, Hkv, _ = t["k"].shape
    ptr = [t[n].data_ptr() for n in ("k", "v", "start", "cached", "tab", "lens")]
    rc = _native.lib.gqa_prompt_selftest_late_start(
        t["q"].data_ptr(), t["q"].stride(0), *ptr, out.data_ptr(), len(x["cached"]), T, Hq, Hkv, D,
        _native.v_dtype_code(t["k"].dtype), bs, nb, t["tab"].shape[1], D ** -0.5, wait_ns, late_from,
        late_ns, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    torch.cuda.synchronize()


@pytest.mark.gpu
@pytest.mark.parametrize("late_from", [1, 60])
@pytest.mark.parametrize("items", ["few", "many"])
@pytest.mark.parametrize("D,Hkv", [(64, 2), (128, 2), (256, 1)])
def test_late_ctas_are_not_waited_for(gq, D, Hkv, items, late_from):
    # Items that are cut, in few items (every CTA makes the plan) and with room for more tokens
    # (one makes it). The late ones come 30 ms after the others, whose waits last 5 ms.
    x = make(np.random.default_rng(D), 4 * Hkv, Hkv, D, 16, "bf16", [9000, 20, 4000], [40, 3, 1],
             pad=3 if items == "few" else 33 * 128)
    want = check(gq, x)
    out = torch.full_like(want, 7.0)
    late(x, out, 5_000_000, late_from, 30_000_000)
    gq.gqa_prompt_device_status()
    assert torch.equal(out, want)


@pytest.mark.gpu
def test_streams_of_different_priority(gq):
    n = 60
    # Calls of cut items, of both plans, which alone fill the GPU.
    js = [Job(gq, n, 64, 8, 128, 16, "bf16", [2600, 130, 9000], [70, 200, 127]),
          Job(gq, n, 16, 1, 256, 64, "fp16", [30000, 63, 640], [40, 2, 9], tree=True),
          Job(gq, n, 8, 2, 64, 8, "bf16", [20000] + list(range(40)), [50] + [1 + i % 7 for i in range(40)]),
          Job(gq, n, 32, 8, 128, 16, "bf16", [16000], [13], tree=True)]
    low, high = 0, -2
    for order in ((low, high, low, high), (high, low, -1, low)):
        streams = [torch.cuda.Stream(priority=p) for p in order]
        for j in js:
            for o in j.outs:
                o.fill_(7.0)
        torch.cuda.synchronize()
        for i in range(n):
            for j, s in zip(js, streams):
                j.call(i, s)
        torch.cuda.synchronize()
        gq.gqa_prompt_device_status()
        for j in js:
            j.verify()
