"""A bounded wait inside the shared-prefix attention kernel that runs out is
reported, whatever workspace the call ran in, and the next call is correct
(failure detection without a GPU fault).

gqa_prefix_selftest_wait_timeout runs the kernel with its waits limited to
200 us and query loads that are never issued: the MMA warp's wait for them runs
out, the other roles' waits follow, each waits for what it has in flight, sets
the status word and leaves.
"""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from test_gpu_prefix import check, i32, make

pytestmark = pytest.mark.gpu

WAIT_NS = 200_000


@pytest.fixture(scope="module")
def gq():
    from gqa_attention_weighted_gb300 import build
    build.build()
    import gqa_attention_weighted_gb300 as pkg
    pkg.gqa_prefix_device_status()
    return pkg


def case(D, rng):
    # 4 KV heads x 60 sequences: more own units than SMs, so some CTA loads queries twice.
    return make(rng, 60, 16, 4, D, 16, "bf16", [900], None, [1 + 5 * i for i in range(60)])


def on_gpu(x):
    d = {n: x[n].cuda() for n in "qkv"}
    d.update({n: i32(x[n]) for n in ("ptab", "plens", "starts", "tab", "lens")})
    d["out"] = torch.zeros_like(d["q"])
    return d


def selftest(d, withhold_from, wait_ns=WAIT_NS):
    from gqa_attention_weighted_gb300 import _native
    ptr = [None if d[n] is None else d[n].data_ptr()
           for n in ("q", "k", "v", "ptab", "plens", "starts", "tab", "lens", "out")]
    B, Hq, D = d["q"].shape
    nb, bs, Hkv, _ = d["k"].shape
    return _native.lib.gqa_prefix_selftest_wait_timeout(
        *ptr, B, len(d["plens"]), Hq, Hkv, D, _native.v_dtype_code(d["k"].dtype), bs, nb,
        d["ptab"].shape[1], d["tab"].shape[1], D ** -0.5, wait_ns, withhold_from,
        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))


def timed_out(gq, clear):
    try:
        gq.gqa_prefix_device_status(clear=clear)
    except gq.GqaAvError as e:
        assert "ran out" in str(e)
        return True
    return False


@pytest.mark.parametrize("withhold_from", [0, 1])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_wait_that_runs_out_is_reported_and_cleared(gq, D, withhold_from):
    x = case(D, np.random.default_rng(D))
    check(gq, x)
    assert selftest(on_gpu(x), withhold_from) == 0
    assert timed_out(gq, clear=False)            # reported, and still reported
    assert timed_out(gq, clear=True)
    assert not timed_out(gq, clear=False)
    check(gq, x)                                 # the context and the unit counter are intact


def child():
    """In a process of its own, whose first workspace is a small one."""
    import gqa_attention_weighted_gb300 as gq
    rng = np.random.default_rng(1)
    small = on_gpu(make(rng, 2, 4, 2, 64, 16, "bf16", [40], None, [3, 20]))
    large = make(rng, 300, 64, 8, 128, 16, "bf16", [140], None, [3] * 300)
    check(gq, make(rng, 2, 4, 2, 64, 16, "bf16", [40], None, [3, 20]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert selftest(small, 0) == 0
    assert selftest(small, 0) == 0
    torch.cuda.synchronize()
    d = on_gpu(large)                            # outgrows the workspace, before any status is read
    gq.gqa_prefix_attn_decode(d["q"], d["k"], d["v"], d["ptab"], d["plens"], d["starts"], d["tab"],
                              d["lens"], d["out"])
    assert timed_out(gq, clear=True), "lost by the growth"
    check(gq, large)
    graph.replay()                               # in the workspace from before the growth
    assert timed_out(gq, clear=True), "lost in the outgrown workspace"
    check(gq, large)
    print("status ok")


def test_reports_survive_a_workspace_that_grows():
    from gqa_attention_weighted_gb300 import build
    build.build()
    here = os.path.dirname(os.path.abspath(__file__))
    code = (f"import sys; sys.path[:0] = [{here!r}, {os.path.dirname(here)!r}]; "
            "import test_gpu_prefix_timeout as t; t.child()")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "status ok" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
