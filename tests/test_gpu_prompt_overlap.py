"""Calls of gqa_prompt_attn and gqa_tree_attn that may overlap on the GPU (streams,
host threads, graph replays) give the bits of the same calls one after another;
graphs follow lengths; a wait that runs out is reported and the next call is correct."""
import ctypes
import threading

import numpy as np
import pytest
import torch

from test_gpu_prompt import check, i32, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    from gqa_attention_weighted_gb300 import build
    build.build()
    import gqa_attention_weighted_gb300 as pkg
    yield pkg
    pkg.gqa_prompt_device_status()


def on_gpu(x):
    t = {m: x[m].cuda() for m in "qkv"}
    t.update({m: i32(x[m]) for m in ("start", "cached", "mask", "tab", "lens")})
    return t


class Job:
    """A case on the GPU, its outputs for n calls, and what each should be."""

    def __init__(self, gq, n, *case, tree=False):
        self.gq, x = gq, make(np.random.default_rng(len(case[5]) + case[2]), *case, tree=tree)
        self.want = check(gq, x)
        self.t = on_gpu(x)
        self.outs = [torch.full_like(self.want, 7.0) for _ in range(n)]

    def call(self, i, stream=None):
        t = self.t
        rest = (t["tab"], t["lens"], self.outs[i])
        if t["mask"] is None:
            self.gq.gqa_prompt_attn(t["q"], t["k"], t["v"], t["start"], t["cached"], *rest, stream=stream)
        else:
            self.gq.gqa_tree_attn(t["q"], t["k"], t["v"], t["start"], t["cached"], t["mask"], *rest,
                                  stream=stream)

    def verify(self):
        assert [i for i, o in enumerate(self.outs) if not torch.equal(o, self.want)] == []


def jobs(gq, n):
    # Head layouts, unit counts and cuts that differ: one call's plan fits none of the others.
    return [Job(gq, n, 8, 2, 64, 8, "bf16", list(range(40)), [1 + i % 7 for i in range(40)]),
            Job(gq, n, 64, 8, 128, 16, "bf16", [2600, 130, 0], [70, 200, 127]),
            Job(gq, n, 16, 1, 256, 64, "fp16", [3000, 63, 640], [40, 2, 9], tree=True)]


def test_streams_in_flight_together(gq):
    js = jobs(gq, 40)
    streams = [torch.cuda.Stream() for _ in js]
    torch.cuda.synchronize()
    for i in range(40):
        for j, s in zip(js, streams):
            j.call(i, s)
    torch.cuda.synchronize()
    for j in js:
        j.verify()


def test_host_threads_on_streams_of_their_own_and_on_one(gq):
    for shared in (False, True):
        js = jobs(gq, 40)
        one = torch.cuda.Stream()
        torch.cuda.synchronize()

        def work(j, s):
            for i in range(40):
                j.call(i, s)

        threads = [threading.Thread(target=work, args=(j, one if shared else torch.cuda.Stream()))
                   for j in js]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        for j in js:
            j.verify()


def test_graphs_replayed_together_beside_calls(gq):
    js = jobs(gq, 3)
    graphs = []
    capture = torch.cuda.Stream()
    torch.cuda.synchronize()
    for j in js:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=capture):
            j.call(0)
            j.call(1)
        graphs.append(g)
    for j in js:
        assert all((o == 7.0).all() for o in j.outs), "a capture ran something"
    streams = [torch.cuda.Stream() for _ in js]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        for j in js:
            j.call(2)
    torch.cuda.synchronize()
    for j in js:
        j.verify()
    del graphs
    gq.gqa_prompt_release_graph_workspaces()
    js[0].call(2)                                 # uncaptured calls keep theirs
    torch.cuda.synchronize()
    js[0].verify()


def test_a_graph_follows_lengths(gq):
    x = make(np.random.default_rng(4), 32, 8, 128, 16, "bf16", [900, 40, 0], [60, 100, 40])
    t = on_gpu(x)
    out = torch.full(x["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gq.gqa_prompt_attn(t["q"], t["k"], t["v"], t["start"], t["cached"], t["tab"], t["lens"], out)
    for start, cached, lens in (([0, 60, 160, 200], [900, 40, 0], [960, 140, 40]),
                                ([0, 1, 1, 9], [17, 0, 12], [18, 0, 20]),
                                ([30, 30, 30, 30], [0, 0, 0], [9, 9, 9]),
                                ([0, 200, 200, 200], [700, 0, 0], [900, 0, 0])):
        y = dict(x, start=np.array(start), cached=cached, lens=lens)
        for n in ("start", "cached", "lens"):
            t[n].copy_(i32(y[n]))
        out.fill_(7.0)
        g.replay()
        want = check(gq, y)
        assert torch.equal(out, want)
    del g
    gq.gqa_prompt_release_graph_workspaces()


def test_offsets_past_32_bits(gq):
    # Pools of 2.3 GB each: the sequences lie in their last blocks.
    nb, bs, Hkv, D = 18000, 64, 8, 128
    k, v = (torch.zeros((nb, bs, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    x = make(np.random.default_rng(5), 16, Hkv, D, bs, "bf16", [300, 0], [20, 70])
    n = x["k"].shape[0]
    k[nb - n:], v[nb - n:] = x["k"].cuda(), x["v"].cuda()
    want = check(gq, x)
    t = on_gpu(x)
    out = torch.full_like(want, 7.0)
    tab = torch.where((t["tab"] >= 0) & (t["tab"] < n), t["tab"] + nb - n, 0)
    gq.gqa_prompt_attn(t["q"], k, v, t["start"], t["cached"], tab, t["lens"], out)
    assert torch.equal(out, want)


def test_largest_batches(gq):
    x = make(np.random.default_rng(6), 4, 1, 64, 8, "bf16", [i % 3 for i in range(8192)],
             [i % 2 for i in range(8192)], tree=True)
    check(gq, x)
    x["mask"] = None
    check(gq, x)


# ------------------------------------------------------- waits that run out
def selftest(t, out, withhold_from, wait_ns=200_000):
    from gqa_attention_weighted_gb300 import _native
    T, Hq, D = t["q"].shape
    nb, bs, Hkv, _ = t["k"].shape
    ptr = [t[n].data_ptr() for n in ("k", "v", "start", "cached", "tab", "lens")]
    return _native.lib.gqa_prompt_selftest_wait_timeout(
        t["q"].data_ptr(), t["q"].stride(0), *ptr, out.data_ptr(), len(t["cached"]), T, Hq, Hkv, D,
        _native.v_dtype_code(t["k"].dtype), bs, nb, t["tab"].shape[1], D ** -0.5, wait_ns, withhold_from,
        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))


def timed_out(gq, clear):
    try:
        gq.gqa_prompt_device_status(clear=clear)
    except gq.GqaAvError as e:
        assert "ran out" in str(e)
        return True
    return False


@pytest.mark.parametrize("withhold_from", [0, 1])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_wait_that_runs_out_is_reported_and_cleared(gq, D, withhold_from):
    # 4 KV heads x 60 sequences: more units than SMs, so some CTA loads queries twice.
    x = make(np.random.default_rng(D), 16, 4, D, 16, "bf16", [5 * i for i in range(60)], [1 + i % 9 for i in
                                                                                   range(60)])
    want = check(gq, x)
    t = on_gpu(x)
    assert selftest(t, torch.empty_like(want), withhold_from) == 0
    assert timed_out(gq, clear=False)            # reported, and still reported
    assert timed_out(gq, clear=True)
    assert not timed_out(gq, clear=False)
    assert torch.equal(check(gq, x), want)       # the context and the header are intact
