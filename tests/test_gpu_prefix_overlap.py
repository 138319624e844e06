"""Calls of gqa_prefix_attn_decode that may overlap on the GPU (streams, host
threads, graph replays) give the bits of the same calls one after another."""
import gc
import threading

import numpy as np
import pytest
import torch

from test_gpu_prefix import check, i32, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    from gqa_attention_weighted_gb300 import build
    build.build()
    import gqa_attention_weighted_gb300 as pkg
    yield pkg
    pkg.gqa_prefix_device_status()


class Job:
    """A case on the GPU, its outputs for n calls, and what each should be."""

    def __init__(self, gq, n, *case):
        self.gq, x = gq, make(np.random.default_rng(len(case[6]) + case[3]), *case)
        self.want = check(gq, x)
        self.t = {m: x[m].cuda() for m in "qkv"}
        self.t.update({m: i32(x[m]) for m in ("ptab", "plens", "starts", "tab", "lens")})
        self.outs = [torch.zeros_like(self.want) for _ in range(n)]

    def call(self, i, stream=None):
        t = self.t
        self.gq.gqa_prefix_attn_decode(t["q"], t["k"], t["v"], t["ptab"], t["plens"], t["starts"],
                                       t["tab"], t["lens"], self.outs[i], stream=stream)

    def verify(self):
        assert [i for i, o in enumerate(self.outs) if not torch.equal(o, self.want)] == []


def jobs(gq, n):
    # Different head layouts, groups and unit counts: one call's plan fits none of the others.
    return [Job(gq, n, 70, 8, 2, 64, 8, "bf16", [200], [3, 66], list(range(70))),
            Job(gq, n, 9, 64, 8, 128, 16, "bf16", [2600, 130], [0, 4, 9], [127, 300, 0] * 3),
            Job(gq, n, 6, 16, 1, 256, 64, "fp16", [1700], None, [1, 63, 640, 65, 0, 9])]


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
    # Captured on one stream without a call on it before, replayed on others.
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
        assert not any(o.any() for o in j.outs), "a capture ran something"
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


def test_branches_of_one_capture(gq):
    a, b = jobs(gq, 1)[:2]
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        side.wait_stream(main)
        with torch.cuda.stream(side):
            b.call(0)
        a.call(0)
        main.wait_stream(side)
    for _ in range(10):
        g.replay()
    torch.cuda.synchronize()
    a.verify()
    b.verify()


def test_workspaces_of_captures_are_released(gq):
    j = jobs(gq, 1)[1]
    free = []
    for i in range(8):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            j.call(0)
        g.replay()
        torch.cuda.synchronize()
        j.verify()
        j.outs[0].zero_()
        del g
        gc.collect()
        if i >= 4:
            gq.gqa_prefix_release_graph_workspaces()
        free.append(torch.cuda.mem_get_info()[0])
    # A workspace of this case is above 40 MB: 152 SMs x 2 slots x 2 streams x 64 KB.
    assert free[0] - free[3] > 3 * 40e6 and free[4] > free[0], free
    j.call(0)                                     # uncaptured calls keep theirs
    torch.cuda.synchronize()
    j.verify()
