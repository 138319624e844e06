"""What captured calls of gqa_prompt_attn and gqa_tree_attn hold on the device (CUDA GPU)."""
import numpy as np
import pytest
import torch

from test_gpu_prompt import check, make
from test_gpu_prompt_overlap import on_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    from gqa_attention_weighted_gb300 import build
    build.build()
    import gqa_attention_weighted_gb300 as pkg
    yield pkg
    pkg.gqa_prompt_device_status()


def attend(gq, t, out):
    rest = (t["tab"], t["lens"], out)
    if t["mask"] is None:
        gq.gqa_prompt_attn(t["q"], t["k"], t["v"], t["start"], t["cached"], *rest)
    else:
        gq.gqa_tree_attn(t["q"], t["k"], t["v"], t["start"], t["cached"], t["mask"], *rest)


def test_graphs_of_small_calls_hold_little(gq):
    x = make(np.random.default_rng(0), 8, 2, 64, 16, "bf16", [500], [7], tree=True)
    want, t = check(gq, x), on_gpu(x)
    outs = [torch.full_like(want, 7.0) for _ in range(16)]
    gq.gqa_prompt_release_graph_workspaces()
    graphs = []
    before = None
    for i, out in enumerate(outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            attend(gq, t, out)
        graphs.append(g)
        g.replay()
        torch.cuda.synchronize()
        if i == 3:                               # graphs themselves have taken what they take by now
            before = torch.cuda.mem_get_info()[0]
    # 8 slots of 2 * 128 * 66 floats and some lists are 0.6 MB, and cudaMalloc takes 2 at a time.
    assert before - torch.cuda.mem_get_info()[0] <= 12 * 4 * 2 ** 20
    assert all(torch.equal(o, want) for o in outs)
    del graphs
    gq.gqa_prompt_release_graph_workspaces()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_capture_of_calls_that_need_more_and_more(gq, D):
    # Cut items of both calls, small ones first; pairs of query tiles among them.
    rng = np.random.default_rng(D)
    cases = [(4, 1, D, 16, "bf16", [30], [5]), (8, 2, D, 8, "bf16", [600, 900], [9, 40]),
             (8, 2, D, 16, "bf16", [3000, 40], [20, 70]),
             (4, 4, D, 32, "bf16", [6000] + [100] * 40, [33] + [3] * 40),
             (16, 4, D, 16, "bf16", [5000, 4500], [20, 17])]
    xs = [make(rng, *c, tree=tree) for c in cases for tree in (False, True)]
    wants, ts = [check(gq, x) for x in xs], [on_gpu(x) for x in xs]
    outs = [torch.full_like(w, 7.0) for w in wants]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for t, out in zip(ts, outs):
            attend(gq, t, out)
    for _ in range(3):
        for out in outs:
            out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        gq.gqa_prompt_device_status()
        for i, (out, want) in enumerate(zip(outs, wants)):
            assert torch.equal(out, want), i
    del g
    gq.gqa_prompt_release_graph_workspaces()
