"""Prompts, forks, drafted steps, kept paths and releases as the example runs them, the
steps replayed from a graph, against the fp64 oracles chained the same way."""
import os
import random
import sys

import numpy as np
import pytest
import torch

from oracle import gqa_kv, gqa_prompt

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


@pytest.mark.parametrize("Hq,Hkv,D,block", [(8, 2, 64, 8), (6, 2, 128, 16)])
def test_a_life_of_requests_matches_the_oracles(Hq, Hkv, D, block):
    from gqa_attention_weighted_gb300 import build
    build.build()
    import draft_steps as ex
    import gqa_attention_weighted_gb300 as gq
    parents, copies, layers, steps = 2, 2, 2, 7
    lens = [37, 130]
    s = ex.Server(parents, copies, layers, Hq, Hkv, D, block, max_rows=200, width=2, depth=3)
    g, rng = torch.Generator(device="cuda").manual_seed(3), random.Random(4)
    inv = s.inv_freq.cpu().numpy()
    eps = torch.finfo(torch.bfloat16).eps

    def draw(n):
        return torch.randn((layers, n, (Hq + 2 * Hkv) * D), generator=g, device="cuda").bfloat16()

    def heads(x, a, b):
        return x[:, a * D:b * D].reshape(len(x), b - a, D)

    def turn(x, a, b, pos):
        return gqa_kv.norm_rotate(heads(x, a, b), np.ones(D), 1e-6, 0.0, [np.asarray(pos)], inv,
                                  [D // 2], False)[0]

    def check(made, tokens, rows, mask, new):
        """Layers' queries and outputs of sequences with `new` tokens each behind `rows[b]`, the
        lists of (token's projections, position) of their cached rows."""
        for layer, (q, out) in enumerate(made):
            q, out = q.double().cpu().numpy(), out.double().cpu().numpy()
            t = 0
            for b, n in enumerate(new):
                if n == 0:
                    continue
                mine = tokens[layer][t:t + n]
                pos = [len(rows[b]) + d for d in (s.depths.tolist() if mask is not None else range(n))]
                old = np.array([x[layer] for x, _ in rows[b]]).reshape(-1, mine.shape[1])
                allx = np.concatenate([old, mine])
                at = [p for _, p in rows[b]] + pos
                assert at[:len(old)] == list(range(len(old)))
                k, v = turn(allx, Hq, Hq + Hkv, at)[None], heads(allx, Hq + Hkv, Hq + 2 * Hkv)[None]
                want_q = turn(mine, 0, Hq, pos)
                assert (np.abs(q[t:t + n] - want_q) <= eps / 2 * np.abs(want_q) + 1e-5 * D ** 0.5).all()
                # The oracle from the queries that the step rounded, and keys that it did not: a
                # score is off by eps/2 sum |q k| / sqrt(D), at most eps/2 sqrt(D) (both normed);
                # weights by twice that, by half a step, and the output by half a step.
                ref, size = gqa_prompt.attention(q[t:t + n], k, v, [0, n], [len(old)],
                                                 None if mask is None else mask[:n],
                                                 np.array([[0]]), None, D ** -0.5, q[t:t + n])
                tol = eps / 2 * np.abs(ref) + (eps / 2 + 2 * eps / 2 * D ** 0.5) * size + 1e-5
                assert (np.abs(out[t:t + n] - ref) <= tol).all(), (layer, b)
                t += n

    rows = [[] for _ in range(s.B)]
    x = draw(sum(lens))
    made = s.prompts(lens, x)
    tokens = x.double().cpu().numpy()
    new = [0] * s.B
    new[::s.step_rows] = lens
    check(made, tokens, rows, None, new)
    t = 0
    for b, n in enumerate(new):
        rows[b] = [(tokens[:, t + i], i) for i in range(n)]
        t += n
    served = s.fork().tolist()
    assert all((x >= 0) if len(rows[b - b % s.step_rows]) % block else (x == -1) for x, b in
               zip(served, [b for b in range(s.B) if b % s.step_rows]))
    for b in range(s.B):
        rows[b] = list(rows[b - b % s.step_rows])
    mask = s.mask.cpu().numpy()[:s.drafts]
    qkv = draw(s.B * s.drafts)
    graph, made = None, None
    for step in range(steps):
        qkv.copy_(draw(s.B * s.drafts))
        paths = s.accept(rng)
        if step == 0:
            made = s.step(qkv)
        elif step == 1:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                made = s.step(qkv)
            graph.replay()
        else:
            graph.replay()
        gq.gqa_prompt_device_status()
        tokens = qkv.double().cpu().numpy()
        check(made, tokens, rows, mask, [s.drafts] * s.B)
        for b, path in enumerate(paths):
            rows[b] += [(tokens[:, b * s.drafts + a], len(rows[b]) + i) for i, a in enumerate(path)]
        assert s.cached.tolist() == [len(r) for r in rows]
        # Every block is free or has as many owners as its count says.
        owners = np.zeros(s.num_blocks, dtype=int)
        table = s.block_table.tolist()
        for b, r in enumerate(rows):
            for x in table[b][:-(-len(r) // block)]:
                owners[x] += 1
        free = s.free_list[:s.free_count.item()].tolist()
        assert sorted(free) == [x for x in range(s.num_blocks) if owners[x] == 0]
        assert [max(0, n - 1) for n in owners] == s.shares.tolist()
    assert s.end() == s.num_blocks and sorted(s.free_list.tolist()) == list(range(s.num_blocks))
    assert s.shares.sum().item() == 0
    del graph
    gq.gqa_prompt_release_graph_workspaces()


def test_the_example_runs():
    import draft_steps as ex
    assert ex.main(steps=3, parents=2, copies=1, layers=1, Hq=8, Hkv=2, D=64)
