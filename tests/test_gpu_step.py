"""The paged serving step as the example runs it, replayed from a graph, against
the fp64 oracles chained the same way."""
import os
import sys

import numpy as np
import pytest
import torch

from oracle import gqa_kv, gqa_prefix

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


def test_steps_from_a_graph_match_the_oracles():
    from gqa_attention_weighted_gb300 import build
    build.build()
    import shared_prefix_steps as ex
    B, Hq, Hkv, D, bs, rows, steps = 5, 8, 2, 64, 8, 150, 12
    g = torch.Generator(device="cuda").manual_seed(3)

    def draw(n):
        return torch.randn((n, (Hq + 2 * Hkv) * D), generator=g, device="cuda").bfloat16()

    batch = ex.PagedSteps(B, Hq, Hkv, D, bs, rows, steps + 1)
    prefix = draw(rows)
    batch.prefill_prefix(prefix)
    qkv = draw(B)
    batch.step(qkv)
    batch.reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        batch.step(qkv)
    tokens, outs, queries = [], [], []
    for _ in range(steps):
        qkv.copy_(draw(B))
        graph.replay()
        tokens.append(qkv.double().cpu().numpy())
        outs.append(batch.out.double().cpu().numpy())
        queries.append(batch.q.double().cpu().numpy())
    inv = batch.inv_freq.cpu().numpy()

    def heads(x, a, b):
        return x[:, a * D:b * D].reshape(len(x), b - a, D)

    def keys(x, pos):
        return gqa_kv.norm_rotate(heads(x, Hq, Hq + Hkv), np.ones(D), 1e-6, 0.0, [pos], inv,
                                  [D // 2], False)[0]

    pre = prefix.double().cpu().numpy()
    pk, pv = keys(pre, np.arange(rows)), heads(pre, Hq + Hkv, Hq + 2 * Hkv)
    eps = torch.finfo(torch.bfloat16).eps
    for s in range(steps):
        own_k = np.stack([keys(t, np.full(B, rows + i)) for i, t in enumerate(tokens[:s + 1])], 1)
        own_v = np.stack([heads(t, Hq + Hkv, Hq + 2 * Hkv) for t in tokens[:s + 1]], 1)
        ref_q, size_q = gqa_kv.norm_rotate(heads(tokens[s], 0, Hq), np.ones(D), 1e-6, 0.0,
                                           [np.full(B, rows + s)], inv, [D // 2], False)
        assert (np.abs(queries[s] - ref_q) <= eps / 2 * np.abs(ref_q) + 4e-6 * size_q).all()
        for b in range(B):
            k, v = np.concatenate([pk, own_k[b]]), np.concatenate([pv, own_v[b]])
            n = len(k)
            pool = [x[None] for x in (k, v)]
            # The oracle from the queries that the step rounded, and keys that it did not.
            ref, size = gqa_prefix.attention(queries[s][b:b + 1], *pool, None, None, None,
                                             np.array([[0]]), [n], D ** -0.5)
            # Keys rounded to bf16: a score is off by eps/2 sum |q k| / sqrt(D), at most
            # eps/2 |q| |k| / sqrt(D) = eps/2 sqrt(D) (both normed); weights by twice that,
            # by half a step, and the output by half a step.
            tol = eps / 2 * np.abs(ref) + (eps / 2 + 2 * eps / 2 * D ** 0.5) * size + 1e-5
            assert (np.abs(outs[s][b:b + 1] - ref) <= tol).all(), (s, b)
    assert batch.seq_lens.tolist() == [steps] * B
    assert batch.free_left.item() == B * batch.max_blocks - B * -(-steps // bs)
