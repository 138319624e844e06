"""GPU parity of the calls of include/gqa_kv.h against their oracles."""
import numpy as np
import pytest
import torch

from helpers import TORCH_V
from oracle import gqa_kv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    from gqa_attention_weighted_gb300 import build
    build.build()
    import gqa_attention_weighted_gb300 as pkg
    return pkg


def i32(x):
    return torch.tensor(np.array(x, order="C", copy=True).astype(np.int32), device="cuda")


def run_tables(gq, cached, new, free_list, free_count, table, T, bs, nb, base=None):
    dev = "cuda"
    B = len(cached)
    tab = i32(table)
    out = [torch.full((n,), -77, dtype=torch.int32, device=dev) for n in (B, B + 1, T, T, 1)]
    gq.gqa_kv_tables(i32(cached), i32(new), i32(free_list), i32([free_count]), tab, *out,
                     block_size=bs, num_blocks=nb, pos_base=None if base is None else i32(base))
    ref = gqa_kv.tables(cached, new, free_list, free_count, table, T, bs, nb, base)
    for name, g, r in zip(("table", "seq_lens", "token_start", "slots", "positions", "free_left"),
                          [tab] + out, ref):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(r).reshape(-1)), name


@pytest.mark.parametrize("B", [1, 3, 511, 513, 1500])
@pytest.mark.parametrize("bs", [1, 16, 48])
@pytest.mark.parametrize("short", [0, 1, 2], ids=["enough", "short", "none"])
def test_tables_match_the_oracle(gq, B, bs, short):
    rng = np.random.default_rng(B * 100 + bs + short)
    cached = rng.integers(0, 200, size=B)
    new = rng.integers(0, 40, size=B) * (rng.random(B) < 0.8)
    held, want = -(-cached // bs), -(-(cached + new) // bs)
    need = int((want - held).sum())
    max_blocks = int(want.max()) + 1
    nb = int(held.sum()) + need + 5
    perm = rng.permutation(nb)
    table = rng.integers(-3, nb + 3, size=(B, max_blocks))   # past a length: anything
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    count = (need, need // 2, 0)[short]
    T = int(new.sum()) + int(rng.integers(0, 70))
    run_tables(gq, cached, new, perm[at:], count, table, T, bs, nb,
               rng.integers(0, 10000, size=B) if B != 3 else None)


def test_tables_odd_inputs(gq):
    # Negative lengths, a count past the list, entries outside the pool, a request past
    # max_blocks, and tokens that end past T (T = 6): those requests are not served.
    run_tables(gq, [-5, 9, 2, 0, 0], [2, 1, -1, 1, 9], [1, 99, -4], 50,
               [[0, 0], [3, 4], [2, 2], [0, 0], [0, 0]], 6, 4, 8)
    run_tables(gq, [3], [0], [], 0, [[5]], 0, 4, 8)           # nothing new, no list, no tokens
    run_tables(gq, [0], [1], [], 0, [[5]], 1, 4, 8)           # no free block at all


def test_tables_long_request_spans_many_ctas(gq):
    run_tables(gq, [5, 0], [9000, 3], np.arange(700)[::-1].copy(), 700, np.zeros((2, 600)), 9003,
               16, 700, [0, 7])


ROPE = [
    # T, Hq, Hkv, D, rot, sections, norm, interleaved, q32
    (1, 8, 2, 64, 64, [32], True, False, True),
    (5, 32, 8, 128, 128, [64], True, False, False),
    (3, 24, 8, 128, 64, [32], False, False, True),
    (7, 16, 1, 256, 256, [32, 48, 48], True, True, False),
    (4, 3, 1, 72, 32, [0, 16], True, False, False),
    (6, 5, 5, 8, 8, [4], True, True, True),
    (2, 4, 2, 24, 0, [0], True, False, False),
    (33, 4, 4, 248, 240, [100, 10, 5, 5], False, False, False),
    (40, 7, 1, 40, 24, [12], False, True, True),
    (20000, 2, 1, 64, 64, [32], True, False, False),
]


@pytest.mark.parametrize("vd", ["bf16", "fp16"])
@pytest.mark.parametrize("case", ROPE, ids=[f"T{c[0]}-D{c[3]}-rot{c[4]}-{'i' if c[7] else 's'}"
                                            for c in ROPE])
def test_norm_rope_append_matches_the_oracle(gq, case, vd):
    T, Hq, Hkv, D, rot, sections, norm, interleaved, q32 = case
    rng = np.random.default_rng(T + D)
    dt, dev = TORCH_V[vd], "cuda"
    bs = 16
    nb = -(-T // bs) + 2
    qkv = torch.tensor(rng.standard_normal((T, (Hq + 2 * Hkv) * D)) * 3, dtype=torch.float32).to(dt)
    cut = [Hq * D, Hkv * D, Hkv * D]
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.to(dev).split(cut, dim=1))
    qc, kc, vc = (x.unflatten(1, (-1, D)).double().numpy() for x in qkv.split(cut, dim=1))
    qw, kw = ((torch.tensor(rng.standard_normal(D), dtype=torch.float32).to(dt) for _ in "qk")
              if norm else (None, None))
    pos = rng.integers(0, 1 << 20, size=(len(sections), T))
    inv = (10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)
    slots = rng.permutation(nb * bs)[:T]
    if T > 3:
        slots[1], slots[-1] = -1, nb * bs       # padding and out of the pool: not written
    k_pool, v_pool = (torch.full((nb, bs, Hkv, D), float("nan"), dtype=dt, device=dev)
                      for _ in "kv")
    q_out = torch.full((T, Hq, D), float("nan"), dtype=torch.float32 if q32 else dt, device=dev)
    off, eps = (0.5, 1e-5)
    gq.gqa_kv_norm_rope_append(q, k, v, i32(pos if len(sections) > 1 else pos[0]), i32(slots),
                               torch.tensor(inv, device=dev), q_out, k_pool, v_pool,
                               q_weight=None if qw is None else qw.to(dev),
                               k_weight=None if kw is None else kw.to(dev), eps=eps,
                               weight_offset=off, interleaved=interleaved,
                               sections=sections if len(sections) > 1 else None)
    keep = (slots >= 0) & (slots < nb * bs)
    for name, got, x, w in (("q", q_out, qc, qw), ("k", k_pool, kc, kw)):
        ref, size = gqa_kv.norm_rotate(x, None if w is None else w.double().numpy(), eps, off, pos,
                                       inv, sections, interleaved)
        # fp32: a sum of D squares by 8 in a lane and 5 shuffles, rsqrt within 2 steps, five
        # products and a sum: at most 24 half-steps; cos and sin within 5e-7 (the header's bound).
        tol = (24 * 2.0 ** -24 + 5e-7) * size
        if got.dtype != torch.float32:   # and the final rounding (fp16: subnormal steps of 2^-24)
            tol = tol + torch.finfo(dt).eps / 2 * (np.abs(ref) + tol) + 2.0 ** -25
        g = got.double().cpu().numpy()
        if name == "k":
            g = g.reshape(nb * bs, Hkv, D)[slots[keep]]
            ref, tol = ref[keep], tol[keep]
        bad = ~(np.abs(g - ref) <= tol)
        assert not bad.any(), (name, np.argwhere(bad)[:4], g[bad][:4], ref[bad][:4])
    rows = v_pool.double().cpu().numpy().reshape(nb * bs, Hkv, D)
    assert np.array_equal(rows[slots[keep]], vc[keep])
    other = np.setdiff1d(np.arange(nb * bs), slots[keep])
    for pool in (k_pool, v_pool):
        assert torch.isnan(pool.reshape(nb * bs, -1)[torch.tensor(other, device=dev)]).all()


def test_separate_projections_and_another_stream(gq):
    # k and v from tensors of their own, token rows wider than the heads, on a side stream.
    dev, T, H, D = "cuda", 50, 4, 64
    g = torch.Generator(device=dev).manual_seed(1)
    q = torch.randn((T, H, D), generator=g, device=dev).bfloat16()
    wide = torch.randn((2, T, H * D + 64), generator=g, device=dev).bfloat16()
    k, v = (w[:, :H * D].unflatten(1, (H, D)) for w in wide)
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    inv = torch.rand(D // 2, generator=g, device=dev)
    slots = torch.arange(T, dtype=torch.int32, device=dev)
    outs = []
    side = torch.cuda.Stream()
    for stream in (None, side):
        pools = [torch.zeros((4, 16, H, D), dtype=torch.bfloat16, device=dev) for _ in "kv"]
        q_out = torch.zeros_like(q)
        torch.cuda.synchronize()
        gq.gqa_kv_norm_rope_append(q, k, v, pos, slots, inv, q_out, *pools, stream=stream)
        torch.cuda.synchronize()
        outs.append([q_out] + pools)
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert torch.equal(outs[0][2].flatten(0, 1)[:T], v)
    packed = [torch.zeros((4, 16, H, D), dtype=torch.bfloat16, device=dev) for _ in "kv"]
    q_out = torch.zeros_like(q)
    gq.gqa_kv_norm_rope_append(q, k.contiguous(), v.contiguous(), pos, slots, inv, q_out, *packed)
    assert torch.equal(packed[0], outs[0][1]) and torch.equal(q_out, outs[0][0])


def test_step_is_captured_into_a_graph(gq):
    # Tables and the cache write in one graph follow the lengths given at replay.
    dev, B, H, D, bs = "cuda", 3, 2, 64, 8
    cached, new = i32([0, 5, 8]), i32([1, 1, 1])
    free, count = i32(np.arange(20)[::-1]), i32([20])
    table = torch.zeros((B, 4), dtype=torch.int32, device=dev)
    table[:, 0] = torch.tensor([0, 17, 18])
    lens, start, slots, pos, left = (torch.zeros(n, dtype=torch.int32, device=dev)
                                     for n in (B, B + 1, B, B, 1))
    x = torch.randn((B, H, D), device=dev).half()
    pools = [torch.zeros((20, bs, H, D), dtype=torch.float16, device=dev) for _ in "kv"]
    q_out = torch.zeros((B, H, D), device=dev)
    inv = torch.rand(D // 2, device=dev)

    def step():
        gq.gqa_kv_tables(cached, new, free, count, table, lens, start, slots, pos, left, bs, 20)
        gq.gqa_kv_norm_rope_append(x, x, x, pos, slots, inv, q_out, *pools)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    new.copy_(i32([0, 1, 2]))
    cached.copy_(i32([1, 6, 7]))
    for p in pools:
        p.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert slots.tolist() == [17 * 8 + 6, 18 * 8 + 7, 0] and pos.tolist() == [6, 7, 8]
    assert lens.tolist() == [1, 7, 9] and left.tolist() == [19]
    assert torch.equal(pools[1].flatten(0, 1)[slots.long()], x)


def test_offsets_past_32_bits_and_a_single_token_of_any_stride(gq):
    dev, H, D, far = "cuda", 8, 128, 40000
    x = torch.randn((1, 3 * H * D + 4), device=dev).bfloat16()   # a row of no multiple of 8
    q, k, v = (x[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in range(3))
    inv = torch.rand(D // 2, device=dev)
    big = [torch.empty((far, 64, H, D), dtype=torch.bfloat16, device=dev) for _ in "kv"]
    small = [torch.zeros((1, 64, H, D), dtype=torch.bfloat16, device=dev) for _ in "kv"]
    outs = []
    for pools, slot in ((big, far * 64 - 1), (small, 63)):
        q_out = torch.zeros((1, H, D), device=dev)
        gq.gqa_kv_norm_rope_append(q, k, v, i32([77]), i32([slot]), inv, q_out, *pools)
        outs.append([q_out, pools[0].flatten(0, 1)[slot], pools[1].flatten(0, 1)[slot]])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert torch.equal(outs[0][2], v[0])
