"""GPU parity of gqa_prefix_attn_decode against its fp64 oracle.

Blocks no table uses, rows past a length and the table entries past a length
hold NaN or garbage in every case.
"""
import numpy as np
import pytest
import torch

from helpers import TORCH_V
from oracle import gqa_prefix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    from gqa_attention_weighted_gb300 import build
    build.build()
    import gqa_attention_weighted_gb300 as pkg
    yield pkg
    pkg.gqa_prefix_device_status()


def make(rng, B, Hq, Hkv, D, bs, vd, plens, starts, lens, spread=2.0, k_of=None):
    """A random case on the CPU: pools NaN where no table points, shuffled blocks."""
    dt = TORCH_V[vd]
    plens, lens = list(plens), list(lens)
    need = [-(-max(0, n) // bs) for n in plens + lens]
    nb = sum(need) + 4
    perm = rng.permutation(nb)
    pools = np.full((2, nb, bs, Hkv, D), np.nan, dtype=np.float32)
    P = len(plens)
    ptab = rng.integers(-5, nb + 5, size=(P, max(need[:P], default=0) + 1)) if P else None
    mb = max(need[P:]) + 1
    tab = rng.integers(-5, nb + 5, size=(B, mb))
    at = 0
    for i, (n, r) in enumerate(zip(plens + lens, need)):
        row = ptab[i] if i < P else tab[i - P]
        row[:r] = perm[at:at + r]
        at += r
        for c in range(max(0, n)):
            pools[:, row[c // bs], c % bs] = rng.standard_normal((2, Hkv, D))
            if k_of is not None:
                pools[0, row[c // bs], c % bs] = k_of(i, c)
    q = torch.tensor(rng.standard_normal((B, Hq, D)) * spread, dtype=torch.float32).to(dt)
    k, v = (torch.tensor(x).to(dt) for x in pools)
    return dict(q=q, k=k, v=v, ptab=ptab, plens=plens if P else None, starts=starts, tab=tab,
                lens=lens)


def i32(x):
    return None if x is None else torch.tensor(np.array(x).astype(np.int32), device="cuda")


def call(gq, x, scale=None, stream=None, out=None):
    dev = "cuda"
    if out is None:
        out = torch.full(x["q"].shape, float("nan"), dtype=x["q"].dtype, device=dev)
    gq.gqa_prefix_attn_decode(x["q"].to(dev), x["k"].to(dev), x["v"].to(dev), i32(x["ptab"]),
                              i32(x["plens"]), i32(x["starts"]), i32(x["tab"]), i32(x["lens"]),
                              out, scale=scale, stream=stream)
    return out


def check(gq, x, scale=None):
    sc = x["q"].shape[2] ** -0.5 if scale is None else scale
    got = call(gq, x, scale)
    gq.gqa_prefix_device_status()
    q, k, v = (x[n].double().numpy() for n in "qkv")
    ref, size = gqa_prefix.attention(q, k, v, x["ptab"], x["plens"], x["starts"], x["tab"],
                                     x["lens"], sc)
    D, eps = q.shape[2], torch.finfo(x["q"].dtype).eps
    n = max([0] + (x["plens"] or [])) + max([0] + list(x["lens"] or [x["tab"].shape[1] * k.shape[1]]))
    # A score: D/16 + 4 steps of fp32 accumulation on sum |q k| (here bounded by the norms), and
    # the exponent's argument in fp32; a weight is off by that much, relatively, and by half a
    # step of its type; the sum over keys by n/16 + 8 steps. fp16 weights far below the largest
    # are subnormal: at most 2^-24 of the largest each. The output is rounded once.
    top = abs(sc) * np.abs(q).max() * np.nanmax(np.abs(k)) * D ** 0.5
    ds = (D / 16 + 8) * 2.0 ** -23 * top * 4
    tol = eps / 2 * np.abs(ref) + (eps / 2 + 2 * ds + (n / 16 + 8) * 2.0 ** -23) * size * (1 + eps)
    tol = tol + (n * 2.0 ** -24 * np.nanmax(np.abs(v)) + 2.0 ** -25 if eps < 0.005 else 2.0 ** -40)
    g = got.double().cpu().numpy()
    bad = ~(np.abs(g - ref) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], g[bad][:4], ref[bad][:4], tol[bad][:4])
    return got


# B, Hq, Hkv, D, block, prefix lengths, group starts, own lengths
CASES = [
    (1, 8, 2, 64, 16, [], None, [1]),                            # one row, no prefix
    (1, 1, 1, 128, 8, [1], None, [0]),                           # one prefix row, nothing own
    (2, 8, 2, 64, 16, [512], None, [3, 64]),
    (3, 12, 4, 128, 48, [385], [0, 3], [0, 130, 129]),           # blocks of 48, partial tiles
    (5, 32, 8, 128, 16, [129, 0, 300], [0, 2, 3, 4], [7, 0, 256, 128, 1]),   # groups, one loose
    (4, 16, 1, 256, 64, [700], None, [1, 63, 64, 65]),
    (9, 64, 8, 128, 16, [260], None, [127, 128, 129, 0, 1, 500, 3, 255, 257]),
    (70, 8, 2, 64, 8, [200], [3, 66], list(range(70))),          # 252 rows: two query tiles
    (130, 4, 2, 128, 32, [333, 100], [0, 129, 130], [5] * 130),  # 258 rows: three tiles
    (33, 128, 1, 64, 128, [150], None, [9] * 33),                # G = 128: a sequence a tile
    (45, 9, 3, 128, 16, [140], None, [2] * 45),                  # G = 3: 126 rows a tile
    (2, 14, 2, 256, 256, [90], None, [300, 2]),
    (3, 8, 8, 128, 16, [1000], None, [40, 0, 1]),                # plain multi-head
    (300, 1, 1, 64, 8, [64], [10, 290], [1] * 300),
    (6, 96, 2, 128, 16, [], None, [100, 0, 3, 17, 129, 64]),     # G = 48: two warps of rows
    (70, 4, 2, 64, 8, [3 * i for i in range(32)], [2 * i for i in range(33)],
     [i % 5 for i in range(70)]),                                # 32 groups, some without rows
    (1500, 2, 1, 64, 8, [40], [200, 1400], [i % 11 for i in range(1500)]),
]


@pytest.mark.parametrize("vd", ["bf16", "fp16"])
@pytest.mark.parametrize("case", CASES, ids=[f"B{c[0]}-Hq{c[1]}-Hkv{c[2]}-D{c[3]}-bs{c[4]}"
                                             for c in CASES])
def test_matches_the_oracle(gq, case, vd):
    B, Hq, Hkv, D, bs, plens, starts, lens = case
    check(gq, make(np.random.default_rng(B * D + Hq), B, Hq, Hkv, D, bs, vd, plens, starts, lens))


@pytest.mark.parametrize("D,Hkv,B", [(64, 2, 20), (128, 2, 40), (256, 1, 20)])
@pytest.mark.parametrize("vd", ["bf16", "fp16"])
def test_long_prefix_is_split(gq, D, Hkv, B, vd):
    # Long enough for several splits of the prefix and of one long sequence.
    rng = np.random.default_rng(D)
    x = make(rng, B, 8 * Hkv, Hkv, D, 16, vd, [5000], [0, B - 1], [3000] + [20] * (B - 1))
    a = check(gq, x)
    assert torch.equal(a, call(gq, x)), "not bitwise reproducible"


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("vd", ["bf16", "fp16"])
def test_scores_that_keep_growing(gq, D, vd):
    # Key c is c / 30 on its first element: every tile's maximum is well above the last one's.
    rng = np.random.default_rng(5)

    def k_of(i, c):
        k = np.zeros((1, D))
        k[0, 0] = c / 30.0
        return k

    x = make(rng, 3, 4, 1, D, 16, vd, [900], None, [10, 700, 0], spread=0.0, k_of=k_of)
    x["q"][:, :, 0] = torch.tensor([16.0, -16.0, 4.0, 0.0])
    check(gq, x, scale=0.25)


def test_scales_of_zero_and_below(gq):
    rng = np.random.default_rng(6)
    x = make(rng, 3, 8, 2, 128, 16, "bf16", [200], None, [40, 0, 129])
    check(gq, x, scale=0.0)
    check(gq, x, scale=-0.1)


def test_table_entries_outside_the_pool_are_rows_of_zeros(gq):
    rng = np.random.default_rng(7)
    x = make(rng, 4, 8, 2, 64, 16, "bf16", [200], [0, 3], [100, 30, 17, 40])
    nb = x["k"].shape[0]
    x["ptab"][0, 3], x["ptab"][0, 12] = -1, nb
    x["tab"][0, 6], x["tab"][1, 0], x["tab"][3, 1] = nb + 7, -(1 << 31), (1 << 31) - 1
    check(gq, x)


def test_lengths_and_groups_are_clamped(gq):
    rng = np.random.default_rng(8)
    x = make(rng, 6, 4, 2, 128, 8, "bf16", [40, 24, 16], [-3, 2, 1, 99], [16] * 6)
    for a in ("ptab", "tab"):                    # every table entry a valid block
        x[a] = np.abs(x[a]) % x["k"].shape[0]
    for n in "kv":
        x[n] = torch.nan_to_num(x[n], nan=0.5)
    x["lens"] = [-4, 1000, 16, 0, 3, 1 << 30]
    x["plens"] = [40, -1, 1 << 30]
    check(gq, x)
    x["starts"] = [5, 4, 3, 2]                   # falling: every group but the last start is empty
    check(gq, x)


def test_no_own_rows_no_lengths(gq):
    rng = np.random.default_rng(9)
    x = make(rng, 5, 8, 2, 64, 16, "fp16", [130], None, [0] * 5)
    x["tab"] = x["lens"] = None
    got = call(gq, x)
    x["tab"], x["lens"] = np.zeros((5, 1), dtype=np.int64), [0] * 5
    assert torch.equal(got, check(gq, x))
    y = make(rng, 3, 8, 2, 64, 16, "fp16", [], None, [48, 48, 48])
    y["tab"] = y["tab"][:, :3]
    a = check(gq, y)
    y["lens"] = None                             # NULL: every row that the table holds
    assert torch.equal(a, call(gq, y))
    y["lens"] = [0, 0, 0]
    assert torch.equal(call(gq, y), torch.zeros_like(a))


def test_infinite_and_nan_rows(gq):
    # An infinite score takes the whole weight's place only in its own sequence.
    rng = np.random.default_rng(10)
    x = make(rng, 3, 4, 2, 64, 16, "bf16", [100], None, [20, 20, 20])
    x["k"][x["tab"][1, 0], 3] = float("nan")
    got = call(gq, x)
    assert torch.isnan(got[1]).all() and torch.isfinite(got[[0, 2]]).all()


def test_other_streams_graphs_and_reuse_of_the_workspace(gq):
    rng = np.random.default_rng(11)
    x = make(rng, 4, 8, 2, 128, 16, "bf16", [300], None, [10, 200, 0, 64])
    ref = check(gq, x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(ref)
    torch.cuda.synchronize()
    call(gq, x, stream=side, out=out)
    side.synchronize()
    assert torch.equal(out, ref)
    d = {n: x[n].cuda() for n in "qkv"}
    t = {n: i32(x[n]) for n in ("ptab", "plens", "starts", "tab", "lens")}

    def step():
        gq.gqa_prefix_attn_decode(d["q"], d["k"], d["v"], t["ptab"], t["plens"], t["starts"],
                                  t["tab"], t["lens"], out)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    # A larger call outgrows the workspace that the graph holds; the graph still runs, and
    # follows lengths that change between replays.
    check(gq, make(rng, 200, 32, 8, 128, 16, "bf16", [140], None, [3] * 200))
    t["lens"].copy_(i32([7, 129, 0, 1]))
    t["plens"].copy_(i32([129]))
    x["lens"], x["plens"] = [7, 129, 0, 1], [129]
    want = check(gq, x)
    out.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("D,G", [(64, 5), (128, 3), (256, 7)])
def test_results_do_not_depend_on_earlier_calls(gq, D, G):
    # Query tiles that are not full, own units of a few rows: what an earlier call left in
    # shared and tensor memory lies in the other rows.
    rng = np.random.default_rng(12)
    x = make(rng, 21, 2 * G, 2, D, 16, "bf16", [1500], [0, 20], list(range(0, 840, 40)))
    y = make(rng, 40, 8, 2, D, 16, "bf16", [2500], None, [300] * 40, spread=60.0)
    first = call(gq, x)
    for _ in range(3):
        call(gq, y)
        assert torch.equal(call(gq, x), first)


def test_offsets_past_32_bits(gq):
    # The same rows in a small pool and at the far end of one of 5 GB: equal bits.
    rng = np.random.default_rng(13)
    x = make(rng, 3, 16, 8, 128, 64, "bf16", [200], None, [70, 0, 129])
    near = call(gq, x)
    nb, far = x["k"].shape[0], 40000
    big = [torch.empty((far, 64, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    for b, n in zip(big, "kv"):
        b[far - nb:] = x[n].cuda()
    t = {n: i32(x[n]) for n in ("ptab", "plens", "starts", "tab", "lens")}
    for n in ("ptab", "tab"):
        t[n] = torch.where((t[n] >= 0) & (t[n] < nb), t[n] + (far - nb), t[n])
    out = torch.zeros_like(near)
    gq.gqa_prefix_attn_decode(x["q"].cuda(), *big, t["ptab"], t["plens"], t["starts"], t["tab"],
                              t["lens"], out)
    assert torch.equal(out, near)
