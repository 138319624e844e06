"""GPU parity of gqa_prompt_attn and gqa_tree_attn against their fp64 oracle.

Blocks no table uses, rows past a length, table entries past a length and the
output's rows past the last sequence hold NaN or garbage in every case.
"""
import numpy as np
import pytest
import torch

from helpers import TORCH_V
from oracle import gqa_prompt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    from gqa_attention_weighted_gb300 import build
    build.build()
    import gqa_attention_weighted_gb300 as pkg
    yield pkg
    pkg.gqa_prompt_device_status()


def tree_mask(rng, new, words):
    """Random trees: each token sees itself and what its parent sees."""
    rows = []
    for n in new:
        bits = []
        for i in range(n):
            p = int(rng.integers(-1, i)) if i else -1
            bits.append((bits[p] if p >= 0 else 0) | 1 << i)
        rows += [[x >> 32 * w & 0xffffffff for w in range(words)] for x in bits]
    return np.array(rows, dtype=np.uint32).reshape(-1, words).view(np.int32)


def make(rng, Hq, Hkv, D, bs, vd, cached, new, tree=False, lens=None, pad=3, first=0, words=None,
         spread=2.0):
    """A random case on the CPU: pools NaN where no table points, shuffled blocks."""
    dt = TORCH_V[vd]
    B = len(new)
    rows = [max(0, a) + n for a, n in zip(cached, new)]
    need = [-(-n // bs) for n in rows]
    nb = sum(need) + 4
    perm = rng.permutation(nb)
    pools = np.full((2, nb, bs, Hkv, D), np.nan, dtype=np.float32)
    tab = rng.integers(-5, nb + 5, size=(B, max(need) + 1))
    at = 0
    for b in range(B):
        tab[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        for j in range(need[b]):
            m = min(bs, rows[b] - j * bs)
            pools[:, tab[b, j], :m] = rng.standard_normal((2, m, Hkv, D))
    start = np.concatenate([[0], np.cumsum(new)]) + first
    T = int(start[-1]) + pad
    q = torch.tensor(rng.standard_normal((T, Hq, D)) * spread, dtype=torch.float32).to(dt)
    k, v = (torch.tensor(x).to(dt) for x in pools)
    mask = None
    if tree:
        words = words or -(-max(new) // 32)
        mask = np.zeros((T, words), dtype=np.int32)
        mask[first:first + sum(new)] = tree_mask(rng, new, words)
    return dict(q=q, k=k, v=v, start=start, cached=list(cached), mask=mask, tab=tab,
                lens=rows if lens is None else list(lens))


def i32(x):
    return None if x is None else torch.tensor(np.array(x).astype(np.int32), device="cuda")


def call(gq, x, scale=None, stream=None, q=None, out=None):
    dev = "cuda"
    if out is None:
        out = torch.full(x["q"].shape, 7.0, dtype=x["q"].dtype, device=dev)
    args = [x["q"].to(dev) if q is None else q, x["k"].to(dev), x["v"].to(dev), i32(x["start"]),
            i32(x["cached"])]
    rest = [i32(x["tab"]), i32(x["lens"]), out]
    if x["mask"] is None:
        gq.gqa_prompt_attn(*args, *rest, scale=scale, stream=stream)
    else:
        gq.gqa_tree_attn(*args, i32(x["mask"]), *rest, scale=scale, stream=stream)
    return out


def check(gq, x, scale=None, q=None):
    D = x["q"].shape[2]
    sc = D ** -0.5 if scale is None else scale
    got = call(gq, x, scale, q=q)
    gq.gqa_prompt_device_status()
    qn, k, v = (x[n].double().numpy() for n in "qkv")
    with np.errstate(invalid="ignore"):
        ref, size = gqa_prompt.attention(qn, k, v, x["start"], x["cached"], x["mask"],
                                         np.asarray(x["tab"]), x["lens"], sc,
                                         np.full(qn.shape, 7.0))
    eps = torch.finfo(x["q"].dtype).eps
    n = max(list(x["lens"] or [0]) + [a + b for a, b in zip(x["cached"] or [0], np.diff(x["start"]))])
    # A score: D/16 + 4 steps of fp32 accumulation on sum |q k| (here bounded by the norms), and
    # the exponent's argument in fp32; a weight is off by that much, relatively, and by half a
    # step of its type; the sum over keys by n/16 + 8 steps. fp16 weights far below the largest
    # are subnormal: at most 2^-24 of the largest each. The output is rounded once.
    finite = lambda a: np.abs(a[np.isfinite(a)]).max(initial=0.0)  # noqa: E731
    top = abs(sc) * finite(qn) * finite(k) * D ** 0.5
    ds = (D / 16 + 8) * 2.0 ** -23 * top * 4
    with np.errstate(invalid="ignore"):
        tol = eps / 2 * np.abs(ref) + (eps / 2 + 2 * ds + (n / 16 + 8) * 2.0 ** -23) * size * (1 + eps)
        tol = tol + (n * 2.0 ** -24 * finite(v) + 2.0 ** -25 if eps < 0.005 else 2.0 ** -40)
        g = got.double().cpu().numpy()
        bad = ~((np.abs(g - ref) <= tol) | (g == ref) | (np.isnan(g) & np.isnan(ref)))
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], g[bad][:4], ref[bad][:4], tol[bad][:4])
    return got


# Hq, Hkv, D, block, cached lengths, new lengths
PROMPTS = [
    (8, 2, 64, 16, [0], [1]),                                     # one token
    (8, 2, 64, 16, [0], [61]),
    (1, 1, 128, 8, [0, 3], [200, 1]),                             # plain heads, one of them
    (12, 4, 128, 48, [0, 385, 1], [130, 45, 0]),                  # G = 3: 126 rows a tile; no tokens
    (32, 8, 128, 16, [129, 0, 300], [33, 31, 32]),                # around a query tile of 32
    (16, 1, 256, 64, [63, 0, 700], [9, 65, 17]),                  # D = 256
    (64, 8, 128, 16, [0, 1000], [257, 40]),
    (8, 8, 128, 16, [127, 128, 129], [128, 129, 300]),            # MHA: tiles of 128 tokens
    (128, 1, 64, 128, [150, 0], [5, 3]),                          # G = 128: a token a tile
    (96, 2, 128, 16, [17], [7]),                                  # G = 48: two tokens a tile
    (14, 2, 256, 256, [0, 90], [300, 2]),
    (4, 1, 64, 8, list(range(70)), [1 + i % 5 for i in range(70)]),
    (2, 2, 128, 32, [0] * 300, [i % 4 for i in range(300)]),
]
TREES = [
    (8, 2, 64, 16, [0], [1]),
    (8, 2, 64, 16, [500], [7]),
    (32, 8, 128, 16, [1, 127, 128, 1000], [13, 1, 33, 64]),
    (16, 1, 256, 64, [700, 63], [61, 2]),
    (12, 4, 128, 48, [385, 0, 31], [45, 130, 0]),                 # masks of five words
    (8, 8, 128, 16, [121], [200]),                                # drafts over three key tiles
    (40, 2, 128, 8, [5, 260], [31, 32]),
]
IDS = [f"Hq{c[0]}-Hkv{c[1]}-D{c[2]}-bs{c[3]}-B{len(c[4])}" for c in PROMPTS]
TREE_IDS = [f"Hq{c[0]}-Hkv{c[1]}-D{c[2]}-bs{c[3]}-B{len(c[4])}-n{max(c[5])}" for c in TREES]


@pytest.mark.parametrize("vd", ["bf16", "fp16"])
@pytest.mark.parametrize("case", PROMPTS, ids=IDS)
def test_prompts_match_the_oracle(gq, case, vd):
    check(gq, make(np.random.default_rng(case[0] + case[2]), *case[:4], vd, *case[4:]))


@pytest.mark.parametrize("vd", ["bf16", "fp16"])
@pytest.mark.parametrize("case", TREES, ids=TREE_IDS)
def test_trees_match_the_oracle(gq, case, vd):
    check(gq, make(np.random.default_rng(case[0] + case[2]), *case[:4], vd, *case[4:], tree=True))


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("case", PROMPTS, ids=IDS)
def test_room_for_more_tokens(gq, case, tree):
    # A captured step's padding: above 32 query tiles one CTA makes the plan for all, below it
    # every CTA its own.
    tiles = sum(-(-n // (128 * case[1] // case[0])) for n in case[5])
    x = make(np.random.default_rng(12), *case[:4], "bf16", *case[4:], tree=tree,
             pad=3 if tiles > 32 else 33 * 128)
    check(gq, x)


@pytest.mark.parametrize("D,Hkv", [(64, 2), (128, 2), (256, 1)])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("vd", ["bf16", "fp16"])
def test_long_caches_are_cut(gq, D, Hkv, tree, vd):
    # Few rows and many keys: units of several splits, whose slots the CTAs join.
    x = make(np.random.default_rng(D), 4 * Hkv, Hkv, D, 16, vd, [9000, 20, 4000], [40, 3, 1], tree=tree)
    a = check(gq, x)
    assert torch.equal(a, call(gq, x)), "not bitwise reproducible"
    T = x["q"].shape[0]
    more = torch.zeros((33 * 128, *x["q"].shape[1:]), dtype=x["q"].dtype)
    y = dict(x, q=torch.cat([x["q"], more]))    # the other plan, with the same cuts
    if tree:
        y["mask"] = np.concatenate([x["mask"], np.zeros((len(more), x["mask"].shape[1]), np.int32)])
    assert torch.equal(check(gq, y)[:T], a)


def test_pairs_of_query_tiles(gq):
    # Enough query tiles for pairs, whose tiles end at different key tiles (MHA: a tile is 128 tokens).
    x = make(np.random.default_rng(1), 64, 64, 64, 64, "bf16", [0, 100], [700, 650])
    check(gq, x)


@pytest.mark.parametrize("tree", [False, True])
def test_lengths_that_cut_the_batch(gq, tree):
    # Rows that a request did not get (seq_lens at its cached rows, or at less), none at all,
    # negative ones; a table that cannot hold the tokens.
    rng = np.random.default_rng(2)
    x = make(rng, 8, 2, 128, 16, "bf16", [40, 0, 20, 130, 50], [5, 6, 40, 3, 9], tree=tree,
             lens=[40, 0, 30, 128, -4])
    check(gq, x)
    x["tab"] = x["tab"][:, :4]     # 64 rows a sequence
    x["lens"] = [45, 6, 60, 133, 59]
    check(gq, x)


@pytest.mark.parametrize("tree", [False, True])
def test_lengths_and_starts_may_be_left_out_or_odd(gq, tree):
    rng = np.random.default_rng(3)
    x = make(rng, 8, 2, 64, 16, "bf16", [0, 0, 0], [50, 1, 20], tree=tree)
    if not tree:
        x["cached"] = None
    x["lens"] = None
    check(gq, x)
    x = make(rng, 8, 2, 64, 16, "bf16", [3, 9, 30, 4], [50, 10, 20, 2], tree=tree, first=6, pad=9)
    check(gq, x)                                 # tokens before the first sequence, too
    x["start"] = np.array([6, 56, 50, 70, 1000])   # decreasing, and past the tokens
    x["cached"] = [3, 40, 30, 4]
    x["lens"] = [40, 0, 45, 6]
    check(gq, x)


def test_entries_outside_the_pool_read_zeros(gq):
    x = make(np.random.default_rng(4), 8, 2, 128, 16, "bf16", [100, 3], [30, 40])
    x["tab"][0, 2], x["tab"][1, 0] = -1, 10 ** 6
    check(gq, x)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("tree", [False, True])
def test_values_that_are_not_finite_reach_only_who_sees_them(gq, D, tree):
    # K and V of some new tokens are NaN or infinite, in tiles that others share with them.
    rng = np.random.default_rng(5)
    x = make(rng, 8, 2, D, 16, "bf16", [10, 300], [140, 40], tree=tree)

    def at(b, c):
        return x["tab"][b, c // 16], c % 16

    x["v"][(*at(0, 60), 0, 3)] = float("nan")
    x["v"][(*at(0, 100), 1)] = float("inf")
    x["v"][(*at(0, 149), 0, D - 1)] = float("-inf")
    x["k"][(*at(1, 320), 1)] = float("nan")
    x["v"][(*at(1, 325), 0, 17)] = float("inf")
    check(gq, x)


def test_strided_queries(gq):
    x = make(np.random.default_rng(6), 12, 4, 128, 16, "fp16", [20, 0], [33, 50])
    T, Hq, D = x["q"].shape
    packed = torch.full((T, (Hq + 8) * D), float("nan"), dtype=torch.float16, device="cuda")
    packed[:, :Hq * D] = x["q"].flatten(1).cuda()
    check(gq, x, q=packed[:, :Hq * D].unflatten(1, (Hq, D)))


def test_scales_of_zero_and_below(gq):
    x = make(np.random.default_rng(7), 8, 2, 128, 16, "bf16", [200, 0], [40, 129])
    check(gq, x, scale=0.0)
    check(gq, x, scale=-0.1)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_scores_that_keep_growing(gq, D):
    # Key c is c / 30 on its first element: every tile's maximum is well above the last one's.
    x = make(np.random.default_rng(8), 4, 1, D, 16, "fp16", [900, 0], [10, 500], spread=0.0)
    for b in range(2):
        for c in range(x["cached"][b] + (10, 500)[b]):
            x["k"][x["tab"][b, c // 16], c % 16] = 0
            x["k"][x["tab"][b, c // 16], c % 16, 0, 0] = c / 30.0
    x["q"][:, :, 0] = torch.tensor([16.0, -16.0, 4.0, 0.0])
    check(gq, x, scale=0.25)


def test_chain_masks_are_causal(gq):
    x = make(np.random.default_rng(9), 8, 2, 128, 16, "bf16", [77, 128], [70, 30])
    y = dict(x, mask=np.zeros((x["q"].shape[0], 3), dtype=np.int32))
    for b in range(2):
        for i in range(x["start"][b + 1] - x["start"][b]):
            bits = (1 << i + 1) - 1
            y["mask"][x["start"][b] + i] = np.array([bits >> 32 * w & 0xffffffff for w in range(3)],
                                                    dtype=np.uint32).view(np.int32)
    check(gq, x)
    check(gq, y)      # the same sums, of other units: not bit for bit
    with np.errstate(invalid="ignore"):
        a, b = (gqa_prompt.attention(*(x[n].double().numpy() for n in "qkv"), x["start"], x["cached"],
                                     mask, x["tab"], x["lens"], 0.1, np.zeros(x["q"].shape))[0]
                for mask in (None, y["mask"]))
    assert np.array_equal(a, b)


def test_no_tokens(gq):
    x = make(np.random.default_rng(10), 8, 2, 64, 16, "bf16", [5], [0], pad=0)
    x["tab"] = np.zeros((1, 1))
    assert call(gq, x).shape[0] == 0
    x = make(np.random.default_rng(10), 8, 2, 64, 16, "bf16", [5, 1], [0, 0], pad=4)
    assert (call(gq, x) == 7.0).all()
    gq.gqa_prompt_device_status()


def test_single_token_of_any_stride(gq):
    x = make(np.random.default_rng(11), 8, 2, 64, 16, "bf16", [70], [1], pad=0)
    q = torch.as_strided(x["q"].cuda(), (1, 8, 64), (3, 64, 1))
    check(gq, x, q=q)


# Hq, Hkv, D, block, cached lengths, new lengths: pairs of query tiles, at their edges and in
# batches of few items whose keys are many (mean above 4096 rows), and plain heads of 256.
PAIRS = [
    (64, 64, 64, 64, [0, 100], [700, 650]),
    (32, 4, 128, 32, [4500], [33]),                               # TB = 16: 2 pairs and a single tile
    (8, 2, 64, 16, [5000, 4700], [64, 31]),
    (3, 3, 256, 16, [70, 0], [200, 129]),
    (160, 160, 128, 16, [3, 0, 200], [129, 256, 300]),
]


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("case", PAIRS, ids=[f"Hq{c[0]}-Hkv{c[1]}-D{c[2]}" for c in PAIRS])
def test_pairs_match_the_oracle(gq, case, tree):
    check(gq, make(np.random.default_rng(13), *case[:4], "bf16", *case[4:], tree=tree))


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("case", PAIRS[:4], ids=[f"Hq{c[0]}-Hkv{c[1]}-D{c[2]}" for c in PAIRS[:4]])
def test_pairs_with_values_that_are_not_finite(gq, case, tree):
    # New tokens' values: seen by some rows of a pair, of both of its tiles, of cut items.
    x = make(np.random.default_rng(14), *case[:4], "fp16", *case[4:], tree=tree)
    bs, D = case[3], case[2]
    for b, (a, n) in enumerate(zip(*case[4:])):
        for i, value in ((0, "inf"), (n // 2, "nan"), (n - 1, "-inf"), (n // 3, "inf")):
            c = a + i
            x["v"][x["tab"][b, c // bs], c % bs, i % case[1], (7 * i) % D] = float(value)
    check(gq, x)


def test_rows_that_pass_the_plan_s_numbers(gq):
    # One token behind 2^26 - 1 rows, the longest table row: its entries name three blocks in
    # turn, so the softmax is over many copies of the same 384 rows (and one or two blocks more).
    rng = np.random.default_rng(15)
    bs, Hkv, D = 128, 1, 64
    k, v = (torch.tensor(rng.standard_normal((3, bs, Hkv, D)), dtype=torch.float32).half() for _ in "kv")
    n = 2 ** 26 // bs
    tab = torch.arange(n, dtype=torch.int32, device="cuda")[None] % 3
    q = torch.tensor(2 * rng.standard_normal((1, 2, D)), dtype=torch.float32).half()
    counts = np.array([n // 3 + (i < n % 3) for i in range(3)], dtype=np.float64).repeat(bs)
    counts[(n - 1) % 3 * bs + bs - 1] -= 1           # of 2^26 rows the last is not the token's own
    own = (2 ** 26 - 2) // bs % 3 * bs + (2 ** 26 - 2) % bs
    assert counts.sum() == 2 ** 26 - 1 and own == (n - 1) % 3 * bs + bs - 2
    kd, vd, qd = (x.double().numpy() for x in (k, v, q))
    s = qd[0] @ kd.reshape(-1, D).T * D ** -0.5
    w = np.exp(s) * counts
    ref = (w / w.sum(1, keepdims=True)) @ vd.reshape(-1, D)
    for tree in (False, True):
        args = (q.cuda(), k.cuda(), v.cuda(), i32([0, 1]), i32([2 ** 26 - 2]))
        rest = (tab, None, torch.empty_like(q, device="cuda"))
        got = gq.gqa_tree_attn(*args, i32([[1]]), *rest) if tree else gq.gqa_prompt_attn(*args, *rest)
        gq.gqa_prompt_device_status()
        # fp32 sums of 2^26 / (2 streams, 152 SMs and more) terms a partial, with 2^-24 a step of
        # random sign, and half a step of the weights and of the output.
        size = (w / w.sum(1, keepdims=True)) @ np.abs(vd.reshape(-1, D))
        assert (np.abs(got.double().cpu().numpy()[0] - ref) <= 2.0 ** -11 * (np.abs(ref) + 2 * size)).all()


def test_a_million_tokens(gq):
    # 8192 sequences of 128 tokens whose tables name the same two blocks: each has the outputs
    # of the first.
    rng = np.random.default_rng(16)
    x = make(rng, 1, 1, 64, 128, "bf16", [100], [128], pad=0)
    want = check(gq, x)
    B = 8192
    q = x["q"].cuda().repeat(B, 1, 1)
    out = torch.full_like(q, 7.0)
    start = torch.arange(B + 1, dtype=torch.int32, device="cuda") * 128
    tab = i32(x["tab"]).repeat(B, 1)
    gq.gqa_prompt_attn(q, x["k"].cuda(), x["v"].cuda(), start, i32([100] * B), tab, None, out)
    gq.gqa_prompt_device_status()
    # Other units than the single call's, so other roundings: each is within half a step of the
    # output and of the weights (at most the largest value) of the same sums.
    first = out[:128]
    assert (out.view(B, 128, 64) == first.view(1, 128, 64)).all()
    diff, top = (first.double() - want.double()).abs(), x["v"][~x["v"].isnan()].abs().max().item()
    assert (diff <= 2 * 2.0 ** -8 * (want.double().abs() * (1 + 2.0 ** -8) + top)).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("vd", ["bf16", "fp16"])
def test_sums_that_cross_their_bound(gq, D, vd):
    # Scores that step up by a little, by 2^7, by 2^40 and by 2^90 in the middle of a tile, down
    # again, and equal ones many tiles long: weights made with an old maximum are kept, made
    # again, or past what their type holds.
    steps = [0.0, 0.1, 5.0, -3.0, 33.0, 33.1, 90.0, 90.0, 20.0, 170.0]

    def key(c):
        return steps[c // 70 % len(steps)] * 0.6931472 + (1e-3 * c if c % 7 == 0 else 0.0)

    x = make(np.random.default_rng(17), 4, 1, D, 16, vd, [1500, 0], [9, 800], spread=0.0)
    for b in range(2):
        for c in range(x["cached"][b] + (9, 800)[b]):
            x["k"][x["tab"][b, c // 16], c % 16] = 0
            x["k"][x["tab"][b, c // 16], c % 16, 0, 0] = key(c)
    x["q"][:, :, 0] = torch.tensor([1.0, 0.5, -1.0, 0.0])
    check(gq, x, scale=1.0)
    check(gq, x, scale=-1.0)
