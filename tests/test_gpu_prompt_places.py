"""gqa_prompt_attn and gqa_tree_attn at their largest sizes, with inputs that tell one place from
another: a key that outweighs all others at single columns of the longest table, sequences of
different queries and tables among a million tokens, cut items behind 16384 others; and random
batches (CUDA GPU)."""
import numpy as np
import pytest
import torch

from test_gpu_prompt import call, check, i32, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    from gqa_attention_weighted_gb300 import build
    build.build()
    import gqa_attention_weighted_gb300 as pkg
    yield pkg
    pkg.gqa_prompt_device_status()


@pytest.mark.parametrize("tree", [False, True])
def test_each_part_of_the_longest_row_is_read(gq, tree):
    # One token behind 2^26 - 2 rows whose table names three blocks in turn; at one column it names
    # a fourth, one of whose keys has a score of about 45. The others' are below 9 (asserted), so
    # all of them together weigh 2^26 e^-36 < 2e-8 of it, and the output is its value.
    rng = np.random.default_rng(18)
    bs, D, n = 128, 64, 2 ** 26 // 128
    q = torch.tensor(2 * rng.standard_normal((1, 1, D)), dtype=torch.float32).repeat(1, 2, 1).half()
    k, v = (torch.tensor(rng.standard_normal((4, bs, 1, D)), dtype=torch.float32).half() for _ in "kv")
    q64 = q[0, 0].double()
    k[3, 77, 0] = (q64 * (45 * 8 / (q64 @ q64))).half()
    scores = (k.double()[:, :, 0] @ q64 / 8)
    assert 44 < scores[3, 77] < 46 and scores.flatten().sort().values[-2] < 9
    base = torch.arange(n, dtype=torch.int32, device="cuda")[None] % 3
    kd, vd, qd, want = k.cuda(), v.cuda(), q.cuda(), v[3, 77, 0].double()
    start, cached, mask = i32([0, 1]), i32([2 ** 26 - 2]), i32([[1]])
    columns = [0, 1, n // 2 - 1, n // 2, n - 2, n - 1] + [int(c) for c in rng.integers(0, n, 60)]
    # Between two neighbours of 1/160 of the row each: every unit of 152 SMs or more is met.
    columns += [(2 * i + 1) * n // 320 for i in range(160)]
    for c in columns:
        tab, out = base.clone(), torch.full_like(qd, 7.0)
        tab[0, c] = 3
        if tree:
            gq.gqa_tree_attn(qd, kd, vd, start, cached, mask, tab, None, out)
        else:
            gq.gqa_prompt_attn(qd, kd, vd, start, cached, tab, None, out)
        # Half a step of its weight, and of the output.
        assert ((out[0].double().cpu() - want).abs() <= 2.0 ** -10 * want.abs() + 1e-6).all(), c
    gq.gqa_prompt_device_status()


def test_sequences_of_a_million_tokens_differ(gq):
    # 8192 sequences of 128 tokens: five kinds of queries, four tables of their own rows.
    rng = np.random.default_rng(19)
    x = make(rng, 1, 1, 64, 128, "bf16", [100] * 20, [128] * 20, pad=0)
    q = x["q"].view(20, 128, 1, 64)
    for b in range(20):
        q[b] = q[b % 5]
        x["tab"][b] = x["tab"][b % 4]
    want = check(gq, x).view(20, 128, 64).double()
    assert len({tuple(want[b, 5].tolist()) for b in range(20)}) == 20
    B = 8192
    kind = torch.arange(B, device="cuda") % 20
    big = dict(q=x["q"].cuda().view(20, 128, 1, 64)[kind].flatten(0, 1))
    out = torch.full_like(big["q"], 7.0)
    start = torch.arange(B + 1, dtype=torch.int32, device="cuda") * 128
    gq.gqa_prompt_attn(big["q"], x["k"].cuda(), x["v"].cuda(), start, i32([100] * B),
                       i32(x["tab"])[kind].contiguous(), None, out)
    gq.gqa_prompt_device_status()
    # Units may be others than the small call's, so roundings may: half a step of the output and of
    # the weights each, of values whose weighted mean of |V| is below 2.
    got = out.view(B, 128, 64).double()
    for b in range(0, B, 512):
        ref = want[kind[b:b + 512]]
        assert ((got[b:b + 512] - ref).abs() <= 2 * 2.0 ** -9 * (ref.abs() + 2)).all(), b


def test_cut_items_among_many_others(gq):
    # 128 heads a KV head: a token a query tile. 18000 items of three short tokens a sequence,
    # before and behind them a token whose rows are many; one of its keys outweighs the others.
    rng = np.random.default_rng(20)
    x = make(rng, 128, 1, 64, 16, "bf16", [100000, 5, 100000], [1, 3, 1], pad=0)
    for b, row in ((0, 31234), (2, 98765)):
        one = x["q"][4 * (b > 0), :1].double()
        x["q"][4 * (b > 0)] = one.bfloat16()
        x["k"][x["tab"][b, row // 16], row % 16, 0] = (one[0] * (30 * 8 / (one[0] @ one[0]))).bfloat16()
    want = check(gq, x).double()
    B = 6002
    kind = torch.tensor([0] + [1] * 6000 + [2], device="cuda")
    new = torch.tensor([1] + [3] * 6000 + [1], device="cuda")
    start = torch.cat([torch.zeros(1, device="cuda", dtype=torch.int64), new.cumsum(0)]).int()
    q = torch.cat([x["q"][:1], x["q"][1:4].repeat(6000, 1, 1), x["q"][4:]]).cuda()
    assert q.shape[0] == 18002 and start[-1].item() == 18002
    out = torch.full_like(q, 7.0)
    gq.gqa_prompt_attn(q, x["k"].cuda(), x["v"].cuda(), start, i32(x["cached"])[kind].contiguous(),
                       i32(x["tab"])[kind].contiguous(), None, out)
    gq.gqa_prompt_device_status()
    short = out[1:-1].view(6000, 3, 128, 64)
    assert (short == short[:1]).all()
    got = torch.cat([out[:1], short[0], out[-1:]]).double()
    assert want[0].abs().max() > 1 and want[4].abs().max() > 1 and B == len(start) - 1
    # Other cuts, other roundings: as above.
    assert ((got - want).abs() <= 2 * 2.0 ** -9 * (want.abs() + 2)).all()


@pytest.mark.parametrize("seed", range(48))
def test_random_batches(gq, seed):
    rng = np.random.default_rng(1000 + seed)
    Hq, Hkv, D = [(8, 2, 64), (32, 8, 128), (12, 4, 128), (16, 1, 256), (64, 8, 128), (8, 8, 128),
                  (32, 4, 64), (8, 4, 256), (40, 2, 128), (3, 3, 256), (14, 2, 64)][rng.integers(11)]
    B = int(2 ** rng.uniform(0, 6))
    new = [int(2 ** rng.uniform(0, 7)) - 1 + int(rng.integers(2)) for _ in range(B)]
    cached = [int(2 ** rng.uniform(0, 12)) - 1 if rng.integers(4) else 0 for _ in range(B)]
    bs, vd = int(rng.choice([8, 16, 24, 48, 64, 128, 256])), str(rng.choice(["bf16", "fp16"]))
    lens = None if rng.integers(2) else [max(0, a + n - int(rng.integers(0, 4))) for a, n in zip(cached, new)]
    if sum(new) == 0:
        new[0] = 1
    x = make(rng, Hq, Hkv, D, bs, vd, cached, new, tree=bool(seed & 1), lens=lens,
             pad=int(rng.integers(0, 40)), words=None if seed % 4 else 5)
    got = check(gq, x)
    assert torch.equal(got, call(gq, x))


@pytest.mark.parametrize("words,D", [(1, 64), (2, 128), (9, 256)])
def test_masks_narrower_and_wider_than_the_drafts(gq, words, D):
    # Bits past the mask's words count as 0; words past the drafts are not looked at.
    x = make(np.random.default_rng(21), 8, 2, D, 16, "bf16", [50, 0, 300], [100, 33, 7], tree=True,
             words=words)
    if words == 9:
        x["mask"][:, 5:] = -1
    check(gq, x)
