"""Prompts, drafted tokens and the life of a cache's pages, operator by operator.

Five operators take requests of a paged cache from their prompt to their end:

``prompt``   causal attention of whole prompts, or of chunks of them behind what is
             cached, packed sequence after sequence;
``tree``     attention of a tree of drafted tokens a sequence over its cached rows and
             the drafted tokens on its path;
``keep``     after the drafts are checked: the accepted ones' rows move together, in
             the pools of all layers;
``fork``     several continuations of one request: full blocks shared, a partial one
             copied, in the pools of all layers;
``release``  blocks of ended or cut requests back to the free list, shared ones when
             their last owner lets go.

``own = False`` computes them from elementary torch operations; ``own = True`` calls
the package's entry points.
"""
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}

# (Hq, Hkv, D) of the drawn cases: the head layouts of the package's workloads
# (G = 4, 3, 16, 8), plain multi-head attention and a wide group.
HEADS = [(8, 2, 64), (32, 8, 128), (24, 8, 128), (16, 1, 256), (64, 8, 128), (8, 8, 128),
         (32, 4, 64), (8, 4, 256), (40, 2, 128)]


def listed():
    return [
        # One short prompt on the package's smallest head layout: latency alone.
        dict(name="prompt_t61", op="prompt", B=1, Hq=8, Hkv=2, D=64, lo=61, hi=61, far=0, block=16,
             dtype="bf16"),
        # Chunked prefill of a mixed batch on the G = 3 layout: 37 requests, chunks of 1
        # to 877 tokens behind 0 to 9000 cached rows, blocks of 48.
        dict(name="prompt_chunks_b37", op="prompt", B=37, Hq=24, Hkv=8, D=128, lo=1, hi=877,
             far=9000, block=48, dtype="bf16"),
        # One long document, whole: bound by the products.
        dict(name="prompt_t16384", op="prompt", B=1, Hq=32, Hkv=8, D=128, lo=16384, hi=16384, far=0,
             block=16, dtype="bf16"),
        # One request with a small tree of drafts on the smallest head layout.
        dict(name="tree_b1", op="tree", B=1, Hq=8, Hkv=2, D=64, width=2, depth=3, far=500, block=16,
             dtype="bf16"),
        # A decode batch, up to 13 drafts a sequence (some have none: a single token),
        # G = 4, caches of 1 to 8192 rows.
        dict(name="tree_b64", op="tree", B=64, Hq=32, Hkv=8, D=128, width=3, depth=4, far=8192,
             block=16, dtype="bf16"),
        # Large trees of up to 61 drafts on the MQA layout (G = 16, D = 256, fp16).
        dict(name="tree_b9_mqa", op="tree", B=9, Hq=16, Hkv=1, D=256, width=10, depth=6, far=32768,
             block=64, dtype="fp16"),
        # The accepted path of one sequence, pools of two layers: latency alone.
        dict(name="keep_b1", op="keep", B=1, Hkv=2, D=64, width=2, depth=3, layers=2, far=500,
             block=16, dtype="bf16"),
        # A decode batch's accepted paths in the pools of 24 layers.
        dict(name="keep_b64", op="keep", B=64, Hkv=8, D=128, width=3, depth=6, layers=24, far=200,
             block=16, dtype="bf16"),
        # Four samples of one prompt.
        dict(name="fork_n4", op="fork", parents=1, copies=4, Hkv=2, D=64, layers=2, far=500,
             block=16, dtype="bf16"),
        # Eight samples of each of 24 prompts, 16 layers, blocks of 32.
        dict(name="fork_n192", op="fork", parents=24, copies=8, Hkv=8, D=128, layers=16, far=2000,
             block=32, dtype="fp16"),
        # Three requests, one of which has ended.
        dict(name="release_b3", op="release", B=3, far=700, cut=9, copies=1, block=16),
        # A full server: 256 requests in groups of four samples of one prompt, a third
        # of them ended, the others cut back to their accepted tokens.
        dict(name="release_b256", op="release", B=256, far=8192, cut=61, copies=4, block=16),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "tree", "tree", "keep", "fork", "release"])
    block = rng.choice([8, 16, 32, 48, 64, 128])
    Hq, Hkv, D = rng.choice(HEADS)
    dtype = rng.choice(["bf16", "fp16"])
    if op == "release":
        return dict(op=op, B=_log(rng, 1, 256), far=_log(rng, 16, 8192), cut=_log(rng, 1, 64),
                    copies=rng.choice([1, 2, 5]), block=rng.choice([16, 32, 64]))
    if op == "fork":
        parents, copies, layers = _log(rng, 1, 24), rng.randint(1, 8), _log(rng, 1, 16)
        while parents * copies * layers * Hkv * D * block > 24 * 8 * 16 * 8 * 128 * 32:
            layers = layers // 2
        return dict(op=op, parents=parents, copies=copies, Hkv=Hkv, D=D, layers=layers,
                    far=_log(rng, 1, 2000), block=min(block, 64), dtype=dtype)
    width, depth = rng.randint(1, 10), rng.randint(0, 6)
    if op == "keep":
        B, layers = _log(rng, 1, 64), _log(rng, 1, 24)
        return dict(op=op, B=B, Hkv=Hkv, D=D, width=width, depth=depth, layers=layers,
                    far=_log(rng, 1, 200), block=min(block, 64), dtype=dtype)
    if op == "tree":
        B, far = _log(rng, 1, 64), _log(rng, 1, 32768)
        while B * far * Hkv * D > 64 * 8192 * 8 * 128 or B * far * Hq * D * (1 + width * depth) > 2 ** 37:
            far = far // 2
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, D=D, width=width, depth=depth, far=far, block=block,
                    dtype=dtype)
    B, hi, far = _log(rng, 1, 64), _log(rng, 1, 8192), rng.choice([0, _log(rng, 1, 16384)])
    while B * hi * (hi + far) * Hq * D > 16384 ** 2 * 32 * 128 or B * (hi + far) * Hkv * D > 2 ** 29:
        hi, far = max(1, hi * 3 // 4), far * 3 // 4
    return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, D=D, lo=rng.choice([1, hi]), hi=hi, far=far, block=block,
                dtype=dtype)


# ------------------------------------------------------------------ inputs
def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi]."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _up(a, b):
    return -(-a // b)


def _lengths(c):
    """Cached and new lengths of the sequences, in no particular order."""
    B = c["B"]
    if c["op"] == "prompt":
        return _spread(0, c["far"], B), _spread(c["lo"], c["hi"], B)
    return _spread(1, c["far"], B), [1 + c["width"] * d for d in _spread(0, c["depth"], B)]


def _shuffled(c, seed):
    pairs = list(zip(*_lengths(c)))
    random.Random(seed).shuffle(pairs)
    return [list(x) for x in zip(*pairs)]


def _table(lens, bs, seed, spare=3):
    """A block table for these lengths over shuffled blocks, and the blocks left over."""
    rows = [_up(n, bs) for n in lens]
    perm = torch.randperm(sum(rows) + spare, generator=torch.Generator().manual_seed(seed))
    perm = perm.to(torch.int32)
    table = torch.zeros((len(lens), max(1, max(rows))), dtype=torch.int32)
    at = 0
    for b, r in enumerate(rows):
        table[b, :r] = perm[at:at + r]
        at += r
    return table, perm[at:], perm.numel()


def _tree(rng, width, n):
    """Parents of n drafted tokens: a root, then levels of `width`, each token behind
    one of the level before."""
    parent = []
    for i in range(n):
        level = (i + width - 1) // width
        first = 1 + (level - 2) * width
        parent.append(-1 if i == 0 else 0 if level == 1 else first + rng.randrange(width))
    return parent


def _prepare_attention(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    cached, new = _shuffled(c, seed)
    Hq, Hkv, D, bs, dt = c["Hq"], c["Hkv"], c["D"], c["block"], DTYPES[c["dtype"]]
    lens = [a + n for a, n in zip(cached, new)]
    table, _, num_blocks = _table(lens, bs, seed)
    starts = [sum(new[:b]) for b in range(len(new) + 1)]
    T = starts[-1]
    pool = lambda: torch.empty((num_blocks, bs, Hkv, D), dtype=dt, device="cuda").normal_(  # noqa: E731
        0, 1, generator=g)
    # Scores of spread 2 at the scale 1 / sqrt(D).
    q = (2 * torch.randn((T, Hq, D), generator=g, device="cuda")).to(dt)
    s = dict(c=c, q=q, k_pool=pool(), v_pool=pool(), table=table.cuda(), token_start=_ints(starts),
             cached=_ints(cached), seq_lens=_ints(lens), scale=D ** -0.5, host=(cached, new, starts),
             out=torch.empty_like(q))
    if c["op"] == "tree":
        rng, words = random.Random(seed + 1), _up(max(new), 32)
        rows = []
        for n in new:
            bits = []
            for i, p in enumerate(_tree(rng, c["width"], n)):
                bits.append((bits[p] if p >= 0 else 0) | 1 << i)
            rows += [[(x >> 32 * w & 0xffffffff) for w in range(words)] for x in bits]
        s["mask"] = torch.tensor(rows, dtype=torch.int64).to(torch.int32).cuda()
    return s


def _pools(c, num_blocks, g):
    """K and V pools of all layers, and the handle to them that a server keeps."""
    shape = (num_blocks, c["block"], c["Hkv"], c["D"])
    pools = [torch.empty(shape, dtype=DTYPES[c["dtype"]], device="cuda").normal_(0, 1, generator=g)
             for _ in range(2 * c["layers"])]
    if not own:
        return dict(pools=pools)
    import gqa_attention_weighted_gb300 as gq
    return dict(pools=pools, handle=gq.KvPools(pools))


def _prepare_keep(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    cached, new = _shuffled(c, seed)
    lens = [a + n for a, n in zip(cached, new)]
    table, _, num_blocks = _table(lens, c["block"], seed)
    W = 1 + c["depth"]
    accepted = torch.zeros((c["B"], W), dtype=torch.int32)
    counts = []
    for b, n in enumerate(new):
        depth = (n - 1) // c["width"]
        path = [0] + [1 + d * c["width"] + rng.randrange(c["width"]) for d in range(depth)]
        counts.append(max(1, len(path) - b % 3))  # the last ones were refused, for some
        accepted[b, :len(path)] = torch.tensor(path, dtype=torch.int32)
    return dict(c=c, **_pools(c, num_blocks, g), table=table.cuda(), cached=_ints(cached),
                seq_lens=_ints(lens), accepted=accepted.cuda(), counts=_ints(counts),
                kept=torch.empty(c["B"], dtype=torch.int32, device="cuda"))


def _fork_rows(c):
    """Parents' lengths; each parent's row is followed by its copies' rows."""
    return _spread(1, c["far"], c["parents"]), 1 + c["copies"]


def _prepare_fork(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens, step = _fork_rows(c)
    random.Random(seed).shuffle(lens)
    n = c["parents"] * c["copies"]
    held, free, num_blocks = _table(lens, c["block"], seed, spare=n + 5)
    table = torch.zeros((c["parents"] * step, held.shape[1]), dtype=torch.int32)
    table[::step] = held
    seq_lens = [x for m in lens for x in [m] + [0] * c["copies"]]
    parent = [p * step for p in range(c["parents"]) for _ in range(c["copies"])]
    child = [p * step + 1 + i for p in range(c["parents"]) for i in range(c["copies"])]
    return dict(c=c, **_pools(c, num_blocks, g), table=table.cuda(), seq_lens=_ints(seq_lens),
                parent=_ints(parent), child=_ints(child), free_list=free.cuda(),
                free_count=_ints([free.numel()]),
                shares=torch.zeros(num_blocks, dtype=torch.int32, device="cuda"),
                fork_block=torch.empty(n, dtype=torch.int32, device="cuda"),
                free_left=torch.empty(1, dtype=torch.int32, device="cuda"))


def _release_lengths(c):
    old = _spread(0, c["far"], c["B"])
    last = c["B"] - 1  # the longest one has ended
    new = [0 if (last - b) % 3 == 0 else max(0, n - 1 - b % c["cut"]) for b, n in enumerate(old)]
    return old, new


def _prepare_release(c, seed):
    old, new = _release_lengths(c)
    bs = c["block"]
    order = list(range(c["B"]))
    random.Random(seed).shuffle(order)
    old, new = [old[i] for i in order], [new[i] for i in order]
    table, _, num_blocks = _table(old, bs, seed, spare=64)
    shares = torch.zeros(num_blocks, dtype=torch.int32)
    for b in range(0, c["B"] - c["copies"] + 1, c["copies"]):
        n = min(old[b:b + c["copies"]]) // 2 // bs  # blocks that the group shares
        table[b + 1:b + c["copies"], :n] = table[b, :n]
        shares[table[b, :n].long()] = c["copies"] - 1
    free = torch.arange(num_blocks, dtype=torch.int32).flip(0)
    return dict(c=c, table=table.cuda(), old=_ints(old), new=_ints(new), shares=shares.cuda(),
                free_list=free.cuda(), free_count=_ints([2]), num_blocks=num_blocks,
                free_left=torch.empty(1, dtype=torch.int32, device="cuda"))


def prepare(case, seed):
    return {"prompt": _prepare_attention, "tree": _prepare_attention, "keep": _prepare_keep,
            "fork": _prepare_fork, "release": _prepare_release}[case["op"]](case, seed)


# ------------------------------------------------------------- plain forms
def _visible(s, b, i, j):
    """Which rows 0 .. L-1 of sequence b the new tokens i .. j-1 see: [j - i, L]."""
    cached, new, starts = s["host"]
    rows = torch.arange(cached[b] + new[b], device="cuda")
    if s["c"]["op"] == "prompt":
        return rows[None] <= cached[b] + torch.arange(i, j, device="cuda")[:, None]
    draft = (rows - cached[b]).clamp(min=0)
    words = s["mask"][starts[b] + i:starts[b] + j][:, draft // 32]
    return (rows < cached[b])[None] | ((words >> (draft % 32)[None]) & 1).bool()


def _plain_attention(s):
    c = s["c"]
    cached, new, starts = s["host"]
    Hq, Hkv, D, bs = c["Hq"], c["Hkv"], c["D"], c["block"]
    G = Hq // Hkv
    out = torch.empty(s["q"].shape, device="cuda")
    for b in range(c["B"]):
        blocks = s["table"][b, :_up(cached[b] + new[b], bs)].long()
        k, v = (x[blocks].flatten(0, 1).float().transpose(0, 1) for x in (s["k_pool"], s["v_pool"]))
        step = max(1, 2 ** 28 // (Hq * (cached[b] + new[b])))  # scores of at most 1 GB
        for i in range(0, new[b], step):
            j = min(new[b], i + step)
            # What the tokens of this piece cannot see is left out, or masked.
            L = cached[b] + (j if c["op"] == "prompt" else new[b])
            q = s["q"][starts[b] + i:starts[b] + j].float() * s["scale"]
            q = q.unflatten(1, (Hkv, G)).permute(1, 2, 0, 3).flatten(1, 2)     # [Hkv, G n, D]
            x = (q @ k[:, :L].transpose(1, 2)).unflatten(1, (G, j - i))
            x = x.masked_fill(~_visible(s, b, i, j)[:, :L], float("-inf"))
            x = (x - x.amax(-1, keepdim=True)).exp_()
            y = (x / x.sum(-1, keepdim=True)).flatten(1, 2) @ v[:, :L]
            out[starts[b] + i:starts[b] + j] = y.unflatten(1, (G, j - i)).permute(2, 0, 1, 3).flatten(1, 2)
    return out.to(DTYPES[c["dtype"]])


def _slots(s, b, row):
    bs = s["c"]["block"]
    return s["table"][b, row // bs].long() * bs + row % bs


def _plain_keep(s):
    """Accepted drafts count as long as they ascend."""
    cached, acc = s["cached"].long(), s["accepted"].long()
    W = acc.shape[1]
    i = torch.arange(W, device="cuda")
    prev = torch.cat([torch.full_like(acc[:, :1], -1), acc[:, :-1]], 1)
    ok = (i < s["counts"][:, None]) & (acc > prev) & (cached[:, None] + acc < s["seq_lens"][:, None])
    ok = ok.long().cumprod(1).bool()
    b, at = (ok & (acc != i)).nonzero(as_tuple=True)
    src, dst = _slots(s, b, cached[b] + acc[b, at]), _slots(s, b, cached[b] + at)
    for x in s["pools"]:
        rows = x.flatten(0, 1)
        rows[dst] = rows[src]
    s["kept"].copy_(cached + ok.sum(1))
    return tuple(s["pools"]) + (s["kept"],)


def _plain_fork(s):
    """A fork whose parent ends inside a block takes a block off the end of the free
    list for its copy; the others only share."""
    bs = s["c"]["block"]
    parent, child = s["parent"].long(), s["child"].long()
    lens = s["seq_lens"][parent].long()
    need = (lens % bs > 0).long()
    at = s["free_count"].long() - need.cumsum(0)
    served = (need == 0) | (at >= 0)
    # Before the first fork that needs a block, `at` lies one past the list.
    block = torch.where(need > 0, s["free_list"][at.clamp(0, s["free_list"].numel() - 1)], -1)
    s["fork_block"].copy_(torch.where(served, block, -2))
    rows = s["table"][parent]
    j = torch.arange(rows.shape[1], device="cuda")
    full = j < (lens // bs)[:, None]
    shared = rows[full & served[:, None]].long()
    s["shares"].index_put_((shared,), torch.ones_like(shared, dtype=torch.int32), accumulate=True)
    last = (j == (lens // bs)[:, None]) & (need > 0)[:, None]
    held = full | last
    rows = torch.where(held, torch.where(last, block[:, None], rows), s["table"][child])
    s["table"][child] = torch.where(served[:, None], rows, s["table"][child])
    s["seq_lens"][child] = torch.where(served, lens.int(), s["seq_lens"][child])
    f, r = (served[:, None] & (need > 0)[:, None]
            & (torch.arange(bs, device="cuda") < (lens % bs)[:, None])).nonzero(as_tuple=True)
    src = s["table"][parent[f], lens[f] // bs].long()
    for x in s["pools"]:
        x[block[f].long(), r] = x[src, r]
    s["free_left"].copy_(s["free_count"] - (need * served).sum())
    return tuple(s["pools"]) + (s["table"], s["seq_lens"], s["shares"], s["fork_block"],
                                s["free_left"])


def _plain_release(s):
    """A block goes back when all its owners have let go, at the place of the first."""
    bs, N = s["c"]["block"], s["num_blocks"]
    j = torch.arange(s["table"].shape[1], device="cuda")
    old, new = (-(-s[n].long() // bs) for n in ("old", "new"))
    blocks = s["table"][(j >= new[:, None]) & (j < old[:, None])].long()
    left = s["shares"].long() - torch.bincount(blocks, minlength=N)
    order = torch.arange(blocks.numel(), device="cuda")
    first = torch.full((N,), blocks.numel(), device="cuda").scatter_reduce(0, blocks, order, "amin")
    back = blocks[(left[blocks] < 0) & (first[blocks] == order)]
    n = s["free_count"].long()
    at = n + torch.arange(back.numel(), device="cuda")
    s["free_list"][at] = back.int()
    s["free_left"].copy_(n + back.numel())
    s["shares"].copy_(left.clamp(min=0))
    return s["free_list"], s["free_left"], s["shares"]


# ------------------------------------------------------------------ a pass
def run(state):
    s, c = state, state["c"]
    if not own:
        return {"prompt": _plain_attention, "tree": _plain_attention, "keep": _plain_keep,
                "fork": _plain_fork, "release": _plain_release}[c["op"]](s)
    import gqa_attention_weighted_gb300 as gq
    if c["op"] == "prompt":
        return gq.gqa_prompt_attn(s["q"], s["k_pool"], s["v_pool"], s["token_start"], s["cached"],
                                  s["table"], s["seq_lens"], s["out"], scale=s["scale"])
    if c["op"] == "tree":
        return gq.gqa_tree_attn(s["q"], s["k_pool"], s["v_pool"], s["token_start"], s["cached"],
                                s["mask"], s["table"], s["seq_lens"], s["out"], scale=s["scale"])
    if c["op"] == "keep":
        gq.gqa_kv_keep(s["handle"], s["cached"], s["accepted"], s["counts"], s["table"],
                       s["seq_lens"], s["kept"])
        return tuple(s["pools"]) + (s["kept"],)
    if c["op"] == "fork":
        gq.gqa_kv_fork(s["handle"], s["parent"], s["child"], s["table"], s["seq_lens"], s["shares"],
                       s["free_list"], s["free_count"], s["fork_block"], s["free_left"])
        return tuple(s["pools"]) + (s["table"], s["seq_lens"], s["shares"], s["fork_block"],
                                    s["free_left"])
    gq.gqa_kv_release(s["table"], s["old"], s["new"], s["shares"], s["free_list"], s["free_count"],
                      s["free_left"], block_size=c["block"])
    return s["free_list"], s["free_left"], s["shares"]


def work(case):
    c = case
    if c["op"] == "release":
        old, new = _release_lengths(c)
        n = sum(_up(a, c["block"]) - _up(b, c["block"]) for a, b in zip(old, new))
        # Lengths, and for each block its table entry, its count in and out, its place.
        return {"bytes": 8 * c["B"] + 16 * n, "flops": 0}
    if c["op"] == "fork":
        lens, _ = _fork_rows(c)
        rows = sum(n % c["block"] for n in lens) * c["copies"]
        full = sum(n // c["block"] for n in lens) * c["copies"]
        return {"bytes": rows * 2 * c["layers"] * 2 * c["Hkv"] * c["D"] * 2 + 16 * full, "flops": 0}
    cached, new = _lengths(c)
    if c["op"] == "keep":
        # All but the first and the refused ones move.
        rows = sum(max(0, (n - 1) // c["width"] - b % 3) for b, n in enumerate(new))
        moved = rows if c["width"] > 1 else 0
        return {"bytes": moved * 2 * c["layers"] * 2 * c["Hkv"] * c["D"] * 2 + 24 * c["B"],
                "flops": 0}
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    rows, T = sum(cached) + sum(new), sum(new)
    if c["op"] == "prompt":
        seen = sum(n * a + n * (n + 1) // 2 for a, n in zip(cached, new))
    else:  # a token's path: the root and one of each level
        seen = sum(n * a + 1 + sum(2 + i // c["width"] for i in range(n - 1)) for a, n in zip(cached, new))
    return {"bytes": rows * Hkv * D * 4 + 2 * T * Hq * D * 2 + 4 * rows // c["block"],
            "flops": 4 * seen * Hq * D}


# --------------------------------------------------------- 64-bit answers
def _exact_attention(c, s):
    """A KV head at a time, a softmax over the rows that each query sees."""
    cached, new, starts = s["host"]
    Hkv, D, bs = c["Hkv"], c["D"], c["block"]
    out = torch.zeros((s["q"].shape[0], Hkv, c["Hq"] // Hkv, D), dtype=torch.float64, device="cuda")
    q = s["q"].double().reshape(out.shape)
    for b in range(c["B"]):
        a, n, t0 = cached[b], new[b], starts[b]
        at = torch.arange(a + n, device="cuda")
        slot = s["table"][b].long()[at // bs] * bs + at % bs
        hide = torch.zeros((n, a + n), dtype=torch.bool, device="cuda")
        if c["op"] == "prompt":
            hide = torch.ones_like(hide).triu(a + 1)
        else:
            word = s["mask"][t0:t0 + n].long()
            for i in range(n):
                hide[:, a + i] = (word[:, i // 32] >> i % 32) % 2 == 0
        for h in range(Hkv):
            k, v = (x.flatten(0, 1)[slot, h].double() for x in (s["k_pool"], s["v_pool"]))
            for i in range(0, n, 512):
                j = min(n, i + 512)
                L = a + j if c["op"] == "prompt" else a + n
                x = torch.einsum("ngd,sd->ngs", q[t0 + i:t0 + j, h], k[:L]) * s["scale"]
                w = torch.softmax(x.masked_fill(hide[i:j, None, :L], float("-inf")), -1)
                out[t0 + i:t0 + j, h] = torch.einsum("ngs,sd->ngd", w, v[:L])
    return out.flatten(1, 2)


def exact(case, seed):
    if case["op"] not in ("prompt", "tree"):
        return None  # whole numbers and copied rows: the plain form's are the definition's
    if work(case)["flops"] > 6e12:
        return None
    return _exact_attention(case, prepare(case, seed))
