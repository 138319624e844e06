"""The paged serving step around decode attention, operator by operator.

Three operators take a batch from its request lengths to its attention output:

``tables``   block tables, slots and positions of a step's new tokens, made on the
             GPU from the requests' lengths and a list of free blocks;
``rope``     per-head RMS norm of queries and keys, rotary positions with one or
             several axes, and the write of K and V into a paged cache, in one pass;
``prefix``   decode attention over a paged cache for a batch whose sequences share
             long prefixes, each prefix read once for all of its sequences.

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
        # One decode step of a full server: 256 requests, one new token each.
        dict(name="tables_decode_b256", op="tables", B=256, cached=8192, new=1, block=16,
             refused=0, base=False),
        # Chunked prefill of a mixed batch: 96 requests, chunks of 0 to 2731 tokens
        # (131 thousand tokens in all) behind shared prefixes, the last requests
        # finding no free block.
        dict(name="tables_prefill_b96", op="tables", B=96, cached=20000, new=2731, block=32,
             refused=5, base=True),
        # The package's smallest decode shape, a single token: latency alone.
        dict(name="rope_decode_t1", op="rope", T=1, Hq=8, Hkv=2, D=64, rot=64, axes=1, norm=True,
             interleaved=False, dtype="bf16", q32=True, block=16, far=512, skip=0),
        # One decode step of 64 sequences on the G = 3 layout, half of each head
        # rotated, no norms, far positions, fp32 queries for the fused decode call.
        dict(name="rope_decode_t64", op="rope", T=64, Hq=24, Hkv=8, D=128, rot=64, axes=1,
             norm=False, interleaved=False, dtype="fp16", q32=True, block=16, far=131072, skip=0),
        # A prefill chunk of 16 thousand tokens on the G = 4 layout.
        dict(name="rope_prefill_t16384", op="rope", T=16384, Hq=32, Hkv=8, D=128, rot=128, axes=1,
             norm=True, interleaved=False, dtype="bf16", q32=False, block=16, far=32768, skip=0),
        # An image's patches with time, height and width axes on the MQA layout:
        # an odd count, neighbouring pairs rotated, the last tokens padding.
        dict(name="rope_image_t4097", op="rope", T=4097, Hq=16, Hkv=1, D=256, rot=256, axes=3,
             norm=True, interleaved=True, dtype="fp16", q32=False, block=64, far=8192, skip=17),
        # Two sequences behind a short system prompt: the smallest call.
        dict(name="prefix_b2_p512", op="prefix", B=2, Hq=8, Hkv=2, D=64, groups=1, prefix=512,
             loose=0, lo=1, hi=64, block=16, dtype="bf16"),
        # A small batch behind one long document, G = 4.
        dict(name="prefix_b16_p8192", op="prefix", B=16, Hq=32, Hkv=8, D=128, groups=1,
             prefix=8192, loose=0, lo=1, hi=512, block=16, dtype="bf16"),
        # G = 3, an odd batch, a prefix that ends inside a block, blocks of 48.
        dict(name="prefix_b41_p16001", op="prefix", B=41, Hq=24, Hkv=8, D=128, groups=1,
             prefix=16001, loose=0, lo=1, hi=2000, block=48, dtype="bf16"),
        # The MQA layout (G = 16, D = 256, fp16), 32 thousand shared positions.
        dict(name="prefix_b64_p32768_mqa", op="prefix", B=64, Hq=16, Hkv=1, D=256, groups=1,
             prefix=32768, loose=0, lo=128, hi=2048, block=64, dtype="fp16"),
        # Three system prompts of different lengths and eight requests without one.
        dict(name="prefix_b48_groups3", op="prefix", B=48, Hq=32, Hkv=8, D=128, groups=3,
             prefix=4000, loose=8, lo=0, hi=4096, block=16, dtype="bf16"),
        # A large batch (G = 8) behind a long shared context: bound by the products.
        dict(name="prefix_b256_p32768", op="prefix", B=256, Hq=64, Hkv=8, D=128, groups=1,
             prefix=32768, loose=0, lo=1, hi=1024, block=16, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["tables", "rope", "prefix", "prefix"])
    block = rng.choice([8, 16, 32, 48, 64, 128])
    if op == "tables":
        B = _log(rng, 1, 1024)
        return dict(op=op, B=B, cached=_log(rng, 1, 20000),
                    new=rng.choice([1, _log(rng, 1, max(1, 262144 // B))]), block=block,
                    refused=rng.choice([0, 0, B // 8]), base=rng.random() < 0.5)
    Hq, Hkv, D = rng.choice(HEADS)
    dtype = rng.choice(["bf16", "fp16"])
    if op == "rope":
        T = _log(rng, 1, 16384 * 48 * 128 // ((Hq + 2 * Hkv) * D))
        return dict(op=op, T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2]),
                    axes=rng.choice([1, 1, 3]), norm=rng.random() < 0.6,
                    interleaved=rng.random() < 0.4, dtype=dtype, q32=rng.random() < 0.4,
                    block=block, far=_log(rng, 64, 131072), skip=rng.choice([0, T // 10]))
    B = _log(rng, 1, 256)
    hi = _log(rng, 1, 4096)
    while B * hi * Hkv * D > 256 * 1024 * 8 * 128:
        hi //= 2
    prefix = _log(rng, 1, 32768)
    groups = rng.choice([1, 1, min(B, 3)])
    while B * Hq * D * prefix > 256 * 64 * 128 * 32768 or groups * prefix * Hkv * D > 2 ** 26:
        prefix //= 2
    return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, D=D, groups=groups, prefix=prefix,
                loose=rng.choice([0, 0, B // 4]) if B > groups + B // 4 else 0,
                lo=rng.choice([0, 1, hi]), hi=hi, block=block, dtype=dtype)


# ------------------------------------------------------------------ inputs
def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi]."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _up(a, b):
    return -(-a // b)


def _table_lengths(c):
    """Cached and new lengths of the requests, in no particular order."""
    cached = _spread(0, c["cached"], c["B"])
    new = [1] * c["B"] if c["new"] == 1 else _spread(0, c["new"], c["B"])
    return cached, new


def _prepare_tables(c, seed):
    rng = random.Random(seed)
    cached, new = _table_lengths(c)
    rng.shuffle(cached)
    rng.shuffle(new)
    bs, B = c["block"], c["B"]
    held = [_up(x, bs) for x in cached]
    need = [_up(x + n, bs) - h for x, n, h in zip(cached, new, held)]
    free = sum(need[:B - c["refused"]])
    num_blocks = sum(held) + sum(need) + 16
    max_blocks = _up(max(cached) + max(new), bs)  # the longest request of any batch
    perm = torch.randperm(num_blocks, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.zeros((B, max_blocks), dtype=torch.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = perm[at:at + h]
        at += h
    T = sum(new) + 64  # room for the padding of a captured step
    dev = "cuda"
    return dict(c=c, cached=_ints(cached), new=_ints(new), free_list=perm[at:].to(dev),
                free_count=_ints([free]), table=table.to(dev), T=T, num_blocks=num_blocks,
                base=_ints([rng.randrange(0, 4096) for _ in range(B)]) if c["base"] else None,
                seq_lens=torch.empty(B, dtype=torch.int32, device=dev),
                token_start=torch.empty(B + 1, dtype=torch.int32, device=dev),
                slots=torch.empty(T, dtype=torch.int32, device=dev),
                positions=torch.empty(T, dtype=torch.int32, device=dev),
                free_left=torch.empty(1, dtype=torch.int32, device=dev))


def _sections(c):
    """Pairs of each axis: one part of time, equal parts of height and width."""
    pairs = c["rot"] // 2
    if c["axes"] == 1:
        return [pairs]
    side = 3 * pairs // 8
    return [pairs - 2 * side, side, side]


def _prepare_rope(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    T, Hq, Hkv, D, bs = c["T"], c["Hq"], c["Hkv"], c["D"], c["block"]
    dt = DTYPES[c["dtype"]]
    qkv = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device="cuda").to(dt)
    num_blocks = _up(T, bs) + 4
    slots = torch.randperm(num_blocks * bs, generator=g, device="cuda")[:T].to(torch.int32)
    if c["skip"]:
        slots[T - c["skip"]:] = -1
    if c["axes"] == 1:
        positions = torch.randint(0, c["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
    else:
        side = max(1, int(T ** 0.5))
        t = torch.arange(T, device="cuda", dtype=torch.int32)
        start = rng.randrange(0, c["far"])
        positions = torch.stack([torch.full_like(t, start), start + t // side, start + t % side])
    pairs = c["rot"] // 2
    inv_freq = (1e6 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float().cuda()
    w = lambda: (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)  # noqa: E731
    pool = lambda: torch.randn((num_blocks, bs, Hkv, D), generator=g, device="cuda").to(dt)  # noqa: E731
    q, k, v = qkv.split([Hq * D, Hkv * D, Hkv * D], dim=1)  # views of the packed projection
    return dict(c=c, q=q.unflatten(1, (Hq, D)), k=k.unflatten(1, (Hkv, D)),
                v=v.unflatten(1, (Hkv, D)), slots=slots, positions=positions, inv_freq=inv_freq,
                qw=w() if c["norm"] else None, kw=w() if c["norm"] else None, k_pool=pool(),
                v_pool=pool(), eps=1e-6, sections=_sections(c),
                q_out=torch.empty((T, Hq, D), dtype=torch.float32 if c["q32"] else dt,
                                  device="cuda"))


def _prefix_lengths(c):
    """Prefix lengths, the groups' first sequences, the sequences' own lengths."""
    P = c["groups"]
    plens = [c["prefix"] * (p + 1) // P for p in range(P)]
    together = c["B"] - c["loose"]
    return plens, [together * p // P for p in range(P + 1)], _spread(c["lo"], c["hi"], c["B"])


def _prepare_prefix(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    plens, starts, lens = _prefix_lengths(c)
    random.Random(seed).shuffle(lens)
    B, Hq, Hkv, D, bs = c["B"], c["Hq"], c["Hkv"], c["D"], c["block"]
    dt = DTYPES[c["dtype"]]
    max_p, max_s = max(1, _up(max(plens), bs)), max(1, _up(max(lens), bs))
    rows = [_up(n, bs) for n in plens] + [_up(n, bs) for n in lens]
    num_blocks = sum(rows) + 3
    perm = torch.randperm(num_blocks, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    prefix_table = torch.zeros((len(plens), max_p), dtype=torch.int32)
    table = torch.zeros((B, max_s), dtype=torch.int32)
    at = 0
    for i, r in enumerate(rows):
        row = prefix_table[i] if i < len(plens) else table[i - len(plens)]
        row[:r] = perm[at:at + r]
        at += r
    pool = lambda: torch.empty((num_blocks, bs, Hkv, D), dtype=dt, device="cuda").normal_(  # noqa: E731
        0, 1, generator=g)
    # Scores of spread 2 at the scale 1 / sqrt(D).
    q = (2 * torch.randn((B, Hq, D), generator=g, device="cuda")).to(dt)
    return dict(c=c, q=q, k_pool=pool(), v_pool=pool(), prefix_table=prefix_table.cuda(),
                prefix_lens=_ints(plens), group_start=_ints(starts), table=table.cuda(),
                seq_lens=_ints(lens), scale=D ** -0.5, host=(plens, starts, max(lens)),
                out=torch.empty((B, Hq, D), dtype=dt, device="cuda"))


def prepare(case, seed):
    return {"tables": _prepare_tables, "rope": _prepare_rope,
            "prefix": _prepare_prefix}[case["op"]](case, seed)


# ------------------------------------------------------------- plain forms
def _plain_tables(s):
    """Blocks come off the end of the free list in request order. A request is
    served when it needs no block, or the needs up to its own fit the list."""
    bs = s["c"]["block"]
    cached, new, table = s["cached"].long(), s["new"].long(), s["table"]
    held = (cached + bs - 1) // bs
    need = (cached + new + bs - 1) // bs - held
    upto = need.cumsum(0)
    free = s["free_count"].long()
    served = (need == 0) | (upto <= free)
    taken = (need * served).cumsum(0)
    token_start = torch.cat([torch.zeros_like(upto[:1]), new.cumsum(0)])

    def from_list(j, b):  # block of column j of request b (past what it held)
        at = free - 1 - (upto[b] - need[b] + j - held[b])
        return s["free_list"][at.clamp(0, s["free_list"].numel() - 1)]

    b = torch.arange(table.shape[0], device="cuda")[:, None].expand_as(table)
    j = torch.arange(table.shape[1], device="cuda").expand_as(table)
    fresh = served[b] & (j >= held[b]) & (j < held[b] + need[b])
    full = torch.where(fresh, from_list(j, b), table)

    t = torch.arange(s["T"], device="cuda")
    b = torch.searchsorted(token_start[1:], t, right=True)
    real = b < cached.numel()
    b = b.clamp(max=cached.numel() - 1)
    row = cached[b] + t - token_start[b]
    slot = full[b, (row // bs).clamp(0, table.shape[1] - 1)].long() * bs + row % bs
    slots = torch.where(real & served[b], slot, -1)
    pos = row if s["base"] is None else row + s["base"].long()[b]
    positions = torch.where(real, pos, 0)
    i32 = torch.int32
    return (full, (cached + new * served).to(i32), token_start.to(i32), slots.to(i32),
            positions.to(i32), (free - taken[-1:]).to(i32))


def _angles(s):
    """cos and sin [T, pairs], the angle in 64 bits: positions reach far."""
    c = s["c"]
    if c["axes"] == 1:
        pos = s["positions"].double()[:, None]
    else:
        axis = torch.repeat_interleave(torch.arange(c["axes"], device="cuda"),
                                       torch.tensor(s["sections"], device="cuda"),
                                       output_size=c["rot"] // 2)
        pos = s["positions"].double()[axis].T
    angle = pos * s["inv_freq"].double()
    return angle.cos().float(), angle.sin().float()


def _norm_rotate(s, x, w, cos, sin):
    c = s["c"]
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
    r = c["rot"]
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
    cos, sin = cos[:, None], sin[:, None]
    y = (a * cos - b * sin, b * cos + a * sin)
    y = torch.stack(y, -1).flatten(-2) if c["interleaved"] else torch.cat(y, -1)
    return torch.cat([y, x[..., r:]], -1)


def _plain_rope(s):
    c = s["c"]
    dt = DTYPES[c["dtype"]]
    cos, sin = _angles(s)
    q = _norm_rotate(s, s["q"], s["qw"], cos, sin).to(s["q_out"].dtype)
    k = _norm_rotate(s, s["k"], s["kw"], cos, sin).to(dt)
    n = c["T"] - c["skip"]
    at = s["slots"][:n].long()
    s["k_pool"].flatten(0, 1)[at] = k[:n]
    s["v_pool"].flatten(0, 1)[at] = s["v"][:n]
    return q, s["k_pool"], s["v_pool"]


def _softmax_part(scores, values):
    """Maximum, sum of exp and weighted sum of one part of the keys."""
    m = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (scores - m).exp()
    return m, p.sum(-1, keepdim=True), p @ values


def _plain_prefix(s):
    c = s["c"]
    B, Hq, Hkv, D, bs = c["B"], c["Hq"], c["Hkv"], c["D"], c["block"]
    G = Hq // Hkv
    plens, starts, longest = s["host"]
    out = torch.empty((B, Hq, D), device="cuda")
    group = lambda p: (starts[p], starts[p + 1], plens[p])  # noqa: E731
    spans = [group(p) + (p,) for p in range(len(plens))] + [(starts[-1], B, 0, 0)]
    for b0, b1, plen, p in spans:
        n = b1 - b0
        if n == 0:
            continue
        # Each sequence's own keys, at most 2^27 elements of them at a time.
        step = max(1, 2 ** 27 // (max(longest, 1) * Hkv * D))
        if plen:
            blocks = s["prefix_table"][p, :_up(plen, bs)].long()
            pk = s["k_pool"][blocks].flatten(0, 1)[:plen].float()
            pv = s["v_pool"][blocks].flatten(0, 1)[:plen].float()
        q = s["q"][b0:b1].float().unflatten(1, (Hkv, G)) * s["scale"]
        if plen:
            parts = []
            for h in range(Hkv):
                m, l, o = _softmax_part(q[:, h].reshape(n * G, D) @ pk[:, h].T, pv[:, h])
                parts.append([x.reshape(n, G, -1) for x in (m, l, o)])
            pm, pl, po = (torch.stack([x[i] for x in parts], 1) for i in range(3))
        for i in range(0, n, step):
            j = min(n, i + step)
            blocks = s["table"][b0 + i:b0 + j].long()
            k = s["k_pool"][blocks].flatten(1, 2).float().transpose(1, 2)  # [n, Hkv, S, D]
            v = s["v_pool"][blocks].flatten(1, 2).float().transpose(1, 2)
            dead = (torch.arange(k.shape[2], device="cuda")
                    >= s["seq_lens"][b0 + i:b0 + j, None])[:, None, None]
            scores = (q[i:j] @ k.transpose(2, 3)).masked_fill(dead, float("-inf"))
            m, l, o = _softmax_part(scores, v.masked_fill(dead[:, :, 0, :, None], 0))
            if plen:
                top = torch.maximum(m, pm[i:j])
                e, f = (m - top).exp(), (pm[i:j] - top).exp()
                l, o = l * e + pl[i:j] * f, o * e + po[i:j] * f
            o = torch.where(l > 0, o / l.clamp(min=1e-30), 0)
            out[b0 + i:b0 + j] = o.flatten(1, 2)
    return out.to(DTYPES[c["dtype"]])


# ------------------------------------------------------------------ a pass
def run(state):
    s, c = state, state["c"]
    if not own:
        return {"tables": _plain_tables, "rope": _plain_rope, "prefix": _plain_prefix}[c["op"]](s)
    import gqa_attention_weighted_gb300 as gq
    if c["op"] == "tables":
        gq.gqa_kv_tables(s["cached"], s["new"], s["free_list"], s["free_count"], s["table"],
                         s["seq_lens"], s["token_start"], s["slots"], s["positions"],
                         s["free_left"], block_size=c["block"], num_blocks=s["num_blocks"],
                         pos_base=s["base"])
        return (s["table"], s["seq_lens"], s["token_start"], s["slots"], s["positions"],
                s["free_left"])
    if c["op"] == "rope":
        gq.gqa_kv_norm_rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"],
                                   s["inv_freq"], s["q_out"], s["k_pool"], s["v_pool"],
                                   q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"],
                                   sections=s["sections"], interleaved=c["interleaved"])
        return s["q_out"], s["k_pool"], s["v_pool"]
    return gq.gqa_prefix_attn_decode(s["q"], s["k_pool"], s["v_pool"], s["prefix_table"],
                                     s["prefix_lens"], s["group_start"], s["table"],
                                     s["seq_lens"], s["out"], scale=s["scale"])


def work(case):
    c = case
    if c["op"] == "tables":
        cached, new = _table_lengths(c)
        bs, T = c["block"], sum(new) + 64
        # Lengths in and out, slots and positions of every token, and the new
        # blocks' entries out of the list and into the table.
        blocks = sum(new) // bs
        return {"bytes": 4 * (4 * c["B"] + 2 * T + 2 * blocks), "flops": 0}
    if c["op"] == "rope":
        T, Hq, Hkv, D, live = c["T"], c["Hq"], c["Hkv"], c["D"], c["T"] - c["skip"]
        read = 2 * D * (T * Hq + live * 2 * Hkv) + T * 4 * (c["axes"] + 1)
        write = T * Hq * D * (4 if c["q32"] else 2) + live * 2 * Hkv * D * 2
        return {"bytes": read + write, "flops": T * (Hq + Hkv) * (3 * c["rot"] + 4 * D)}
    plens, starts, lens = _prefix_lengths(c)
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    rows = sum(plens) + sum(lens)
    seen = sum(lens) + sum(n * (b - a) for n, a, b in zip(plens, starts, starts[1:]))
    return {"bytes": rows * Hkv * D * 4 + 2 * c["B"] * Hq * D * 2 + 4 * rows // c["block"],
            "flops": 4 * seen * Hq * D}


# --------------------------------------------------------- 64-bit answers
def _exact_rope(c, s):
    """Rotation as a product with a unit complex number, in 64 bits."""
    pos = s["positions"].double().reshape(c["axes"], c["T"])
    at = torch.cat([pos[a, :, None].expand(-1, n) for a, n in enumerate(s["sections"])], 1)
    turn = torch.polar(torch.ones_like(at), at * s["inv_freq"].double())[:, None]
    r = c["rot"]

    def rotated(x, w):
        x = x.double()
        if w is not None:
            x = x / ((x ** 2).sum(-1, keepdim=True) / c["D"] + s["eps"]).sqrt() * w.double()
        y = x.clone()
        if c["interleaved"]:
            z = torch.view_as_complex(x[..., :r].unflatten(-1, (r // 2, 2)).contiguous()) * turn
            y[..., :r] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * turn
            y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
        return y

    k_pool, v_pool = s["k_pool"].double(), s["v_pool"].double()
    k, live = rotated(s["k"], s["kw"]), s["slots"] >= 0
    block, row = s["slots"][live].long() // c["block"], s["slots"][live].long() % c["block"]
    k_pool[block, row] = k[live]
    v_pool[block, row] = s["v"][live].double()
    return rotated(s["q"], s["qw"]), k_pool, v_pool


def _exact_prefix(c, s):
    """All keys of a head's sequences side by side, one softmax over them."""
    B, Hkv, D, bs = c["B"], c["Hkv"], c["D"], c["block"]
    plens, starts, longest = s["host"]
    out = torch.zeros((B, Hkv, c["Hq"] // Hkv, D), dtype=torch.float64, device="cuda")
    q = s["q"].double().reshape(out.shape)
    own_at = torch.arange(longest, device="cuda")
    for p, (first, end) in enumerate(zip(starts, starts[1:] + [B])):
        plen = plens[p] if p < len(plens) else 0
        at = torch.arange(plen, device="cuda")
        shared = s["prefix_table"][p, at // bs].long() * bs + at % bs if plen else at
        for i in range(first, end, 64):
            n = min(64, end - i)
            mine = s["table"][i:i + n][:, own_at // bs].long() * bs + own_at % bs  # [n, S]
            hide = own_at >= s["seq_lens"][i:i + n, None]
            for h in range(Hkv):
                kh, vh = s["k_pool"].flatten(0, 1)[:, h], s["v_pool"].flatten(0, 1)[:, h]
                x = q[i:i + n, h]
                left = torch.einsum("ngd,sd->ngs", x, kh[shared].double())
                right = torch.einsum("ngd,nsd->ngs", x, kh[mine].double())
                right = right.masked_fill(hide[:, None], float("-inf"))
                w = torch.softmax(torch.cat([left, right], -1) * s["scale"], -1).nan_to_num(0.0)
                v_own = torch.where(hide[..., None], 0.0, vh[mine].double())
                out[i:i + n, h] = (torch.einsum("ngs,sd->ngd", w[..., :plen], vh[shared].double())
                                   + torch.einsum("ngs,nsd->ngd", w[..., plen:], v_own))
    return out.flatten(1, 2)


def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers: the plain form's are the definition's
    s = prepare(case, seed)
    return (_exact_rope if case["op"] == "rope" else _exact_prefix)(case, s)
