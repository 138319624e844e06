"""CPU oracle of forks, accepted drafts and released blocks of a paged KV cache,
written from the definitions, request by request; it shares no code with the
library.
"""
import numpy as np


def fork(pools, parent, child, table, seq_lens, shares, free_list, free_count):
    """Returns (pools, table, seq_lens, shares, fork_block, free_left)."""
    pools = [np.array(p) for p in pools]
    table, seq_lens, shares = (np.array(x, dtype=np.int64) for x in (table, seq_lens, shares))
    B, max_blocks = table.shape
    nb, bs = pools[0].shape[:2]
    left = [int(x) for x in free_list[:max(0, min(int(free_count), len(free_list)))]]
    parents = {int(a) for a in parent if 0 <= a < B}
    named, asked, total, taken = set(), 0, len(left), 0
    out = []
    for a, c in zip((int(x) for x in parent), (int(x) for x in child)):
        good = 0 <= a < B and 0 <= c < B and c not in named and c not in parents
        named.add(c)
        if not good:
            out.append(-2)
            continue
        L = min(max(int(seq_lens[a]), 0), max_blocks * bs)
        full, rest = divmod(L, bs)
        asked += rest > 0
        if rest and asked > total:
            out.append(-2)
            continue
        table[c, :full] = table[a, :full]
        for x in table[a, :full]:
            if 0 <= x < nb:
                shares[x] += 1
        block = -1
        if rest:
            block = left.pop()
            taken += 1
            block = 2 ** 31 - 1 if block < 0 else block
            src = int(table[a, full])
            if 0 <= block < nb and 0 <= src < nb:
                for p in pools:
                    p[block, :rest] = p[src, :rest]
            table[c, full] = block
        seq_lens[c] = L
        out.append(block)
    return pools, table, seq_lens, shares, np.array(out, dtype=np.int64), total - taken


def keep(pools, cached, accepted, count, table, seq_lens):
    """Returns (pools, kept_lens)."""
    pools = [np.array(p) for p in pools]
    old = [np.array(p) for p in pools]
    B, max_blocks = np.shape(table)
    nb, bs = pools[0].shape[:2]
    cap, kept = max_blocks * bs, []
    for b in range(B):
        have, end = min(max(int(cached[b]), 0), cap), min(int(seq_lens[b]), cap)
        n, last = 0, -1
        while n < min(int(count[b]), len(accepted[b])):
            a = int(accepted[b][n])
            if a <= last or have + a >= end:
                break
            src, dst = int(table[b][(have + a) // bs]), int(table[b][(have + n) // bs])
            if 0 <= src < nb and 0 <= dst < nb:
                for p, o in zip(pools, old):
                    p[dst, (have + n) % bs] = o[src, (have + a) % bs]
            last, n = a, n + 1
        kept.append(have + n)
    return pools, np.array(kept, dtype=np.int64)


def release(table, old_lens, new_lens, shares, free_list, free_count, num_blocks, block_size):
    """Returns (shares, free_list, free_left)."""
    free_list = np.array(free_list, dtype=np.int64)
    counts = np.zeros(num_blocks, dtype=np.int64) if shares is None else np.array(shares, dtype=np.int64)
    B, max_blocks = np.shape(table)
    n = max(0, min(int(free_count), len(free_list)))
    order, let_go = [], {}
    for b in range(B):
        old = min(max(int(old_lens[b]), 0), max_blocks * block_size)
        new = min(max(int(new_lens[b]), 0), old)
        for j in range(-(-new // block_size), -(-old // block_size)):
            x = int(table[b][j])
            if 0 <= x < num_blocks:
                if x not in let_go:
                    order.append(x)
                let_go[x] = let_go.get(x, 0) + 1
    for x in order:
        if let_go[x] > counts[x]:
            counts[x] = 0
            if n < len(free_list):
                free_list[n] = x
                n += 1
        else:
            counts[x] -= let_go[x]
    return (None if shares is None else counts), free_list, n
