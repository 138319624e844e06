"""CPU oracle of decode attention with shared prefixes over a paged cache
(numpy, 64 bits), written from the definition: for each sequence the rows of
its group's prefix and its own rows, side by side, and one softmax over them.
"""
import numpy as np


def rows_of(pool, table_row, n, block_size):
    """The first n rows [n, Hkv, D] that a table row lists; zeros outside the pool."""
    out = np.zeros((n,) + pool.shape[2:], dtype=np.float64)
    for c in range(n):
        block = int(table_row[c // block_size])
        if 0 <= block < pool.shape[0]:
            out[c] = pool[block, c % block_size]
    return out


def attention(q, k_pool, v_pool, prefix_table, prefix_lens, group_start, block_table, seq_lens,
              scale):
    """q [B, Hq, D] and pools [blocks, block_size, Hkv, D] float64. Returns out
    and, element by element, the weighted sum of |V|."""
    B, Hq, D = q.shape
    _, bs, Hkv, _ = k_pool.shape
    G = Hq // Hkv
    P = 0 if prefix_table is None else len(prefix_table)
    starts = [0, B] if group_start is None else list(np.maximum.accumulate(
        np.clip(np.asarray(group_start), 0, B)))
    out, size = np.zeros_like(q), np.zeros_like(q)
    shared = {}
    for b in range(B):
        ks, vs = [], []
        for p in range(P):
            if starts[p] <= b < starts[p + 1]:
                if p not in shared:
                    n = min(max(int(prefix_lens[p]), 0), len(prefix_table[p]) * bs)
                    shared[p] = [rows_of(x, prefix_table[p], n, bs) for x in (k_pool, v_pool)]
                ks.append(shared[p][0])
                vs.append(shared[p][1])
        if block_table is not None:
            cap = block_table.shape[1] * bs
            n = cap if seq_lens is None else min(max(int(seq_lens[b]), 0), cap)
            ks.append(rows_of(k_pool, block_table[b], n, bs))
            vs.append(rows_of(v_pool, block_table[b], n, bs))
        k = np.concatenate(ks) if ks else np.zeros((0, Hkv, D))
        v = np.concatenate(vs) if vs else np.zeros((0, Hkv, D))
        if len(k) == 0:
            continue
        for h in range(Hq):
            s = scale * (k[:, h // G] @ q[b, h])
            w = np.exp(s - s.max())
            w /= w.sum()
            out[b, h] = w @ v[:, h // G]
            size[b, h] = w @ np.abs(v[:, h // G])
    return out, size
