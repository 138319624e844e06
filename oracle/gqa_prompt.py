"""CPU oracle of attention of several new tokens a sequence over a paged cache
(numpy, 64 bits), written from the definition: for each token the rows that it
sees, one softmax over them, and nothing of the others.
"""
import numpy as np

from .gqa_prefix import rows_of


def attention(q, k_pool, v_pool, token_start, cached_lens, tree_mask, block_table, seq_lens, scale,
              out):
    """q [T, Hq, D] and pools [blocks, block_size, Hkv, D] float64; tree_mask None: causal.
    Returns out, with the tokens of all sequences written over what it holds, and, element by
    element, the weighted sum of |V|."""
    T, Hq, D = q.shape
    _, bs, Hkv, _ = k_pool.shape
    B, max_blocks = block_table.shape
    G, cap = Hq // Hkv, max_blocks * bs
    out, size = np.array(out, dtype=np.float64), np.zeros(q.shape)
    start = np.maximum.accumulate(np.clip(np.asarray(token_start, dtype=np.int64), 0, T))
    for b in range(B):
        n = int(start[b + 1] - start[b])
        have = 0 if cached_lens is None else min(max(int(cached_lens[b]), 0), cap)
        L = have + n if seq_lens is None else max(int(seq_lens[b]), 0)
        L = min(L, cap)
        if n == 0:
            continue
        need = min(L, have + n)
        k, v = (rows_of(x, block_table[b], need, bs) for x in (k_pool, v_pool))
        for i in range(n):
            t = int(start[b]) + i
            if tree_mask is None:
                sees = np.arange(min(have + i + 1, L))
            else:
                words = [int(w) & 0xffffffff for w in tree_mask[t]]
                drafts = [j for j in range(min(n, 32 * len(words))) if words[j // 32] >> j % 32 & 1]
                sees = np.array(list(range(min(have, L))) + [have + j for j in drafts if have + j < L],
                                dtype=np.int64)
            if len(sees) == 0:
                out[t] = 0.0
                continue
            for h in range(Hkv):
                heads = slice(h * G, (h + 1) * G)
                s = scale * (q[t, heads] @ k[sees, h].T)
                w = np.exp(s - s.max(axis=1, keepdims=True))
                w /= w.sum(axis=1, keepdims=True)
                out[t, heads] = w @ v[sees, h]
                size[t, heads] = w @ np.abs(v[sees, h])
    return out, size
