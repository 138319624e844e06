"""CPU oracle of the calls that feed a paged KV cache (numpy, 64 bits).

Written from the definitions alone, request by request and token by token; it
shares no code with the library.
"""
import numpy as np


def tables(cached, new, free_list, free_count, table, T, block_size, num_blocks, pos_base=None):
    """Returns (table, seq_lens, token_start, slots, positions, free_left)."""
    table = np.array(table, dtype=np.int64)
    B, max_blocks = table.shape
    left = [int(x) for x in free_list[:max(0, min(int(free_count), len(free_list)))]]
    total, asked = len(left), 0
    seq_lens, start = [], [0]
    slots, positions = [-1] * T, [0] * T
    for b in range(B):
        have, more = max(int(cached[b]), 0), max(int(new[b]), 0)
        start.append(start[-1] + more)
        held, want = -(-have // block_size), -(-(have + more) // block_size)
        fits = want <= max_blocks and start[-1] <= T
        need = want - held if fits else 0
        asked += need
        served = fits and (need == 0 or asked <= total)
        if served:
            for i in range(need):
                table[b, held + i] = left.pop()
        seq_lens.append(have + more if served else have)
        for i in range(more):
            t, row = start[b] + i, have + i
            if t >= T:
                break
            positions[t] = row + (int(pos_base[b]) if pos_base is not None else 0)
            if served:
                block = int(table[b, row // block_size])
                if 0 <= block < num_blocks:
                    slots[t] = block * block_size + row % block_size
    return (table, np.array(seq_lens), np.array(start), np.array(slots, dtype=np.int64),
            np.array(positions, dtype=np.int64), len(left))


def norm_rotate(x, weight, eps, weight_offset, positions, inv_freq, sections, interleaved):
    """x [T, H, D] float64, positions [axes, T]. Returns the normed and rotated
    heads and, element by element, |a| + |b| of the rotated pair (|y| outside)."""
    x = np.array(x, dtype=np.float64)
    if weight is not None:
        r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
        x = x * r * (np.asarray(weight, dtype=np.float64) + weight_offset)
    y, size = x.copy(), np.abs(x)
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    half = len(inv_freq)
    for i, f in enumerate(np.asarray(inv_freq, dtype=np.float64)):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        # position (below 2^29) * fp32 frequency is exact in 64 bits.
        w = (np.asarray(positions[axis[i]], dtype=np.float64) * f)[:, None]
        y[..., a] = x[..., a] * np.cos(w) - x[..., b] * np.sin(w)
        y[..., b] = x[..., b] * np.cos(w) + x[..., a] * np.sin(w)
        size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, size
