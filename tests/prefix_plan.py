"""A model of the plan that gqa_prefix_attn_decode makes on the device: how a
batch's prefixes and own rows are cut into units, and how many key tiles each
stream of a unit takes. Plain numbers; it launches nothing. The tests use it to
say which paths of the kernel a case runs.
"""
import math
from collections import namedtuple

import numpy as np

SPLIT, PAIR, OWN = "split", "pair", "own"
# mode, whether of a sequence's own rows, key tiles of the two streams
Unit = namedtuple("Unit", "mode own tiles")
Plan = namedtuple("Plan", "units group_splits pairs cut own_tiles costs")

F = np.float32
C_UNIT = F(4000)


def up(a, b):
    return -(-a // b)


def costs(D):
    """Cycles of a key tile: two query tiles, one, a sequence's own rows."""
    if D == 64:
        return F(2850), F(1450), F(1400)
    return F(3100), F(1580 if D == 128 else 1480), F(2800)


def plan(B, Hq, Hkv, D, plens, starts, lens, sms=152):
    G = Hq // Hkv
    TB, NS, KEYS = 128 // G, (1 if D == 256 else 2), (64 if D == 256 else 128)
    c_pair, c_tile, c_own = costs(D)
    P = len(plens)
    if starts is None:
        starts = [0, B]
    groups = [(min(max(starts[p], 0), B), min(max(starts[p + 1], 0), B)) for p in range(P)]
    own = [up(max(0, n), KEYS) for n in lens]
    work = F(sum(own) * Hkv)
    each = min(max(1, math.ceil(float(work) * 1.00001 / ((2 if NS == 1 else 4) * sms))), 1 << 20)
    own_units = sum(up(t, each) for t in own) * Hkv
    paired = NS == 2 and own_units > sms

    q = [up(max(0, e - a), TB) for a, e in groups]
    tiles = [up(max(0, n), KEYS) if m else 0 for n, m in zip(plens, q)]
    longest = max(tiles, default=0)
    slots = (up(B, TB) + min(P, B)) * Hkv + 2 * sms if P else 0
    units, best, table = [], None, []
    if longest:
        for lane in range(32):
            pairs = NS == 2 and lane & 1
            width = [(m + 1) // 2 if pairs else m for m in q]
            w = float(sum(t * m for t, m in zip(tiles, width)) * Hkv)
            chunk = math.ceil(w / (((lane >> 2) + 1) * sms)) + ((lane >> 1) & 1)
            chunk = longest if lane >= 30 else max(1, min(chunk, longest))
            n = float(sum(up(t, chunk) * m for t, m in zip(tiles, width)) * Hkv)
            c = float(c_pair if pairs else c_tile)
            one = chunk * c + float(C_UNIT)
            everything = (w * c + n * float(C_UNIT) + float(work) * float(c_own)) / sms
            rounds = math.ceil((n - 0.5) / sms)
            est = max(everything, rounds * one) if n <= slots else math.inf
            table.append((est, lane, chunk, int(n)))
            if best is None or est < best[0]:
                best = table[-1] + (pairs,)
        _, lane, cut, _, pairs = best
        for t, m in zip(tiles, q):
            s = up(t, cut)
            pr = bool(pairs) and m > 1
            for i in range(s):
                n = t // s + (i < t % s)
                for j in range(up(m, 2) if pr else m):
                    if pr and 2 * j + 1 < m:
                        units += [Unit(PAIR, False, (n, n))] * Hkv
                    else:
                        units += [Unit(SPLIT, False, split(n, NS))] * Hkv
    parts = []
    for t in own:
        s = up(t, each)
        parts += [t // s + (i < t % s) for i in range(s)] * Hkv if s else []
    if paired:
        parts += [0] * (len(parts) % 2)
        units += [Unit(OWN, True, pair) for pair in zip(parts[::2], parts[1::2])]
    else:
        units += [Unit(SPLIT, True, split(n, NS)) for n in parts]
    return Plan(units, [up(t, best[2]) if best else 0 for t in tiles], bool(best and best[4]),
                best[2] if best else 0, each, table)


def split(n, streams):
    """Key tiles of the two streams when one query tile takes both."""
    return (n, 0) if streams == 1 else ((n + 1) // 2, n // 2)
