"""Batches whose units hold several key tiles a stream, for each way in which
gqa_prefix_attn_decode runs a unit."""
from prefix_plan import OWN, PAIR, SPLIT, plan

# name: D, B, G, Hkv, prefix lengths, group starts, own lengths, (mode, own rows, key tiles of the
# shorter and the longer stream that some unit has at least)
SHORT = [0, 1, 128, 200]
LONG = [100, 2300, 40, 3000, 129, 2650, 300, 3999, 1, 2049]
CASES = {
    "single-d64": (64, 20, 48, 1, [16390], None, SHORT * 5, (SPLIT, False, 4, 5)),
    "single-d128": (128, 20, 48, 1, [16390], None, SHORT * 5, (SPLIT, False, 4, 5)),
    "single-d256": (256, 3, 3, 2, [16390], None, SHORT[1:], (SPLIT, False, 0, 4)),
    "pair-d64": (64, 26, 48, 2, [6001], None, SHORT * 6 + [5, 9], (PAIR, False, 4, 4)),
    "pair-d128": (128, 26, 48, 2, [6001], None, SHORT * 6 + [5, 9], (PAIR, False, 4, 4)),
    "own-d64": (64, 40, 5, 7, [], None, LONG * 4, (OWN, True, 4, 6)),
    "own-d128": (128, 40, 4, 7, [100], [3, 9], LONG * 4, (OWN, True, 4, 6)),
    "own-d256": (256, 20, 8, 4, [], None, LONG * 2, (SPLIT, True, 0, 5)),
}


def case_plan(name, sms=152):
    D, B, G, Hkv, plens, starts, lens, _ = CASES[name]
    return plan(B, G * Hkv, Hkv, D, plens, starts, lens, sms)


def reaches(name, sms=152):
    """Units of the wanted kind, in the plan for this many SMs."""
    mode, own, short, long = CASES[name][-1]
    return [u for u in case_plan(name, sms).units
            if u.mode == mode and u.own == own and min(u.tiles) >= short and max(u.tiles) >= long]
