"""The model of the attention call's plan (tests/prefix_plan.py): it has the
library's constants, it covers every key tile once within the slots that the
host sets aside, and the GPU tests' batches reach what they are for (CPU only)."""
import os
import random
import re

import pytest

import prefix_plan
from prefix_plan import OWN, PAIR, plan, up
from prefix_tile_cases import CASES, case_plan, reaches

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "gqa_attention_weighted_gb300", "csrc")


def source(name):
    return open(os.path.join(CSRC, name)).read()


def test_constants_are_the_library_s():
    api = source("gqa_prefix_api.cu")

    def cost(name, D):
        """The value that a chain of `D == n ? a : b` takes."""
        text = re.search(rf"p\.{name} = (.*?);", api, flags=re.S).group(1)
        while "?" in text:
            size, yes, text = re.match(r"D == (\d+) \? ([\d.]+)f : (.*)", text).groups()
            if int(size) == D:
                return float(yes)
        return float(text.strip("f"))

    for D in (64, 128, 256):
        pair, tile, own = (float(x) for x in prefix_plan.costs(D))
        assert (cost("c_tile", D), cost("c_own", D)) == (tile, own)
        if D < 256:                              # one stream: no pairs
            assert cost("c_pair", D) == pair
        assert cost("c_unit", D) == float(prefix_plan.C_UNIT)
    kernel = source("gqa_prefix_kernel.cuh")
    assert "fmaxf(all, rounds * one)" in kernel  # no factor on the busiest CTA


def random_batch(rng):
    D = rng.choice([64, 128, 256])
    G, Hkv, B = rng.choice([1, 3, 8, 48, 128]), rng.choice([1, 2, 8]), rng.randint(1, 300)
    P = rng.choice([0, 1, 1, 3, 32])
    starts = sorted(rng.randint(0, B) for _ in range(P + 1)) if P else None
    plens = [int(10 ** rng.uniform(0, 4.6)) * rng.choice([0, 1, 1]) for _ in range(P)]
    lens = [int(10 ** rng.uniform(0, rng.choice([2, 4]))) * rng.choice([0, 1, 1]) for _ in range(B)]
    return B, G * Hkv, Hkv, D, plens, starts, lens


@pytest.mark.parametrize("seed", range(60))
def test_every_key_tile_is_taken_once_within_the_slots(seed):
    B, Hq, Hkv, D, plens, starts, lens = random_batch(random.Random(seed))
    sms = (152, 148, 20)[seed % 3]
    p = plan(B, Hq, Hkv, D, plens, starts, lens, sms)
    keys, TB = 64 if D == 256 else 128, 128 // (Hq // Hkv)
    own = [u for u in p.units if u.own]
    prefix = [u for u in p.units if not u.own]
    took = sum(sum(u.tiles) for u in own)
    assert took == sum(up(max(0, n), keys) for n in lens) * Hkv
    want = 0
    for g, n in enumerate(plens):
        q = up(max(0, starts[g + 1] - starts[g]), TB)
        want += up(n, keys) * q * Hkv
    assert sum(sum(u.tiles) for u in prefix) == want      # a pair: both streams, a query tile each
    own_units = sum(2 - (min(u.tiles) == 0) if u.mode == OWN else 1 for u in own)
    assert own_units <= B * Hkv + 4 * sms
    assert len(prefix) <= (up(B, TB) + min(len(plens), B)) * Hkv + 2 * sms
    assert all(u.tiles[0] == u.tiles[1] for u in prefix if u.mode == PAIR)


@pytest.mark.parametrize("name", CASES)
def test_batches_reach_units_of_several_key_tiles(name):
    assert len(reaches(name)) >= 8
    if CASES[name][-1][0] == OWN:                         # and pairs that end apart
        assert len([u for u in case_plan(name).units
                    if u.mode == OWN and abs(u.tiles[0] - u.tiles[1]) >= 2]) >= 4
