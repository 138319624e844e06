"""A model of the barriers between the MMA warp and the two softmax warpgroups of
gqa_prefix_attn_decode's kernel, run under random schedules (CPU only).

A barrier's phase completes with its last arrival; a wait names a parity and
passes when the barrier's current phase has the other one. So a wait goes wrong
when an arriver is two phases ahead of it (it never passes) or behind it (it
passes too early). The roles below make the kernel's waits and arrivals in its
order; the key tiles' own barriers (scores, weights) are kept, loads are always
ready.
"""
import os
import random

import pytest

SPLIT, PAIR, OWN = "split", "pair", "own"
KERNEL = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "gqa_attention_weighted_gb300", "csrc", "gqa_prefix_kernel.cuh")


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1


class Early(Exception):
    """A wait passed before the phase that it is for was complete."""


def streams(unit):
    mode, a, b = unit
    return ((a + 1) // 2, a // 2) if mode == SPLIT else (a, a) if mode == PAIR else (a, b)


def wait(bar, phase):
    """Steps until the wait for this phase's parity passes."""
    while bar.phase & 1 == phase & 1:
        yield False
    if bar.phase <= phase:
        raise Early
    yield True


def mma(units, bars, old_rule):
    for w in range(2):
        yield from wait(bars["ofree", w], 0)
    done = [0, 0]
    for u, unit in enumerate(units):
        mode, n = unit[0], streams(unit)
        if n[1] == 0 and (mode == SPLIT or old_rule):
            yield from wait(bars["ofree", 1], u)
        for t in range(-2, 2 * max(n)):
            w, j = t & 1, t >> 1
            if 0 <= j < n[w]:                              # product with V
                yield from wait(bars["pfull", w], done[w] + j)
                if j == 0:
                    yield from wait(bars["ofree", w], u)
                if j == n[w] - 1:
                    bars["ofull", w].arrive()
            if j + 1 < n[w]:                               # scores
                bars["sfull", w].arrive()
            yield True
        done = [done[0] + n[0], done[1] + n[1]]


def warp(w, units, bars, old_rule):
    """One of a warpgroup's four warps."""
    for b in range(2):                                     # the dry round, kOwn
        if b == w:
            bars["ofree", w].arrive()
            bars["ofree", w].arrive()
    yield True
    done, ends, meets = 0, [0, 0], 0
    for unit in units:
        mode, n = unit[0], streams(unit)
        for j in range(n[w]):
            yield from wait(bars["sfull", w], done + j)
            bars["pfull", w].arrive()
            yield True
        done += n[w]
        if n[0] > 0 and (w == 0 or mode == SPLIT):
            yield from wait(bars["ofull", 0], ends[0])
        if n[1] > 0 and (w == 1 or mode == SPLIT):
            yield from wait(bars["ofull", 1], ends[1])
        ends = [ends[0] + (n[0] > 0), ends[1] + (n[1] > 0)]
        if mode == SPLIT:
            bars["meet", 0].arrive()
            yield from wait(bars["meet", 0], meets)
            meets += 1
            bars["ofree", 0].arrive()
            bars["ofree", 1].arrive()
        elif n[w] > 0 or old_rule:
            bars["ofree", w].arrive()
            yield True
            bars["ofree", w].arrive()
        yield True


def run(units, seed, old_rule=False):
    """Whether all roles come to their end."""
    rng = random.Random(seed)
    bars = {(n, w): Barrier(c) for n, c in (("ofree", 8), ("ofull", 1), ("pfull", 4), ("sfull", 1),
                                            ("meet", 8)) for w in range(2)}
    roles = [mma(units, bars, old_rule)] + [warp(w, units, bars, old_rule) for w in (0, 1) for _ in range(4)]
    weight = [rng.choice([0.05, 1, 1, 20]) for _ in roles]  # some roles are slow
    blocked = set()                                        # since the last step of any role
    while roles and len(blocked) < len(roles):
        i = rng.choices(range(len(roles)), weight)[0]
        try:
            if next(roles[i]):
                blocked.clear()
            else:
                blocked.add(roles[i])
        except StopIteration:
            del roles[i], weight[i]
            blocked.clear()
    return not roles


def random_units(rng):
    """What a CTA may get: prefix units, then own units of one kind, the last perhaps single."""
    units = [rng.choice([(SPLIT, rng.randint(1, 5), 0), (PAIR, rng.randint(1, 3), 0)])
             for _ in range(rng.randint(0, 3))]
    if rng.random() < 0.7:
        units += [(OWN, rng.randint(1, 4), rng.randint(1, 4)) for _ in range(rng.randint(0, 3))]
        if rng.random() < 0.7:
            units.append((OWN, rng.randint(1, 4), 0))
    else:
        units += [(SPLIT, rng.randint(1, 3), 0) for _ in range(rng.randint(0, 3))]
    return units


@pytest.mark.parametrize("seed", range(50))
def test_every_schedule_ends(seed):
    units = random_units(random.Random(seed))
    assert all(run(units, 7 * seed + k) for k in range(3)), units


def test_a_wait_on_the_idle_stream_could_never_end():
    # What the kernel did before: a CTA's last unit without a second stream, as its first one too.
    for units in ([(OWN, 3, 1), (OWN, 2, 0)], [(OWN, 2, 0)]):
        assert not all(run(units, seed, old_rule=True) for seed in range(60))
        assert all(run(units, seed) for seed in range(60))


def test_the_kernel_has_the_rule_of_the_model():
    text = open(KERNEL).read()
    assert "if (n1 == 0 && mode == kSplit) ok = warp_poll(ofree0 + 8, unit_no & 1" in text
    assert text.count("warp_poll(ofree0 + 8,") == 2        # there, and for the dry round
    assert "} else if (dry || mine > 0) {" in text
