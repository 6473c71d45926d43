"""The ring of a pair of warps in the 4-bit cache's split attention kernel (kv4_attn.cuh), as a model (CPU).

Both warps go through the same units.  Each asks for pages ahead of where it is; a ring entry's first page is copied by warp 0, every
later one by whichever warp asks second (the parity of a counter), which it does when it is done with the entry's old page.  Over random
interleavings and copy times: a page is copied once, into an entry that both warps are done with, a wait by parity is for
the right page, and the pair always gets to the end.
"""
import os
import random

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4a8_verify_gb300", "csrc", "kv4_attn.cuh")


class Pair:
    def __init__(self, units, depth, batch=32):
        self.units, self.depth, self.batch = units, depth, batch     # units: page number, or -1 (nothing to copy)
        self.used = [0] * depth
        self.holds = [None] * depth                                  # page that an entry was last filled with
        self.phase = [0] * depth                                     # completed copies of an entry
        self.reading = [[False, False] for _ in range(depth)]
        self.done = [set(), set()]                                   # order numbers of the pages a warp is done with
        self.flying, self.copied = [], []

    def copy(self, entry, order, page):
        assert not any(self.reading[entry]), "refilled while it is read"
        if order >= self.depth:
            assert all(order - self.depth in d for d in self.done), "refilled before both are done"
        assert all(e != entry for e, _, _ in self.flying)
        self.flying.append((entry, order, page))
        self.copied.append(order)

    def land(self, i):
        entry, order, page = self.flying.pop(i)
        self.holds[entry] = (order, page)
        self.phase[entry] += 1

    def warp(self, side):
        """A generator: every yield lets others run; yields a condition to wait for, or None."""
        units, jl, entry_in, in_ring, asked, out, parity, read, base = self.units, 0, 0, 0, 0, 0, 0, 0, 0
        for j in range(len(units)):
            if j - base == self.batch:
                base += self.batch
            while in_ring < self.depth and jl < len(units) and jl < base + 2 * self.batch:
                page = units[jl]
                jl += 1
                if page < 0:
                    continue
                yield None
                if asked < self.depth:
                    mine = side == 0
                else:
                    self.used[entry_in] += 1
                    mine = self.used[entry_in] % 2 == 0
                if mine:
                    self.copy(entry_in, asked, page)
                asked, in_ring, entry_in = asked + 1, in_ring + 1, (entry_in + 1) % self.depth
            if units[j] < 0:
                continue
            yield lambda e=out, p=parity: self.phase[e] % 2 != p     # phase p has completed
            assert self.holds[out] == (read, units[j]), "a wait passed for another page"
            self.reading[out][side] = True
            yield None
            assert self.holds[out] == (read, units[j])
            self.reading[out][side] = False
            self.done[side].add(read)
            read, in_ring = read + 1, in_ring - 1
            out += 1
            if out == self.depth:
                out, parity = 0, parity ^ 1


def _run(units, depth, rng, batch):
    pair = Pair(units, depth, batch)
    warps = [pair.warp(0), pair.warp(1)]
    blocked, alive = [None, None], [True, True]
    slow = rng.choice([0.5, 0.1, 0.9])
    while any(alive):
        ready = [i for i in range(2) if alive[i] and (blocked[i] is None or blocked[i]())]
        assert ready or pair.flying, "nobody can go on"
        if pair.flying and (not ready or rng.random() < slow):
            pair.land(rng.randrange(len(pair.flying)))
            continue
        i = rng.choice(ready) if rng.random() < 0.7 else ready[0]
        try:
            blocked[i] = next(warps[i])
        except StopIteration:
            alive[i] = False
    assert pair.copied == list(range(sum(u >= 0 for u in units))) and not pair.flying


@pytest.mark.parametrize("depth", [3, 6, 12])
@pytest.mark.parametrize("missing", [0.0, 0.3, 0.95])
def test_ring_of_a_pair(depth, missing):
    rng = random.Random(depth * 100 + int(missing * 100))
    for trial in range(150):
        n = rng.choice([1, 2, depth, depth + 1, rng.randint(1, 60)])
        units = [-1 if rng.random() < missing else i for i in range(n)]
        _run(units, depth, rng, rng.choice([2, 4, 32]))


def test_the_source_follows_the_model():
    text = " ".join(open(SRC).read().split())
    for step in ("while (ok && in_ring < NS && jl < nu && jl < cbase + 64)",
                 "if (lane == 0 && (asked < NS ? side == 0 : second(&used[is])))",
                 "atom.acq_rel.cta.shared::cta.add.u32", "return (old & 1u) != 0;",
                 "ok = __all_sync(FULL, mbar_wait(&full[cs], cph, geo.wait_ns));",
                 "if (++cs == NS) cs = 0, cph ^= 1; --in_ring;"):
        assert step in text, step
    assert text.index("half(ring + cs * C::PAGE, left);") < text.index("__syncwarp(); if (++cs == NS)")
