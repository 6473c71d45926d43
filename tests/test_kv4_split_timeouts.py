"""The ring of a pair of warps in the 4-bit cache's split attention kernel when waits run out, as a model with a clock (CPU).

Copies from some page on never come, and a wait gives up after its limit.  One warp of the pair may give up while the other still goes
on: it asks for no more pages, so nothing is copied over what it has not read.  Before it goes on without the ring a
warp waits, within one limit for all of them, for the pages that it asked for.  So when both warps are there no copy is under way, and the pair
is there within a few limits, however deep the ring.
"""
import random

import pytest

LIMIT, FLIGHT = 4000, 50                                             # ticks: of a wait; a copy's longest way


class Pair:
    def __init__(self, units, depth, lost, rng, batch):
        self.units, self.depth, self.lost, self.rng, self.batch = units, depth, lost, rng, batch
        self.now, self.used, self.phase = 0, [0] * depth, [0] * depth
        self.holds, self.reading = [None] * depth, [[False, False] for _ in range(depth)]
        self.flying, self.read, self.gave_up = [], [0, 0], [None, None]

    def copy(self, entry, order):
        assert not any(self.reading[entry]), "refilled while it is read"
        assert min(self.read) >= order - self.depth + 1, "refilled before both are done"
        assert all(e != entry for e, _, _ in self.flying)
        if order < self.lost:
            self.flying.append((entry, order, self.now + self.rng.randint(1, FLIGHT)))

    def tick(self):
        self.now += 1
        for f in [f for f in self.flying if f[2] <= self.now]:
            self.flying.remove(f)
            self.holds[f[0]] = f[1]
            self.phase[f[0]] += 1

    def wait(self, entry, parity, until):
        """Yields until the phase has completed or the time is over; whether it has completed."""
        while self.phase[entry] % 2 == parity:
            if self.now >= until:
                return False
            yield
        return True

    def warp(self, side):
        ok, jl, entry_in, in_ring, asked, out, parity, base = True, 0, 0, 0, 0, 0, 0, 0
        units = self.units
        for j in range(len(units)):
            if j - base == self.batch:
                base += self.batch
            while ok and in_ring < self.depth and jl < len(units) and jl < base + 2 * self.batch:
                here = units[jl]
                jl += 1
                if not here:
                    continue
                yield
                if asked < self.depth:
                    mine = side == 0
                else:
                    self.used[entry_in] += 1
                    mine = self.used[entry_in] % 2 == 0
                if mine:
                    self.copy(entry_in, asked)
                asked, in_ring, entry_in = asked + 1, in_ring + 1, (entry_in + 1) % self.depth
            if not units[j] or not ok:
                continue
            ok = yield from self.wait(out, parity, self.now + LIMIT)
            if ok:
                assert self.holds[out] == self.read[side], "a wait passed for another page"
                self.reading[out][side] = True
                for _ in range(self.rng.randint(0, 5)):
                    yield
                assert self.holds[out] == self.read[side]
                self.reading[out][side] = False
                self.read[side], in_ring = self.read[side] + 1, in_ring - 1
                out, parity = (out + 1) % self.depth, parity ^ (out + 1 == self.depth)
                continue
            self.gave_up[side] = self.now
            until = self.now + LIMIT                                 # one limit for all
            for _ in range(in_ring):
                yield from self.wait(out, parity, until)
                out, parity = (out + 1) % self.depth, parity ^ (out + 1 == self.depth)


def _run(units, depth, lost, rng, batch):
    pair = Pair(units, depth, lost, rng, batch)
    warps, alive, slow = [pair.warp(0), pair.warp(1)], [True, True], rng.choice([(1, 1), (1, 3), (3, 1)])
    while any(alive):
        for i in range(2):
            if alive[i] and rng.randrange(slow[i]) == 0:
                try:
                    next(warps[i])
                except StopIteration:
                    alive[i] = False
        pair.tick()
    assert not pair.flying, "a copy under way when both go on without the ring"
    pages = sum(units)
    if lost >= pages:
        assert pair.read == [pages, pages] and pair.gave_up == [None, None]
    else:
        assert None not in pair.gave_up and max(pair.read) <= lost
        assert pair.now - min(pair.gave_up) <= 3 * LIMIT, "not there within three limits"
    return pair.gave_up


@pytest.mark.parametrize("depth", [3, 6, 12])
def test_pair_whose_waits_run_out(depth):
    rng = random.Random(depth)
    apart = 0
    for trial in range(60):
        units = [rng.random() < rng.choice([1.0, 0.6]) for _ in range(rng.choice([1, depth, depth + 1, rng.randint(1, 60)]))]
        up = _run(units, depth, rng.randint(0, sum(units) + 1), rng, rng.choice([2, 4, 32]))
        apart += None not in up and abs(up[0] - up[1]) > 2
    assert apart > 5                                                 # one gave up while the other went on


def test_one_warp_gives_up_alone():
    """Warp 1 stops for longer than the limit in front of a page that is there: warp 0 then waits for a page that nobody copies."""
    for depth in (3, 6):
        pair = Pair([True] * 30, depth, 30, random.Random(1), 32)
        warps, alive = [pair.warp(0), pair.warp(1)], [True, True]
        stopped = 0
        while any(alive):
            for i in range(2):
                if alive[i] and not (i == 1 and pair.read[1] == 4 and stopped < 2 * LIMIT):
                    try:
                        next(warps[i])
                    except StopIteration:
                        alive[i] = False
            stopped += pair.read[1] == 4
            pair.tick()
            assert pair.now < 20 * LIMIT
        assert not pair.flying and pair.gave_up[0] is not None
