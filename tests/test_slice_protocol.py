"""The copy slices of the scored decode kernel (decode_mma, kWarpSlices), checked
on the CPU under random schedules.

The model has the copy protocol and none of the arithmetic.  Each of 4 warps has a
barrier of its own for each of STAGES (2 or 3) stages and fetches its slice of a
stage itself: tile 0 before the context's length is known, the rest of the first
wave (sized before it too) behind a block barrier, then, each time it has read a
tile, the tile STAGES on into the slice it has just left.  It waits for tile it + 1
with parity ((it + 1) / STAGES) & 1 while it still reads tile it.  A tile behind the
real end expects no bytes, so its phase completes at once.  At the end it waits for
the last STAGES tiles it may have issued; then the four meet, and the stages are
written over by the merge.  A split that lies wholly behind the end waits for its
tile 0 and leaves.

Checked in every schedule: a wait returns only when the warp's own tile has landed;
no copy lands in a slice that is still read; none is in flight when the stages are
written over or the CTA leaves; nothing deadlocks.  Planted mistakes are caught: a
refill before the tile is read, a parity off by one, an empty split that leaves
without waiting."""
import random

import pytest

WARPS = 4


class Warp:
    """One warp's slices: an iterator that yields whenever another party may run."""

    def __init__(self, stages, n_pre, n_tiles, plant):
        self.S, self.n_first, self.n, self.plant = stages, min(n_pre, stages), n_tiles, plant
        self.phase = [0] * stages            # completed phases of each slice's barrier
        self.in_flight, self.landed, self.reading = [], [None] * stages, set()

    def issue(self, t, known=True):
        if known and t >= self.n:            # nothing there: the phase completes without a byte
            self.phase[t % self.S] += 1
            self.landed[t % self.S] = t
        else:
            self.in_flight.append(t)

    def land(self, i):
        t = self.in_flight.pop(i)
        assert all(r % self.S != t % self.S for r in self.reading), f"tile {t} lands in a slice that is read"
        self.landed[t % self.S] = t
        self.phase[t % self.S] += 1

    def wait(self, t, shift=0):
        parity = (t // self.S + shift) & 1
        while (self.phase[t % self.S] & 1) == parity:
            yield "wait"
        assert self.landed[t % self.S] == t, f"tile {t} taken for landed"

    def run(self):
        if self.n_first > 0:
            self.issue(0, known=False)       # (behind the end it fetches what the table names there)
        yield "barrier"
        if self.n == 0:
            if self.n_first > 0 and self.plant != "empty":
                yield from self.wait(0)
            return
        for t in range(1, self.n_first):
            self.issue(t)
            yield
        yield from self.wait(0)
        self.reading.add(0)
        for t in range(self.n):
            if t + 1 < self.n:
                yield from self.wait(t + 1, 1 if self.plant == "parity" and t + 1 >= self.S else 0)
                self.reading.add(t + 1)
            yield
            if self.plant == "early" and t + self.S < self.n:
                self.issue(t + self.S)
                yield
            self.reading.discard(t)
            if self.plant != "early" and t + self.S < self.n:
                self.issue(t + self.S)
            yield
        last = max(self.n, self.n_first)
        for t in range(max(0, last - self.S), last):
            yield from self.wait(t)
        yield "barrier"
        yield "merge"


def schedule(stages, n_pre, n_tiles, rng, plant=None):
    warps = [Warp(stages, n_pre, n_tiles, plant) for _ in range(WARPS)]
    runs = [w.run() for w in warps]
    at = [None] * WARPS                      # what each warp last yielded, "done" at its end
    held = set()                             # warps at a block barrier
    idle = 0
    while any(a != "done" for a in at) or any(w.in_flight for w in warps):
        moves = [("run", i) for i in range(WARPS) if at[i] != "done" and i not in held]
        moves += [("land", i) for i in range(WARPS) if warps[i].in_flight]
        assert moves and idle < 20000, "deadlock"
        what, i = rng.choice(moves)
        if what == "land":
            warps[i].land(rng.randrange(len(warps[i].in_flight)))
            idle = 0
            continue
        before = at[i]
        at[i] = next(runs[i], "done")
        idle = idle + 1 if at[i] == before == "wait" else 0
        if at[i] == "barrier":
            held.add(i)
            if len(held) == WARPS:
                held.clear()
        if at[i] == "merge":
            assert not any(w.in_flight for w in warps), "the merge writes over a slice that a copy is on its way to"
        if at[i] == "done":
            assert not warps[i].in_flight, "a copy in flight when its warp leaves"


@pytest.mark.parametrize("stages", [2, 3])
@pytest.mark.parametrize("n_tiles", [0, 1, 2, 3, 4, 5, 8, 13])
def test_random_schedules(stages, n_tiles):
    for seed in range(60):
        rng = random.Random(seed)
        # the length found may be any at or below what was assumed
        schedule(stages, n_tiles + rng.choice([0, 0, 1, 2, 5]), n_tiles, rng)


@pytest.mark.parametrize("plant", ["early", "parity", "empty"])
def test_planted_mistakes_are_caught(plant):
    caught = 0
    for seed in range(200):
        rng = random.Random(seed)
        n_tiles = 0 if plant == "empty" else rng.choice([4, 7])
        try:
            schedule(rng.choice([2, 3]), n_tiles + 2, n_tiles, rng, plant)
        except AssertionError:
            caught += 1
    assert caught > 20
