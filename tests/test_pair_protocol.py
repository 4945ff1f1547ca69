"""The two warps that share 32 rows of the scored chunk attention, and the merge of
its key splits by remote stores, checked on the CPU.

Pair: each tile a warp waits for its scores (a wait may run out, which it then knows
alone), then both come to a barrier that carries "lost, or my maximum rises".  If
either says so, both write their maximum and whether they are lost, meet again, and
read the other's: a loss ends the loop for both, a rise rescales O behind a wait
that may run out too; its warp goes on to the next tile, whose barrier tells the
other.  Checked under random schedules: both warps come to the same barriers the
same number of times (nothing deadlocks, whatever is lost), each reads what the
other wrote for this tile, and a loss leaves both lost, unless it is met in the
last tile, whose rows are NaN through the sums.  Planted mistakes are caught.

Merge: the 16-byte chunks of a row are shared out over the splits; the owner a
sender computes holds the chunk, and slabs stay apart and inside the stages."""
import random

import pytest


class Pair:
    def __init__(self, n_tiles, rng, chance, plant):
        self.n, self.rng, self.chance, self.plant = n_tiles, rng, chance, plant
        self.slot, self.flag = [None, None], [None, None]
        self.lost, self.barriers = [False, False], [[], []]

    def run(self, w):
        rng, o = self.rng, 1 - w
        for j in range(self.n):
            if not self.lost[w]:
                self.lost[w] = rng.random() < self.chance
            yield
            if self.plant == "leave" and self.lost[w]:
                return
            any_ = yield ("any", self.lost[w] or rng.random() < 0.5)
            if any_:
                self.slot[w], self.flag[w] = (w, j), self.lost[w]
                yield
                if self.plant != "no second barrier":
                    yield ("sync", False)
                yield
                assert self.slot[o] == (o, j), "the other warp's maximum is not this tile's"
                if self.flag[o]:
                    self.lost[w] = True
                yield
                if self.lost[w]:
                    return
                if j > 0 and rng.random() < 0.5:
                    self.lost[w] = rng.random() < self.chance
                    if self.lost[w]:
                        continue
            yield


def schedule(n_tiles, rng, chance, plant=None):
    p = Pair(n_tiles, rng, chance, plant)
    runs, send, at = [p.run(0), p.run(1)], [None, None], [None, None]     # at: the barrier a warp stands at
    done = [False, False]
    while not all(done):
        moves = [w for w in (0, 1) if not done[w] and at[w] is None]
        if not moves:
            assert not any(done) and at[0][0] == at[1][0], "deadlock: the warps are not at the same barrier"
            either = at[0][1] or at[1][1]
            at, send = [None, None], [either, either]
            continue
        w = rng.choice(moves)
        try:
            got, send[w] = runs[w].send(send[w]), None
        except StopIteration:
            done[w] = True
            continue
        if got is not None:
            at[w] = got
            p.barriers[w].append(got[0])
    assert p.barriers[0] == p.barriers[1]
    return p


@pytest.mark.parametrize("chance", [0.0, 0.05, 0.5, 1.0])
def test_random_schedules(chance):
    for seed in range(400):
        rng = random.Random(seed)
        n = rng.choice([0, 1, 2, 3, 9])
        p = schedule(n, rng, chance)
        if p.lost[0] != p.lost[1]:     # only behind the last barrier (a rescale of the last tile)
            assert p.barriers[0].count("any") == n
        if chance == 0.0:
            assert p.lost == [False, False] and p.barriers[0].count("any") == n


@pytest.mark.parametrize("plant", ["leave", "no second barrier"])
def test_planted_mistakes_are_caught(plant):
    caught = 0
    for seed in range(300):
        try:
            schedule(6, random.Random(seed), 0.2, plant)
        except AssertionError:
            caught += 1
    assert caught > 30


@pytest.mark.parametrize("hd,stage_bytes", [(64, 96 * 1024), (128, 192 * 1024), (256, 224 * 1024)])
def test_chunks_and_slabs_of_the_merge(hd, stage_bytes):
    n_chunks, rows = hd // 4, 128
    for n in range(1, 9):
        most = -(-n_chunks // n)
        used = set()
        for ch in range(n_chunks):
            owner = ((ch + 1) * n - 1) // n_chunks
            first, end = owner * n_chunks // n, (owner + 1) * n_chunks // n
            assert 0 <= owner < n and first <= ch < end and ch - first < most
            for z in range(n):             # the slab place of split z's copy of it in its owner
                used.add((owner, z * most + ch - first))
        assert len(used) == n * n_chunks   # no two alike
        assert (max(i for _, i in used) + 1) * rows * 16 + 8 * rows * 8 <= stage_bytes
