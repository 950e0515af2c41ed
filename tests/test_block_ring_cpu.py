"""The ring of rows of the norms at a block's ends (csrc/block_rows.cuh) as a
model: barriers whose waits look at a phase's parity, copies that land in any
order, producers and groups that run at any pace.  Every group reads the chunk
that it waits for and no chunk is filled over one that is still to be read, for
every ring that the launch may choose; a ring whose stages change hands shows
that the model would notice."""
import math
import random

import pytest

from tests.test_block_rows_cpu import ring_of


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase, self.tx = count, count, 0, 0

    def arrive(self):
        self.left -= 1
        assert self.left >= 0, "more arrivals than a phase has"
        self.turn()

    def turn(self):
        if self.left == 0 and self.tx == 0:
            self.phase, self.left = self.phase + 1, self.count

    def passed(self, parity):
        """Whether a wait for the phase of this parity returns."""
        return (self.phase & 1) != parity


class Wrong(AssertionError):
    pass


def run(groups, chunk, stages, producers, turns, seed):
    rng = random.Random(seed)
    step = groups // chunk
    full, empty = [Barrier(1) for _ in range(stages)], [Barrier(chunk) for _ in range(stages)]
    holds, landed, flying = [None] * stages, [False] * stages, []
    total = turns * step
    make = [p for p in range(producers)]                       # next chunk of each producer
    read = [[g, g // chunk, 0, 0] for g in range(groups)]       # group, stage, phase, turns done
    pace = [rng.random() + 0.02 for _ in range(producers + groups + 1)]
    for _ in range(200000):
        if all(r[3] == turns for r in read):
            return
        who = rng.choices(range(producers + groups + 1), pace)[0]
        if who == producers + groups:
            if flying:
                s, q = flying.pop(rng.randrange(len(flying)))
                if holds[s] != q:
                    raise Wrong("filled over a copy in flight")
                landed[s] = True
                full[s].tx -= 1
                full[s].turn()
        elif who < producers:
            q = make[who]
            if q >= total:
                continue
            s, ph = q % stages, q // stages & 1
            if not empty[s].passed(ph ^ 1):
                continue
            if holds[s] is not None and holds[s][1] > 0:
                raise Wrong("filled over rows still to be read")
            holds[s], landed[s] = [q, chunk], False
            full[s].tx += 1
            full[s].arrive()
            flying.append((s, holds[s]))
            make[who] += producers
        else:
            r = read[who - producers]
            g, s, ph, done = r
            if done == turns or not full[s].passed(ph):
                continue
            if holds[s] is None or holds[s][0] != done * step + g // chunk or not landed[s]:
                raise Wrong("read another chunk")
            holds[s][1] -= 1
            empty[s].arrive()
            r[1] += step
            if r[1] >= stages:
                r[1], r[2] = r[1] - stages, ph ^ 1
            r[3] += 1
    raise AssertionError("no end")


@pytest.mark.parametrize("groups", [1, 2, 3, 4, 5, 8, 16])
def test_rings_that_a_launch_chooses(groups):
    for chunk in (c for c in range(1, 9) if groups % c == 0):
        for room in (2, 3, 5, 7, 10, 13, 16, 22, 37):
            ring = ring_of(groups, chunk, room)
            if ring is None:
                continue
            stages, producers = ring
            assert stages <= room and stages % producers == 0 and stages % (groups // chunk) == 0 and stages >= 2 * (groups // chunk)
            for seed in range(3):
                run(groups, chunk, stages, producers, 12, seed)


def test_the_model_notices_a_stage_that_changes_hands():
    assert math.gcd(13, 4) == 1
    with pytest.raises((Wrong, AssertionError)):
        for seed in range(200):
            run(16, 4, 13, 4, 40, seed)
