"""How the norms at a block's ends lay their rows out, csrc/block_plan.h itself
on the host: what the shared memory holds, the groups' sums in front of the
ring's barriers, and every ring that it gives as a model (one or two rows a
group, last turns that are not whole, the producers' last waits behind the
groups' sums)."""
import os
import random
import shutil
import subprocess

import pytest

from tests.test_block_ring_cpu import Barrier, Wrong

SOURCE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c_api", "block_plan_test.cpp")


@pytest.fixture(scope="module")
def rings(tmp_path_factory):
    from accelerator_row_major_gb300 import build as build_mod
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no C++ compiler")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build_mod.nvcc()))), "include")
    exe = str(tmp_path_factory.mktemp("plan") / "block_plan_test")
    subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror", "-isystem", cuda, SOURCE, "-o", exe], check=True)
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stdout[-2000:] + run.stderr
    return [tuple(int(v) for v in line.split()[1:]) for line in run.stdout.splitlines() if line.startswith("ring ")]


def run(groups, each, chunk, stages, producers, total, seed):
    """A CTA's `total` rows through the ring: copies land in any order, everyone goes at a pace of their own."""
    rng = random.Random(seed)
    turn = groups * each
    step, readers = turn // chunk, chunk // each
    full, empty = [Barrier(1) for _ in range(stages)], [Barrier(readers) for _ in range(stages)]
    holds, flying = [None] * stages, []                        # stage: [chunk, groups still to read it, landed]
    first_row = lambda q: q // step * turn + q % step * chunk  # noqa: E731
    make, drain = list(range(producers)), [None] * producers   # next chunk; of the last waits, then -1
    read = [[g, g * each // chunk, 0, g * each] for g in range(groups)]       # group, stage, phase, next row
    sums = False
    pace = [rng.random() + 0.02 for _ in range(producers + groups + 1)]
    for _ in range(200000):
        if not sums and all(r[3] >= total for r in read):
            assert not flying, "a copy may land over the groups' sums"
            sums = True                                        # they lie over the ring from here on, not over its barriers
        if sums and all(d == -1 for d in drain):
            return
        who = rng.choices(range(producers + groups + 1), pace)[0]
        if who == producers + groups:
            if flying:
                s, h = flying.pop(rng.randrange(len(flying)))
                if holds[s] is not h:
                    raise Wrong("filled over a copy in flight")
                h[2] = True
                full[s].tx -= 1
                full[s].turn()
        elif who < producers:
            q = make[who]
            if drain[who] is not None:
                q = drain[who]
                if q >= 0 and full[q % stages].passed(q // stages & 1):
                    drain[who] = q - producers if q - producers >= max(0, make[who] - stages) else -1
                continue
            if first_row(q) >= total:
                drain[who] = q - producers if q - producers >= max(0, q - stages) else -1
                continue
            s, ph = q % stages, q // stages & 1
            if not empty[s].passed(ph ^ 1):
                continue
            if holds[s] is not None and holds[s][1] > 0:
                raise Wrong("filled over rows still to be read")
            rows = min(chunk, total - first_row(q))
            holds[s] = [q, -(-rows // each), False]
            full[s].tx += 1
            full[s].arrive()
            flying.append((s, holds[s]))
            make[who] += producers
        else:
            r = read[who - producers]
            g, s, ph, row = r
            if row >= total or not full[s].passed(ph):
                continue
            q = row // turn * step + g * each // chunk
            if holds[s] is None or holds[s][0] != q or not holds[s][2]:
                raise Wrong("read another chunk")
            holds[s][1] -= 1
            empty[s].arrive()
            r[1] += step
            if r[1] >= stages:
                r[1], r[2] = r[1] - stages, ph ^ 1
            r[3] += turn
    raise AssertionError("no end")


def test_every_ring_of_the_plan(rings):
    assert len(rings) > 100 and {r[1] for r in rings} == {1, 2} and {r[0] for r in rings} >= {1, 2, 3, 4, 6, 8, 9, 12, 16}
    for i, (groups, each, chunk, stages, producers) in enumerate(rings):
        turn = groups * each
        whole = stages * chunk * 2 // turn + 3                 # turns: the ring goes round twice and more
        for seed, total in enumerate((1, turn, whole * turn, whole * turn + 1, whole * turn + turn // 2, (whole + 1) * turn - 1)):
            run(groups, each, chunk, stages, producers, total, 1000 * i + seed)


def test_the_model_notices_a_stage_that_changes_hands():
    with pytest.raises((Wrong, AssertionError)):
        for seed in range(200):
            run(8, 2, 4, 13, 4, 640, seed)
