"""The streaming norms' rings of rows after a wait that ran out: the stages and
phases that the issuing thread then waits for (RowRing::finish) are those of
the copies that it had issued and not waited for.  A model of the ring's
bookkeeping with the source's own expressions."""
import os
import random
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "accelerator_row_major_gb300", "csrc")


def _c_rem(a, b):
    """a % b as in C."""
    return a - b * int(a / b)


def test_the_source_still_reads_as_the_model():
    with open(os.path.join(CSRC, "layer_norm_stream.cuh")) as f:
        text = re.sub(r"\s+", " ", f.read())
    for line in ("const long long first = next - stages * step, since = (row - first) / step;",
                 "int at = static_cast<int>(((s - since) % stages + stages) % stages);",
                 "uint32_t parity = ph ^ (static_cast<uint32_t>((at + since) / stages) & 1u);",
                 "for (int k = 0; k < stages && first + k * step < a.rows; ++k) {"):
        assert line in text
    assert text.count("if (t == 0 && !ring.lost) ring.load(ring.s);") == 2 and text.count("if (t == 0) ring.finish(row);") == 2


def test_copies_in_flight_after_a_lost_wait():
    rng = random.Random(5)
    for _ in range(3000):
        stages, step = rng.randint(2, 8), rng.randint(1, 50)
        start = rng.randint(0, step - 1)
        rows, lose, later = start + rng.randint(1, 400), rng.randint(0, 60), rng.random() < 0.5
        issued, phase = [], [0] * stages
        nxt, s, ph, row, i, lost, waited = start, 0, 0, start, 0, False, None

        def load(at, nxt):
            if nxt < rows:
                issued.append((at, phase[at], nxt))
                phase[at] ^= 1
            return nxt + step

        for k in range(stages):
            nxt = load(k, nxt)
        while row < rows:
            if i == lose and not later:               # the wait for this row's copy
                lost, waited = True, row
            if not lost:
                nxt = load(s, nxt)
            s += 1
            if s == stages:
                s, ph = 0, ph ^ 1
            if i == lose and later:                   # the wait for the other CTAs, with the next copy issued
                lost, waited = True, row + step
            row, i = row + step, i + 1
        if not lost:
            continue
        first = nxt - stages * step
        since = (row - first) // step
        at = _c_rem(_c_rem(s - since, stages) + stages, stages)
        parity = ph ^ ((at + since) // stages & 1)
        drained = []
        for k in range(stages):
            if first + k * step >= rows:
                break
            drained.append((at, parity, first + k * step))
            at += 1
            if at == stages:
                at, parity = 0, parity ^ 1
        assert drained == [c for c in issued if c[2] >= waited]
