"""How the norms at a block's ends lay a row out (csrc/block_rows.cuh, plan_rows
of csrc/block_norm.cu), restated on the host: every column has one thread's
element and one slot, the shared memory holds the ring, and a row's copies
stay within its matrix and its place in the ring."""
import pytest

THREADS, MOST_SHARED, MOST_STAGES, UNIT = 512, 224 * 1024, 8, 512
WIDTHS = [1, 2, 7, 31, 32, 33, 64, 255, 256, 257, 777, 1000, 1024, 1280, 2048, 2056, 4095, 4096, 4097, 5000, 8192, 8193, 12288,
          16384, 16385, 20001, 32768]


def source_bytes(size, cols):
    return size * cols if size else (cols + 31) // 32


def plan(width, rows, sizes, vectors, ne, aligned, sms=152):
    """(ctas, slice, lanes, groups, stages, stage bytes, offsets, bytes, grid), or None."""
    ctas = 1
    while ctas <= 8:
        cut = width if ctas == 1 else ((width - 1) // ctas // UNIT + 1) * UNIT
        if cut <= THREADS * ne:
            lanes = 32 * ((cut - 1) // (32 * ne) + 1)
            units = sms // ctas
            groups = min(1 if ctas > 1 else THREADS // lanes, (rows - 1) // units + 1)
            columns = vectors * ne * lanes * 4
            stage, at = 0, []
            for size in sizes:
                at.append(stage)
                stage += (source_bytes(size, cut) + 15) // 16 * 16 + (0 if aligned or size < 2 else 16)
            while True:
                stages = (MOST_SHARED - columns) // (groups * (stage + 8))
                if stages >= 2 or groups == 1:
                    break
                groups -= 1
            if columns < MOST_SHARED and stages >= 2:
                stages = min(stages, MOST_STAGES)
                total = max(columns + groups * stages * (stage + 8), groups * ne * lanes * 4)
                return ctas, cut, lanes, groups, stages, stage, at, total, min(units, (rows - 1) // groups + 1) * ctas
        ctas *= 2
    return None


def column(t, i, lanes, v):
    return (i // v * lanes + t) * v + i % v if v else i * lanes + t


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("es", [2, 4])
def test_columns_and_slots(width, es):
    for ne in (8, 16):
        for v in (0, 16 // es):                                   # single elements, vectors
            if v and width * es % 16:
                continue
            p = plan(width, 1000, [es] * 4, 3, ne, bool(v))
            if p is None:
                continue
            ctas, cut, lanes = p[:3]
            seen = set()
            for rank in range(ctas):
                n = max(0, min(cut, width - rank * cut))
                assert not v or n % v == 0
                cols = [[column(t, i, lanes, v) for i in range(ne)] for t in range(lanes)]
                flat = sorted(c for of in cols for c in of)
                assert flat == list(range(ne * lanes)) and n <= ne * lanes
                seen |= {rank * cut + c for c in flat if c < n}
                slots = set()
                for t in range(lanes):
                    for i in range(ne):
                        slot = 4 * (i // 4 * lanes + t) + i % 4    # quad(q) + j
                        quad = slot // 4                           # column_of_slot
                        assert column(quad % lanes, quad // lanes * 4 + slot % 4, lanes, v) == cols[t][i]
                        slots.add(slot)
                assert slots == set(range(ne * lanes))
            assert seen == set(range(width))


# forward: branch, residual, gate; gradient: dy, dh, h, branch and a gate, as a vector or a matrix, or h and branch in 8 bits
CASES = [([2, 2], 1, 8), ([4, 4, 4], 5, 8), ([2, 2, 2], 5, 16), ([4, 4], 2, 16), ([4, 4, 4, 4], 4, 8), ([4, 4, 4, 4, 4], 3, 8), ([2, 2, 2, 2, 2], 3, 8),
         ([2, 2, 1, 0, 1, 0, 2], 3, 8), ([4, 4, 1, 0, 1, 0, 4], 3, 8)]


@pytest.mark.parametrize("sizes,vectors,ne", CASES)
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("rows", [1, 3, 200, 100000])
def test_shared_memory_and_launch(width, rows, sizes, vectors, ne):
    for aligned in (True, False):
        p = plan(width, rows, sizes, vectors, ne, aligned)
        if p is None:
            assert ne == 16 or width > 32768                       # every row of up to 32768 columns has a plan of 8
            continue
        ctas, cut, lanes, groups, stages, stage, at, total, grid = p
        assert lanes * groups <= THREADS and lanes % 32 == 0 and 2 <= stages <= MOST_STAGES
        assert total <= MOST_SHARED and total + 1024 <= 227 * 1024
        assert (vectors * ne * lanes * 4) % 16 == 0 and stage % 16 == 0 and all(a % 16 == 0 for a in at)
        assert 1 <= grid <= 152 and grid % ctas == 0 and (ctas == 1 or groups == 1)
        assert groups == 1 or lanes == 32 or groups <= 15          # named barriers 1 ..
        assert cut % UNIT == 0 or ctas == 1


@pytest.mark.parametrize("width", [1, 3, 7, 8, 9, 31, 100, 777, 1001, 5001])
@pytest.mark.parametrize("es", [2, 4])
@pytest.mark.parametrize("base", [0, 4, 12])
def test_copies_stay_within_the_matrix_and_the_stage(width, es, base):
    for ld in (width, width + 1, width + 8):
        for rows in (1, 2, 5):
            start = 4096 + base
            end = start + ((rows - 1) * ld + width) * es
            p = plan(width, rows, [es], 1, 8, False)
            if p is None:
                continue
            ctas, cut, stage = p[0], p[1], p[5]
            for row in range(rows):
                for rank in range(ctas):
                    n = max(0, min(cut, width - rank * cut))
                    first = start + row * ld * es + rank * cut * es
                    last = first + n * es
                    lo, hi = first // 16 * 16, (last + 15) // 16 * 16
                    if lo < start:
                        lo += 16
                    if hi > end:
                        hi -= 16
                    if lo >= hi:
                        lo = hi = first
                    assert lo == hi or (start <= lo and hi <= end and lo % 16 == 0 and hi % 16 == 0)
                    at = lo - first // 16 * 16                       # of the copy in the stage
                    assert lo == hi or (at >= 0 and at + hi - lo <= stage)
                    got = set(range(lo, hi))
                    if lo == hi:
                        got |= set(range(first, last))
                    else:
                        got |= set(range(first, lo)) | set(range(hi, last))
                    assert set(range(first, last)) <= got
                    assert first % 16 + n * es <= stage
                    assert min(got, default=start) >= start and max(got, default=start) < max(end, start + 1)
