"""How the norms at a block's ends lay a row out (csrc/block_rows.cuh, plan_rows
of csrc/block_norm.cu), restated on the host: every column has one thread's
element and one slot, the shared memory holds the ring, and a row's copies
stay within its matrix and its place in the ring."""
import math

import pytest

WARPS, MOST_SHARED, MOST_STAGES, UNIT, LEAST_CHUNK = 16, 220 * 1024, 16, 512, 16 * 1024
MOST_CHUNK, MOST_LOOSE, STATS = 8, 4, 4
WIDTHS = [1, 2, 7, 31, 32, 33, 64, 255, 256, 257, 777, 1000, 1024, 1280, 2048, 2056, 4095, 4096, 4097, 5000, 8192, 8193, 12288,
          16384, 16385, 20001, 32768]


def source_bytes(size, cols):
    return size * cols if size else (cols + 31) // 32


def ring_of(groups, chunk, room):
    """(stages, producers) of a ring with room for so many stages, or None."""
    step = groups // chunk
    if room < 2 or (room < 2 * step and groups > 1):
        return None
    most = min(room, max(MOST_STAGES, 2 * step))
    for producers in (4, 2, 1):
        unit = math.lcm(step, producers)
        stages = most // unit * unit
        if stages >= 2 * step and (4 * stages >= 3 * most or producers == 1):
            break
    return stages, producers


def plan(width, rows, sizes, vectors, ctas, ne, stats, sums, aligned, packed=True, sms=152):
    """The layout as a dict, or None."""
    cut = width if ctas == 1 else ((width - 1) // ctas // UNIT + 1) * UNIT
    if ctas > sms or cut > WARPS * 32 * ne:
        return None
    lanes = 32 * ((cut - 1) // (32 * ne) + 1)
    units = sms // ctas
    columns = vectors * ne * lanes * 4
    packed = packed and ctas == 1

    def stage_of(n):
        stage, at, pitches = 0, [], []
        for size in sizes:
            row = source_bytes(size, cut)
            # codes and exponents are padded: packed where that adds nothing
            whole = packed and (size > 1 or (size == 1 and width % 32 == 0) or (size == 0 and row % 16 == 0))
            pitches.append((row if whole else (row + 15) // 16 * 16 + (0 if aligned or size < 2 else 16), whole))
            at.append(stage)
            stage += (n * pitches[-1][0] + 15) // 16 * 16 + (16 if whole and not aligned else 0)
        return stage + (n * STATS * 4 if stats else 0), at, pitches

    groups = min(WARPS * 32 // lanes, (rows - 1) // units + 1)
    while True:
        chunk, n = 1, 2
        while n <= groups and stage_of(chunk)[0] < LEAST_CHUNK:
            loose = any(not w for _, w in stage_of(chunk)[2])
            if groups % n == 0 and n <= (MOST_LOOSE if loose else MOST_CHUNK):
                chunk = n
            n += 1
        stage, at, pitches = stage_of(chunk)
        room = (MOST_SHARED - columns) // (stage + 16) if columns < MOST_SHARED else 0
        if room >= 2 * (groups // chunk) or groups == 1:
            break
        groups -= 1
    if room < 2:
        return None
    stages, producers = ring_of(groups, chunk, room)
    return dict(ctas=ctas, cut=cut, lanes=lanes, groups=groups, chunk=chunk, stages=stages, producers=producers, stage=stage, at=at,
                pitches=pitches, columns=columns, bytes=max(columns + stages * (stage + 16), sums * groups * ne * lanes * 4),
                grid=min(units, (rows - 1) // groups + 1) * ctas)


def column(t, i, ne, v):
    """Column of element i of thread t: a warp's are side by side."""
    return t // 32 * 32 * ne + (t % 32 * v + i // v * 32 * v + i % v if v else t % 32 + i * 32)


def column_of_slot(slot, ne, v):
    warp, of = divmod(slot, 32 * ne)
    return column(warp * 32 + of % 128 // 4, of // 128 * 4 + of % 4, ne, v)


@pytest.mark.parametrize("es", [2, 4])
@pytest.mark.parametrize("ne", [8, 16, 32])
def test_columns_and_slots(es, ne):
    for v in (0, 16 // es):                                           # single elements, vectors
        for lanes in (32, 64, 96, 512):
            slots = {}
            for t in range(lanes):
                for i in range(ne):
                    slot = t // 32 * 32 * ne + 128 * (i // 4) + 4 * (t % 32) + i % 4
                    assert column_of_slot(slot, ne, v) == column(t, i, ne, v)
                    slots[slot] = column(t, i, ne, v)
            assert sorted(slots) == list(range(ne * lanes)) == sorted(slots.values())


@pytest.mark.parametrize("width", WIDTHS)
def test_slices_cover_the_row(width):
    for ctas in (1, 2, 4, 8):
        p = plan(width, 1000, [4, 4], 1, ctas, 32, False, 0, False)
        if p:
            cuts = [max(0, min(p["cut"], width - r * p["cut"])) for r in range(ctas)]
            assert sum(cuts) == width and max(cuts) <= p["lanes"] * 32 and (ctas == 1 or p["cut"] % UNIT == 0)


# forward: branch, residual, gate; gradient: dy, dh, h, branch and a gate, as a vector or a matrix, or h and branch in 8 bits
CASES = [([2, 2], 1, False), ([4, 4, 4], 4, False), ([4, 4], 5, False), ([2, 2, 2], 4, False), ([4, 4, 4, 4], 4, True),
         ([4, 4, 4, 4, 4], 3, True), ([2, 2, 2, 2, 2], 3, True), ([2, 2, 1, 0, 1, 0, 2], 3, True), ([4, 4, 1, 0, 1, 0, 4], 3, True)]


@pytest.mark.parametrize("sizes,vectors,grad", CASES)
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("rows", [1, 3, 200, 100000])
def test_shared_memory_and_launch(width, rows, sizes, vectors, grad):
    for aligned in (True, False):
        for packed in (True, False):
            some = False
            for ctas in (1, 2, 4, 8):
                for ne in (8, 16) if grad else (8, 16, 32):
                    p = plan(width, rows, sizes, vectors, ctas, ne, grad, vectors if grad else 0, aligned, packed)
                    if p is None:
                        continue
                    some = some or ne == 8 or not grad
                    threads = p["lanes"] * p["groups"]
                    assert threads <= 512 and p["groups"] % p["chunk"] == 0 and p["chunk"] <= MOST_CHUNK
                    step = p["groups"] // p["chunk"]
                    assert p["stages"] % step == 0 and p["stages"] % p["producers"] == 0 and p["stages"] >= 2
                    assert p["bytes"] <= MOST_SHARED and p["bytes"] + 4096 <= 227 * 1024
                    assert p["columns"] % 16 == 0 and p["stage"] % 16 == 0 and all(a % 16 == 0 for a in p["at"])
                    assert 1 <= p["grid"] <= 152 and p["grid"] % ctas == 0
                    assert p["lanes"] == 32 or p["groups"] <= 8                    # named barriers 1 .. 8, and 15
                    # a lane for every copy and statistic; each within its part of the stage
                    lanes = len(sizes) * p["chunk"] if any(not w for _, w in p["pitches"]) else len(sizes)
                    assert lanes <= 32 and STATS * p["chunk"] <= 32
                    ends = p["at"][1:] + [p["stage"] - (p["chunk"] * 16 if grad else 0)]
                    for size, at, end, (pitch, whole) in zip(sizes, p["at"], ends, p["pitches"]):
                        row = source_bytes(size, p["cut"])
                        last = (p["chunk"] - 1) * pitch + row
                        spare = 0 if aligned or size < 2 else 15                   # above a boundary
                        assert at + (last + spare + 15) // 16 * 16 <= end
            assert some                                                            # up to 32768 columns have a layout


@pytest.mark.parametrize("width", [1, 3, 7, 8, 9, 31, 100, 777, 1001, 5001])
@pytest.mark.parametrize("es", [2, 4])
@pytest.mark.parametrize("base", [0, 4, 12])
def test_copies_stay_within_the_matrix_and_the_stage(width, es, base):
    for ld in (width, width + 1, width + 8):
        for rows in (1, 2, 5):
            start = 4096 + base
            end = start + ((rows - 1) * ld + width) * es
            for ctas in (1, 2):
                p = plan(width, 152 * rows, [es], 1, ctas, 8, False, 0, False, ld == width)
                if p is None:
                    continue
                (pitch, whole), = p["pitches"]
                n = min(rows, p["chunk"])
                for row in range(rows - n + 1) if whole else range(rows):
                    for rank in range(ctas):
                        cols = max(0, min(p["cut"], width - rank * p["cut"]))
                        first = start + row * ld * es + rank * p["cut"] * es
                        last = first + cols * es + ((n - 1) * pitch if whole else 0)
                        lo, hi = first // 16 * 16, (last + 15) // 16 * 16
                        if lo < start:
                            lo += 16
                        if hi > end:
                            hi -= 16
                        if lo >= hi:
                            lo = hi = first
                        assert lo == hi or (start <= lo and hi <= end and lo % 16 == 0 and hi % 16 == 0)
                        at = lo - first // 16 * 16                    # of the copy in its place
                        room = p["stage"] if whole else pitch
                        assert lo == hi or (at >= 0 and at + hi - lo <= room)
                        assert first % 16 + last - first <= room
                        got = set(range(lo, hi)) | {q for q in range(first, last) if not lo <= q < hi}
                        assert set(range(first, last)) <= got
                        assert min(got, default=start) >= start and max(got, default=start) < max(end, start + 1)
