"""Host check of how the combine finds the row that a work range begins and another one continues: the
balanced plan (ranges of equal cost over the rows' cost line), and the search of the plan table as the
kernel does it, against the plan's ranges counted out."""
import random

import bench

SEG = bench.SEG_COST


def plan(tiles, P):
    """(cost offsets, total cost, {range: the row it begins and leaves to later ranges})."""
    off, tot = [0], [0]
    for t in tiles:
        off.append(off[-1] + (SEG + t if t else 0))
        tot.append(tot[-1] + t)
    C = off[-1]

    def bound(p):
        x = p * C // P
        for b, t in enumerate(tiles):
            if p < P and t and off[b] <= x < off[b + 1]:
                return tot[b] + max(0, x - off[b] - SEG)
        return tot[-1]

    bounds = [bound(p) for p in range(P + 1)]
    split = {}
    for b, t in enumerate(tiles):
        holds = [p for p in range(P) if bounds[p] < bounds[p + 1] and bounds[p] < tot[b + 1] and bounds[p + 1] > tot[b]]
        if t and len(holds) > 1:
            split[holds[0]] = b
    return off, C, split


def search(off, B, key):
    """The last row whose offset is at most key, 32 probes a round."""
    lo, n = 0, B
    while n > 1:
        step = (n + 31) // 32
        last = sum(lane * step < n and off[lo + lane * step] <= key for lane in range(32)) - 1
        lo, n = lo + last * step, min(step, n - last * step)
    return lo


def test_every_split_row_is_found_by_the_range_that_begins_it():
    rng = random.Random(1)
    for _ in range(600):
        B, P = rng.randint(1, 120), rng.randint(1, 90)
        tiles = [0 if rng.random() < 0.3 else rng.randint(1, rng.choice([2, 9, 60])) for _ in range(B)]
        off, C, split = plan(tiles, P)
        found = {}
        for p in range(P):
            key = (p + 1) * C // P - 1
            if key < 0:
                continue
            b = search(off, B, key)
            span = off[b + 1] - off[b]
            if span == 0:
                continue
            first, last = (-(-(y + 1) * P // C) - 1 for y in (off[b] + SEG, off[b] + span - 1))
            if first == p and last != first:
                found[p] = b
        assert found == split


def test_search_in_tables_of_any_length():
    rng = random.Random(2)
    for B in (1, 2, 31, 32, 33, 1000, 1024, 1025, 16384):
        off = [0]
        for _ in range(B):
            off.append(off[-1] + rng.choice([0, 0, 3, 5]))
        for key in [0, 1, off[B] - 1, off[B]] + [rng.randint(0, off[B]) for _ in range(20)]:
            if key >= 0:
                assert search(off, B, key) == max(i for i in range(B) if off[i] <= key)
