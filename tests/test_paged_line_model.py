"""CPU model of how paged attention's work is cut (attn_paged_kernel.cuh: the
line of key tiles, its shares, the join of cut units), with the kernel's
arithmetic in plain integers.  For random batches and share counts: every tile
of every unit is taken by exactly one share, units whose end a share holds are
written by it or left as parts that one join gathers, every row of a cut unit
is joined by exactly one block, and the shares' costs differ by at most one."""

import numpy as np
import pytest

UNIT_COST = 2  # kUnitCost


def cut(total, shares):
    each, rest = divmod(total, shares)

    def start(c):
        return c * each + min(c, rest)

    def holder(x):
        big = rest * (each + 1)
        return x // (each + 1) if x < big else rest + (x - big) // each

    return start, holder


def walk(seqs, shares):
    """The pieces (share, seq, unit, first tile, end tile, tiles) that the
    producers hand over, and the join marks {share: (seq, unit, first, parts)}.
    seqs: (units, tiles) of every sequence."""
    total = sum(u * (t + UNIT_COST) for u, t in seqs)
    start, holder = cut(total, shares)
    pieces, marks = [], {}
    for c in range(shares):
        begin, end = start(c), start(c + 1)
        if begin >= end:
            continue
        at, s = 0, 0
        while not begin < at + seqs[s][0] * (seqs[s][1] + UNIT_COST):
            at += seqs[s][0] * (seqs[s][1] + UNIT_COST)
            s += 1
        units, tiles = seqs[s]
        unit = (begin - at) // (tiles + UNIT_COST)
        u0 = at + unit * (tiles + UNIT_COST)
        tile = max(0, begin - u0 - UNIT_COST)
        if tile > 0:
            first = holder(u0 + UNIT_COST)
            marks[c] = (s, unit, first, holder(u0 + UNIT_COST + tiles - 1) - first + 1)
        while True:
            stop = max(0, min(tiles, end - u0 - UNIT_COST))
            if tile < stop:
                pieces.append((c, s, unit, tile, stop, tiles))
            u0 += tiles + UNIT_COST
            if u0 >= end:
                break
            tile = 0
            unit += 1
            if unit == units:
                unit, s = 0, s + 1
                while seqs[s][0] == 0:
                    s += 1
                units, tiles = seqs[s]
    return pieces, marks


@pytest.mark.parametrize("seed", range(60))
def test_every_tile_once_and_every_cut_unit_joined_once(seed):
    rng = np.random.default_rng(seed)
    S = int(rng.integers(1, 12))
    seqs = [(int(rng.choice([0, 1, 2, 5])), int(rng.choice([1, 1, 2, 7, 40]))) for _ in range(S)]
    if sum(u for u, _ in seqs) == 0:
        seqs.append((1, 1))
    shares = int(rng.choice([1, 2, 3, 7, 16, 64, 304, 1000]))
    pieces, marks = walk(seqs, shares)

    seen = {}
    for c, s, unit, a, b, tiles in pieces:
        for t in range(a, b):
            assert (s, unit, t) not in seen
            seen[(s, unit, t)] = c
    assert len(seen) == sum(u * t for u, t in seqs)

    by_unit = {}
    for c, s, unit, a, b, tiles in pieces:
        by_unit.setdefault((s, unit), []).append((c, a, b, tiles))
    joined = {}
    for c, (s, unit, first, parts) in marks.items():
        joined.setdefault((s, unit), []).append((c, first, parts))
    slots = set()
    for key, ps in by_unit.items():
        if len(ps) == 1:
            assert ps[0][1:3] == (0, ps[0][3]) and key not in joined  # whole: written by its share
            continue
        shares_of = sorted(c for c, *_ in ps)
        assert shares_of == list(range(shares_of[0], shares_of[-1] + 1))
        for c, a, b, tiles in ps:  # slot 1 for the part with tile 0, slot 0 for one that began earlier
            slot = (c, 1 if a == 0 else 0)
            assert slot not in slots
            slots.add(slot)
            assert (a == 0) == (c == shares_of[0])
        # every continuing share carries the same mark, and their blocks take every row once
        assert sorted(j[0] for j in joined[key]) == shares_of[1:]
        assert all(j[1:] == (shares_of[0], len(ps)) for j in joined[key])
        for rows in (1, 5, 16, 32):
            taken = sorted(r for c, first, parts in joined[key] for r in range(c - first - 1, rows, parts - 1))
            assert taken == list(range(rows))
    assert set(joined) <= set(by_unit) and all(len(by_unit[k]) > 1 for k in joined)


def test_shares_are_equally_long():
    start, _ = cut(1003, 7)
    lengths = [start(c + 1) - start(c) for c in range(7)]
    assert sum(lengths) == 1003 and max(lengths) - min(lengths) == 1


@pytest.mark.parametrize("total,shares", [(1, 5), (10, 3), (100, 100), (7, 2), (12345, 304)])
def test_the_holder_is_the_inverse_of_the_cut(total, shares):
    start, holder = cut(total, shares)
    for c in range(shares):
        for x in range(start(c), start(c + 1)):
            assert holder(x) == c
