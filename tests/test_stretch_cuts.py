"""The rule by which blocks cut the line of work units between them, restated: every
tile of every unit is taken by exactly one block, in order, parts are never empty
between a unit's first and last one, and the merge's last block is the one that
holds the unit's last tile."""
import random

import pytest


def tile(x, u0, n, lead, snap):
    o = x - u0 - lead
    return n if o >= n else 0 if o <= 0 or o < snap else n if o > n - snap else o


def cut(units, blocks, lead, snap):
    total = sum(n + lead for n in units)
    share = -(-total // blocks)
    parts = [[] for _ in units]
    for b in range(blocks):
        at, end = b * share, min(b * share + share, total)
        if at >= end:
            continue
        u0 = 0
        for i, n in enumerate(units):
            # a block looks from the unit that holds its first position on
            if u0 + n + lead > at and u0 < end:
                t0, t1 = tile(at, u0, n, lead, snap), tile(end, u0, n, lead, snap)
                if t0 < t1:
                    parts[i].append((b, t0, t1))
            u0 += n + lead
    u0 = 0
    for n, p in zip(units, parts):
        last = (u0 + lead + n - 1) // share
        if tile(last * share, u0, n, lead, snap) == n:
            last -= 1
        assert [x for _, a, b in p for x in range(a, b)] == list(range(n)), (n, p)
        assert [b for b, _, _ in p] == list(range(p[0][0], p[-1][0] + 1)), p
        assert p[-1][0] == last, (p, last)
        u0 += n + lead


@pytest.mark.parametrize("seed", range(3))
def test_every_tile_is_taken_once(seed):
    r = random.Random(seed)
    for _ in range(60):
        blocks = r.choice([1, 2, 7, 152])
        units = [r.choice([1, 1, 2, 3, r.randint(1, 60)]) for _ in range(r.randint(1, 200))]
        long_enough = sum(units) >= 12 * blocks
        cut(units, blocks, 2 if long_enough else 0, 2 if long_enough else 0)


def test_one_tile_units_whose_ends_meet_the_cuts():
    for n in range(1, 40):
        cut([1] * (24 * n), 2 * n, 2, 2)
        cut([1] * (27 * n), n, 2, 2)
