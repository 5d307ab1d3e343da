"""How the attention kernels cut their work, replayed on the CPU with the
arithmetic of kv4_plan.cuh: whatever the sequences, every unit of every item
belongs to one part, and the parts that an item goes over are those that the
joining kernel is told."""
import random

import pytest

PAGE = 32


def span(seq, tile, G, T, unit, window, sinks, max_pages):
    """(sink units, first, end) of a tile."""
    n, before = seq
    if before < 0:
        return 0, 0, 0
    t0, t1 = tile * T // G, (min((tile + 1) * T, n * G) - 1) // G
    lo = max(0, before + t0 - window + 1) if window else 0
    to = min(before + t1, max_pages * PAGE - 1) // unit + 1
    s = min((min(sinks, lo) + unit - 1) // unit, to)
    return s, min(max(s, lo // unit), to), to


def units(sp):
    return max(1, sp[0] + sp[2] - sp[1])


def cut(items, extra, least, parts):
    """The pieces of each part, (item, first unit, units), and the joins {part: (item, parts)}; items: units each."""
    line = sum(extra + u for u in items)
    share = max(least, -(-line // parts))
    pieces, joins = [], {}
    for k in range(parts):
        lo = min(share * k, line)
        left = min(share, line - lo)
        mine = []
        pieces.append(mine)
        if left <= 0:
            continue
        i = 0
        place = lo
        while place >= extra + items[i]:
            place -= extra + items[i]
            i += 1
        while left > 0:
            end = min(place + left, extra + items[i])
            unit = max(0, place - extra)
            n = max(0, end - extra) - unit
            if n <= 0:
                break
            mine.append((i, unit, n))
            over = 0 if unit else 1 + -(-(items[i] - n) // share)
            if over > 1:
                joins[k] = (i, over)
            left -= extra + unit + n - place
            place = 0
            i += 1
    return pieces, joins


@pytest.mark.parametrize("seed", range(150))
def test_every_unit_once(seed):
    rng = random.Random(seed)
    tile, unit, extra = rng.choice([(8, 32, 4), (16, 32, 4), (128, 64, 10), (256, 64, 10)])
    least = extra + rng.choice([4, 8])
    G, window, sinks = rng.choice([1, 3, 4, 6, 20]), rng.choice([0, 0, 1, 31, 32, 100, 1000]), rng.choice([0, 4, 33, 200])
    seqs = [(rng.choice([0, 1, 2, 5, 40, 300]), rng.choice([-1, 0, 1, 31, 32, 63, 500, 3000])) for _ in range(rng.randint(1, 12))]
    max_pages = rng.choice([1, 3, 200])
    items = [units(span(s, t, G, tile, unit, window, sinks, max_pages)) for s in seqs for t in range(-(-s[0] * G // tile))]
    items = items * rng.choice([1, 2, 5])       # heads
    pieces, joins = cut(items, extra, least, rng.choice([1, 2, 7, 152, 608]))
    seen = [[] for _ in items]
    for k, mine in enumerate(pieces):
        for i, first, n in mine:
            seen[i].append((first, n, k))
    for i, (u, s) in enumerate(zip(items, seen)):
        assert sorted(s) == s and sum(n for _, n, _ in s) == u
        assert all(a + n == b for (a, n, _), (b, _, _) in zip(s, s[1:])) and s[0][0] == 0
        over = [j for j in joins.items() if j[1][0] == i]
        if len(s) == 1:
            assert not over
        else:
            assert over == [(s[0][2], (i, len(s)))] and [k for _, _, k in s] == list(range(s[0][2], s[0][2] + len(s)))
    for mine in pieces:                         # slot 1 for an item that starts in a part, slot 0 for one that goes on: one of each at most
        partial = [(i, first) for i, first, n in mine if n < items[i]]
        assert sum(f == 0 for _, f in partial) <= 1 and sum(f > 0 for _, f in partial) <= 1


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (16, 4), (33, 32), (100, 40), (257, 1000), (64, 64)])
@pytest.mark.parametrize("unit", [32, 64])
def test_span_covers_what_is_seen(window, sinks, unit):
    for before in (0, 1, 30, 31, 32, 63, 64, 100, 333):
        for n, G, tile in ((1, 6, 8), (5, 4, 16), (40, 3, 128), (100, 4, 256)):
            for t in range(-(-n * G // tile)):
                a, first, end = span((n, before), t, G, tile, unit, window, sinks, 10 ** 6)
                have = set(range(a * unit)) | set(range(first * unit, end * unit))
                assert a <= first
                for r in range(t * tile, min((t + 1) * tile, n * G)):
                    p = before + r // G
                    assert {j for j in range(p + 1) if not window or p - j < window or j < sinks} <= have
