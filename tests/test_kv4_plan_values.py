"""The cut of the attention kernels' work with the very values that the library
cuts with (test_kv4_plan.py has the replay and other values): a part may lie
inside an item's start and have no unit of its own."""
import os
import random
import re

import pytest

from test_kv4_plan import cut, span, units

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_verify_gb300", "csrc")


def values():
    """(extra with tiles, without; least) of attn_plan."""
    with open(os.path.join(CSRC, "attn_ops.cu")) as f:
        text = f.read()
    extra = re.search(r"a\.extra = a\.tiles \? (\d+) : (\d+);", text)
    least = re.search(r"a\.least = (\d+);", text)
    return int(extra[1]), int(extra[2]), int(least[1])


def lines(seed):
    """(units of the items, extra, least, parts) of a call with drawn sequences."""
    rng = random.Random(seed)
    tc, few, least = values()
    tile, unit, extra = rng.choice([(8, 32, few), (16, 32, few), (128, 64, tc), (256, 64, tc)])
    G, window, sinks = rng.choice([1, 3, 4, 6, 20]), rng.choice([0, 0, 1, 31, 32, 100, 1000]), rng.choice([0, 4, 33, 200])
    seqs = [(rng.choice([0, 1, 2, 5, 40, 300]), rng.choice([-1, 0, 1, 31, 32, 63, 500, 3000, 1 << 30])) for _ in range(rng.randint(1, 12))]
    max_pages = rng.choice([1, 3, 200])
    items = [units(span(s, t, G, tile, unit, window, sinks, max_pages)) for s in seqs for t in range(-(-s[0] * G // tile))]
    return items * rng.choice([1, 2, 5]), extra, least, rng.choice([1, 2, 7, 152, 608, 760])


@pytest.mark.parametrize("seed", range(300))
def test_every_unit_once(seed):
    items, extra, least, parts = lines(seed)
    pieces, joins = cut(items, extra, least, parts)
    at = {}                                     # (item, unit): part
    for k, mine in enumerate(pieces):
        assert [i for i, _, _ in mine] == sorted({i for i, _, _ in mine})
        for i, first, n in mine:
            for u in range(first, first + n):
                assert at.setdefault((i, u), k) == k
    assert sorted(at) == [(i, u) for i, n in enumerate(items) for u in range(n)]
    for i, n in enumerate(items):
        over = sorted({at[i, u] for u in range(n)})
        # an item of several parts: those from the one with its first unit on, and the joining kernel is told their number
        assert over == list(range(over[0], over[0] + len(over)))
        assert [j for j in joins.items() if j[1][0] == i] == ([(over[0], (i, len(over)))] if len(over) > 1 else [])
    for mine in pieces:                         # one slot for an item that goes on from here, one for one that came from before
        partial = [first for i, first, n in mine if n < items[i]]
        assert sum(f == 0 for f in partial) <= 1 and sum(f > 0 for f in partial) <= 1


def test_parts_without_units():
    """Among the drawn lines are parts with work on the line but no unit: inside an item's start."""
    found = 0
    for seed in range(300):
        items, extra, least, parts = lines(seed)
        line = sum(extra + n for n in items)
        share = max(least, -(-line // parts))
        found += sum(share * k < line and not mine for k, mine in enumerate(cut(items, extra, least, parts)[0]))
    assert found > 100
