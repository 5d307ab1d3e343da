"""The barrier protocol of the tcgen05 attention kernel, replayed on the CPU.

Each role of `kv4_attn_tc_kernel` (the copying lanes, the two conversion groups' warps,
products, the tiles' softmax warps) is written here as the sequence of mbarrier
waits and arrivals it performs, with the same counts and phase arithmetic as
the kernel; the tensor core's completions come later, in order.  A random
scheduler runs the roles.  A wait is checked the way the hardware answers it
(the parity of the barrier's current phase): the run fails if a wait could be
answered before its phase completed or after the barrier moved two phases past
it, or if no role can move.  What the barriers protect is checked too: the
codes in an entry when they are read, the block in a ring slot when a product
reads it, the scores, probabilities and outputs in tensor memory, and the marks
of missing pages."""
import os
import random
import re

import pytest

from test_tc_protocol import Bar

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_verify_gb300", "csrc",
                   "kv4_attn_tc.cuh")


def step(s, n):
    """The block of step s: (unit, whether it is of values)."""
    if s == 2 * n - 1:
        return n - 1, True
    return ((s + 1) >> 1, False) if s & 1 else ((s >> 1) - 1, True) if s else (0, False)


def run(NT, BLOCKS, PIECES, TURN, MARKS, items, rng, warps=2):
    """items: (units, active tiles).  warps: of a conversion group, and of a tile's softmax."""
    ENTRIES = 2 * TURN
    raw_full = [Bar("raw_full%d" % i, 2 // PIECES) for i in range(ENTRIES)]
    raw_empty = [Bar("raw_empty%d" % i, warps) for i in range(ENTRIES)]
    b_full = [Bar("b_full%d" % i, warps) for i in range(BLOCKS)]
    b_empty = [Bar("b_empty%d" % i, 1) for i in range(BLOCKS)]
    s_full, o_done = ([[Bar("%s%d.%d" % (x, t, i), 1) for i in range(2)] for t in range(NT)] for x in "so")
    p_full = [[Bar("p_full%d.%d" % (t, i), warps) for i in range(2)] for t in range(NT)]
    q_full = [Bar("q_full%d" % t, warps) for t in range(NT)]
    tensor = []                                  # operations of the product warp, completing in order
    entry_holds, slot_holds = [[None] * (2 // PIECES) for _ in range(ENTRIES)], [[None] * warps for _ in range(BLOCKS)]
    S = [[None, None] for _ in range(NT)]        # ("s" | "p", item, unit, parts written)
    O = [None] * NT                              # (item, units added)
    Q = [[None] * warps for _ in range(NT)]
    marks = [[None, None] for _ in range(MARKS)] # the unit that a mark is of
    names, unit0 = [], []                        # every block in order: (item, unit, v); units before an item
    for k, (n, _) in enumerate(items):
        unit0.append(sum(m for m, _ in items[:k]))
        names += [(k, *step(s, n)) for s in range(2 * n)]

    def entries(e):
        """(slot, round) of the entries of block e."""
        for x in range(PIECES):
            i = e // 2 * PIECES + x
            yield e % 2 * TURN + i % TURN, i // TURN

    def copies(ring, sub):
        """A lane: its page of every block of a ring."""
        for e in range(ring, len(names), 2):
            if not names[e][2]:
                marks[(unit0[names[e][0]] + names[e][1]) % MARKS][sub] = names[e][:2]
            at, rnd = list(entries(e))[sub if PIECES == 2 else 0]
            if rnd:
                yield raw_empty[at], rnd - 1
            entry_holds[at][0 if PIECES == 2 else sub] = names[e]
            yield None
            raw_full[at].arrive()

    def convert(group, w):
        for e in range(group, len(names), 2):
            for at, rnd in entries(e):
                yield raw_full[at], rnd
                assert all(x == names[e] for x in entry_holds[at])
                yield None
                assert all(x == names[e] for x in entry_holds[at])
            for at, rnd in entries(e):
                raw_empty[at].arrive()
            at, rnd = e % BLOCKS, e // BLOCKS
            if rnd:
                yield b_empty[at], rnd - 1
            slot_holds[at][w] = names[e]
            yield None
            b_full[at].arrive()

    def products():
        block, items_of, units_of = 0, [0] * NT, [0] * NT

        def holds(b, name):
            assert all(x == name for x in slot_holds[b % BLOCKS]), (slot_holds[b % BLOCKS], name)

        def scores(t, buf, k, i, b):
            def done():
                holds(b, (k, i, False))
                assert all(q == k for q in Q[t])
                S[t][buf] = ("s", k, i, set())
            tensor.extend([("op", done), ("commit", s_full[t][buf])])

        def values(t, buf, k, i, b):
            def done():
                holds(b, (k, i, True))
                assert S[t][buf][:3] == ("p", k, i) and len(S[t][buf][3]) == warps, S[t][buf]
                if i:
                    assert O[t] == (k, i)
                O[t] = (k, i + 1)
            tensor.extend([("op", done), ("commit", o_done[t][buf])])

        for k, (n, tiles) in enumerate(items):
            for t in range(tiles):
                yield q_full[t], items_of[t]
                items_of[t] += 1
            for i in range(-1, n):
                if i + 1 < n:
                    yield b_full[block % BLOCKS], block // BLOCKS
                    for t in range(tiles):
                        scores(t, (units_of[t] + (i >= 0)) & 1, k, i + 1, block)
                    tensor.append(("commit", b_empty[block % BLOCKS]))
                    block += 1
                if i < 0:
                    continue
                yield b_full[block % BLOCKS], block // BLOCKS
                for t in range(tiles):
                    yield p_full[t][units_of[t] & 1], units_of[t] >> 1
                    values(t, units_of[t] & 1, k, i, block)
                    units_of[t] += 1
                tensor.append(("commit", b_empty[block % BLOCKS]))
                block += 1

    arrived = {}

    def meet(key, who):                          # a named barrier of a tile
        arrived.setdefault(key, set()).add(who)
        while len(arrived[key]) < warps:
            yield None

    def softmax(t, me):
        u = 0
        for k, (n, tiles) in enumerate(items):
            if t >= tiles:
                continue
            yield from meet(("before", k, t), me)
            Q[t][me] = k
            yield None
            q_full[t].arrive()
            yield from meet(("q", k, t), me)
            for i in range(n):
                buf = u & 1
                yield s_full[t][buf], u >> 1
                assert S[t][buf][1:3] == (k, i) and (S[t][buf][0] == "s" or me not in S[t][buf][3]), (S[t][buf], k, i)
                assert marks[(unit0[k] + i) % MARKS] == [(k, i)] * 2, (marks, k, i)
                yield None
                if NT == 1:
                    yield from meet(("max", k, i), me)
                if i and rng.random() < 0.5:     # the maximum moved: O is rescaled
                    yield o_done[t][(u - 1) & 1], (u - 1) >> 1
                    assert O[t] == (k, i), (O[t], k, i)
                    yield None
                    assert O[t] == (k, i)
                yield None
                S[t][buf] = ("p", k, i, S[t][buf][3] | {me})
                p_full[t][buf].arrive()
                u += 1
            if NT == 1:
                yield from meet(("sum", k), me)
            yield o_done[t][(u - 1) & 1], (u - 1) >> 1
            assert O[t] == (k, n)
            yield None
            assert O[t] == (k, n)

    gens = {"products": products()}
    gens.update({"copies%d.%d" % (r, i): copies(r, i) for r in range(2) for i in range(2)})
    gens.update({"convert%d.%d" % (g, w): convert(g, w) for g in range(2) for w in range(warps)})
    gens.update({"softmax%d.%d" % (t, w): softmax(t, w) for t in range(NT) for w in range(warps)})
    want = dict.fromkeys(gens)
    speed = {g: rng.random() ** 2 + 0.02 for g in gens}
    drain, idle = rng.random() ** 2 + 0.02, 0
    while gens or tensor:
        moved = False
        if tensor and rng.random() < drain:
            kind, x = tensor.pop(0)
            x() if kind == "op" else x.arrive()
            moved = True
        for g in rng.sample(list(gens), len(gens)):
            if rng.random() > speed[g]:
                continue
            w = want[g]
            if w and not w[0].done(w[1]):
                continue
            try:
                want[g] = next(gens[g])
                moved = True
            except StopIteration:
                del gens[g]
                moved = True
        idle = 0 if moved else idle + 1
        assert idle < 3000, ("nothing moves", {g: (w[0].name, w[1], w[0].ph) if w else None for g, w in want.items() if g in gens})
    return True


def items(rng, NT):
    return [(rng.choice([1, 1, 2, 3, 4, 7, 11, 25]), rng.randint(1, NT)) for _ in range(rng.randint(1, 8))]


def constants():
    """(blocks, entries of a block, entries of a group, marks) of d 256, and of the others, as the kernel has them."""
    s = open(SRC).read()
    b = re.search(r"BLOCKS = D == 256 \? (\d+) : (\d+);", s)
    e = re.search(r"PIECES = D == 256 \? (\d+) : (\d+);", s)
    t, m = re.search(r"TURN = (\d+),", s), re.search(r"BARS = MASK \+ (\d+) \* 2;", s)
    return tuple((int(b[i]), int(e[i]), int(t[1]), int(m[1])) for i in (1, 2))


@pytest.mark.parametrize("NT,wide", [(1, True), (1, False), (2, False)])
@pytest.mark.parametrize("seed", range(60))
def test_protocol(NT, wide, seed):
    rng = random.Random(seed)
    assert run(NT, *constants()[0 if wide else 1], items(rng, NT), rng)
