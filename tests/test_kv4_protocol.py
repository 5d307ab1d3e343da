"""The barrier protocol of the tcgen05 attention kernel, replayed on the CPU.

Each role of `kv4_attn_tc_kernel` (copies, the two conversion groups' warps,
products, the softmax warpgroups' warps) is written here as the sequence of
mbarrier waits and arrivals it performs, with the same counts and phase
arithmetic as the kernel; the tensor core's completions come later, in order.
A random scheduler runs the roles.  A wait is checked the way the hardware
answers it (the parity of the barrier's current phase): the run fails if a
wait could be answered before its phase completed or after the barrier moved
two phases past it, or if no role can move.  What the barriers protect is
checked too: the codes in an entry when they are read, the block in a ring slot
when a product reads it, the scores, probabilities and outputs in tensor memory."""
import os
import random
import re

import pytest

from test_tc_protocol import Aliasing, Bar

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_verify_gb300", "csrc",
                   "kv4_attn_tc.cuh")


def step(s, n, NT):
    if NT == 2:
        return s >> 1, bool(s & 1)
    if s == 2 * n - 1:
        return n - 1, True
    return ((s + 1) >> 1, False) if s & 1 else ((s >> 1) - 1, True) if s else (0, False)


def run(NT, BLOCKS, PIECES, TURN, items, rng, warps=2):
    """items: (units, active tiles).  warps: of a conversion group, and half of a tile's softmax warps."""
    ENTRIES = 2 * TURN
    soft = 2 * warps                             # of a tile
    raw_full = [Bar("raw_full%d" % i, 1) for i in range(ENTRIES)]
    raw_empty = [Bar("raw_empty%d" % i, warps) for i in range(ENTRIES)]
    b_full = [Bar("b_full%d" % i, warps) for i in range(BLOCKS)]
    b_empty = [Bar("b_empty%d" % i, 1) for i in range(BLOCKS)]
    s_full, p_full = [Bar("s_full%d" % i, 1) for i in range(2)], [Bar("p_full%d" % i, soft) for i in range(2)]
    o_done, q_full = [Bar("o_done%d" % i, 1) for i in range(2)], [Bar("q_full%d" % i, soft) for i in range(2)]
    tensor = []                                  # operations of the product warp, completing in order
    entry_holds, slot_holds = [None] * ENTRIES, [[None] * warps for _ in range(BLOCKS)]
    S = [None, None]                             # ("s" | "p", item, unit, parts written)
    O = [None, None]                             # (item, units added) of a tile
    Q = [[None] * soft for _ in range(2)]
    names = []                                   # every block in order: (item, unit, v, half)
    for k, (n, _) in enumerate(items):
        for s in range(2 * n):
            i, v = step(s, n, NT)
            names += [(k, i, v, 0), (k, i, v, 1)]

    def entries(e):
        """(slot, round) of the entries of block e."""
        for x in range(PIECES):
            i = e // 2 * PIECES + x
            yield e % 2 * TURN + i % TURN, i // TURN

    def copies():
        for e, name in enumerate(names):
            for at, rnd in entries(e):
                if rnd:
                    yield raw_empty[at], rnd - 1
                entry_holds[at] = name
                yield None
                raw_full[at].arrive()

    def convert(group, w):
        for e in range(group, len(names), 2):
            for at, rnd in entries(e):
                yield raw_full[at], rnd
                assert entry_holds[at] == names[e]
                yield None
                assert entry_holds[at] == names[e]
            for at, rnd in entries(e):
                raw_empty[at].arrive()
            at, rnd = e % BLOCKS, e // BLOCKS
            if rnd:
                yield b_empty[at], rnd - 1
            slot_holds[at][w] = names[e]
            yield None
            b_full[at].arrive()

    def products():
        at, items_of, units_of = [0], [0, 0], [0, 0]

        def pair(move=True):
            b = at[0]
            if move:
                at[0] += 2
            return b

        def full(b):
            for h in range(2):
                yield b_full[(b + h) % BLOCKS], (b + h) // BLOCKS

        def blocks(b, name):
            for h in range(2):
                assert all(x == (*name, h) for x in slot_holds[(b + h) % BLOCKS]), (slot_holds[(b + h) % BLOCKS], name, h)

        def scores(buf, tile, k, i, b):
            def done():
                blocks(b, (k, i, False))
                assert all(q == k for q in Q[tile][:soft])
                S[buf] = ("s", k, i, set())
            tensor.append(("op", done))
            tensor.append(("commit", s_full[buf]))

        def values(buf, tile, k, i, b, done_bar):
            def done():
                blocks(b, (k, i, True))
                assert S[buf][:3] == ("p", k, i) and len(S[buf][3]) == soft, S[buf]
                if i:
                    assert O[tile] == (k, i)
                O[tile] = (k, i + 1)
            tensor.append(("op", done))
            tensor.append(("commit", o_done[done_bar]))

        def empty(b):
            for h in range(2):
                tensor.append(("commit", b_empty[(b + h) % BLOCKS]))

        for k, (n, tiles) in enumerate(items):
            for t in range(tiles):
                yield q_full[t], items_of[t]
                items_of[t] += 1
            if NT == 1:
                b = pair()
                yield from full(b)
                scores(units_of[0] & 1, 0, k, 0, b)
                empty(b)
                for i in range(n):
                    j = units_of[0]
                    if i + 1 < n:
                        b = pair()
                        yield from full(b)
                        scores((j + 1) & 1, 0, k, i + 1, b)
                        empty(b)
                    b = pair()
                    yield from full(b)
                    yield p_full[j & 1], j >> 1
                    values(j & 1, 0, k, i, b, j & 1)
                    empty(b)
                    units_of[0] += 1
            else:
                b = pair()
                yield from full(b)
                for t in range(tiles):
                    scores(t, t, k, 0, b)
                empty(b)
                for i in range(n):
                    vb = pair()
                    yield from full(vb)
                    kb = pair(False)
                    for t in range(tiles):
                        yield p_full[t], units_of[t]
                        units_of[t] += 1
                        values(t, t, k, i, vb, t)
                        if t + 1 == tiles:
                            empty(vb)
                        if i + 1 < n:
                            if t == 0:
                                yield from full(kb)
                            scores(t, t, k, i + 1, kb)
                    if i + 1 < n:
                        empty(kb)
                        pair()

    arrived = {}

    def meet(key, who, count):                   # a named barrier
        arrived.setdefault(key, set()).add(who)
        while len(arrived[key]) < count:
            yield None

    def softmax(warp):
        tile, me, run = warp // soft, warp % soft, 0
        for k, (n, tiles) in enumerate(items):
            active = tile < tiles
            if active:
                Q[tile][me] = k
                yield None
                q_full[tile].arrive()
            if active:
                yield from meet(("q", k, tile), me, soft)
            for i in range(n if active else 0):
                buf = tile if NT == 2 else run & 1
                yield s_full[buf], run if NT == 2 else run >> 1
                assert S[buf][1:3] == (k, i) and (S[buf][0] == "s" or me not in S[buf][3]), (S[buf], k, i)
                yield None
                yield from meet(("max", k, tile, i), me, soft)
                if i and rng.random() < 0.5:     # the maximum moved: O is rescaled
                    if NT == 1:
                        yield o_done[(run - 1) & 1], (run - 1) >> 1
                    assert O[tile] == (k, i), (O[tile], k, i)
                    yield None
                    assert O[tile] == (k, i)
                yield None
                S[buf] = ("p", k, i, S[buf][3] | {me})
                p_full[buf].arrive()
                run += 1
            if active:
                yield from meet(("sum", k, tile), me, soft)
            if active:
                if NT == 2:
                    yield o_done[tile], run - 1
                else:
                    yield o_done[(run - 1) & 1], (run - 1) >> 1
                assert O[tile] == (k, n)
                yield None
                assert O[tile] == (k, n)

    gens = {"copies": copies(), "products": products()}
    gens.update({"convert%d.%d" % (g, w): convert(g, w) for g in range(2) for w in range(warps)})
    gens.update({"softmax%d" % w: softmax(w) for w in range(NT * soft)})
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
    return [(rng.choice([1, 1, 2, 3, 4, 7, 11]), rng.randint(1, NT)) for _ in range(rng.randint(1, 8))]


def constants():
    """(blocks, entries of a block, entries of a group) of d 256, and of the others, as the kernel has them."""
    s = open(SRC).read()
    b = re.search(r"BLOCKS = D == 256 \? (\d+) : (\d+);", s)
    e = re.search(r"PIECES = D == 256 \? (\d+) : (\d+);", s)
    t = re.search(r"TURN = (\d+),", s)
    return tuple((int(b[i]), int(e[i]), int(t[1])) for i in (1, 2))


@pytest.mark.parametrize("NT,wide", [(1, True), (1, False), (2, False)])
@pytest.mark.parametrize("seed", range(60))
def test_protocol(NT, wide, seed):
    rng = random.Random(seed)
    assert run(NT, *constants()[0 if wide else 1], items(rng, NT), rng)
