"""Attention layers as decoding uses them: verify cycles that append drafts,
drop the rejected ones by their lengths alone and go on, against the same
tokens one at a time; and examples/hybrid_decode.py with such layers."""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import kv4_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("hybrid_decode", os.path.join(ROOT, "examples", "hybrid_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("d,Hq,Hk", [(64, 6, 2), (128, 8, 1), (256, 24, 4)])
@pytest.mark.parametrize("T,window", [(1, 0), (4, 0), (8, 40)])
def test_cycles_leave_what_single_rows_leave(ex, d, Hq, Hk, T, window):
    """Two ragged prompts, then cycles of T rows of which a drawn number holds.
    The rotated keys of a position do not depend on the rows beside it, so the
    accepted tokens' bytes are those of a cache that was filled in one call; the
    outputs are held to the formula over it."""
    sv = ex.sv
    gen = torch.Generator(device="cuda").manual_seed(5)
    lens, total = [45, 3], 130
    qkv = torch.randn(2, total, Hq + 2 * Hk, d, device="cuda", generator=gen).bfloat16()
    wrong = torch.randn(2, total + T, Hq + 2 * Hk, d, device="cuda", generator=gen).bfloat16()
    f = 1e4 ** (-torch.arange(d // 2, device="cuda") * 2 / d)
    table = ref.shuffled(gen, [5, 5])
    cache = sv.kv4_cache(10, Hk, d)

    def layer(x, pos, at, cu=None):
        q, k, v = x.split((Hq, Hk, Hk), -2)
        q, k = sv.rotary(q, k, pos, f)
        sv.kv4_append(k, v, cache, table, at, cu)
        return q, sv.kv4_attention(q, cache, table, at, cu, window=window, sinks=2)

    step = torch.arange(total, dtype=torch.int32, device="cuda")
    layer(torch.cat([qkv[b, :n] for b, n in enumerate(lens)]), torch.cat([step[:n] for n in lens]), ints([0, 0]),
          ints([0, lens[0], sum(lens)]))
    whole = sv.kv4_cache(10, Hk, d)
    q, k, v = qkv.split((Hq, Hk, Hk), -2)
    _, k = sv.rotary(q, k, step.expand(2, -1).contiguous(), f)
    sv.kv4_append(k, v, whole, table, ints([0, 0]))
    rng = np.random.default_rng(6)
    while max(lens) + T <= total:
        held = [int(rng.integers(1, T + 1)) for _ in lens]
        x = torch.stack([torch.cat([qkv[b, n:n + a], wrong[b, n + a:n + T]]) for b, (n, a) in enumerate(zip(lens, held))])
        at = ints(lens)
        q, o = layer(x, at[:, None] + step[:T], at)
        want = ref.attention(q, whole, table, at, window=window, sinks=2)
        for b, a in enumerate(held):
            ref.check_attention(o[b:b + 1, :a], [w[b:b + 1, :a] for w in want])
        lens = [n + a for n, a in zip(lens, held)]
    got, all_ = (sv.kv4_gather(c, table, ints([0, 0]), total) for c in (cache, whole))
    for g, w in zip(got, all_):
        for b, n in enumerate(lens):
            assert torch.equal(g[b, :n], w[b, :n])
    assert sv.last_device_error() == 0


@pytest.mark.parametrize("every,window", [(1, 0), (2, 0), (2, 50)])
def test_example_runs_with_attention_layers(ex, every, window):
    cfg = ex.Config(layers=4, attention_every=every, window=window)
    model = ex.Model(cfg, seed=3)
    rng = np.random.default_rng(4)
    prompts = [rng.integers(0, cfg.vocab, n).tolist() for n in (131, 1, 70)]
    plain, cycles, _ = ex.generate(model, prompts, 12)
    assert cycles == 11 and all(len(t) == 12 and all(0 <= x < cfg.vocab for x in t) for t in plain)
    new, cycles, _ = ex.generate(model, prompts, 12, 3, ex.drafter([p + t for p, t in zip(prompts, plain)]))
    assert all(len(t) >= 12 for t in new) and cycles <= 11
    assert ex.sv.last_device_error() == 0
