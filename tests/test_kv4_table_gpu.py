"""Page tables and rows as callers may have them: sequences longer than their
table, tables and outputs that are slices of wider ones, a workspace of just
the size that a call asks for."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import kv4_reference as ref  # noqa: E402
from test_kv4_gpu import ints, randn, rng_of, sv  # noqa: E402,F401

INSTANCES = [(d, T, G) for d in (64, 128, 256) for T, G in ((2, 3), (8, 2), (60, 2), (250, 2))]


def within_table(q, cache, table, lens, window, sinks):
    """As ref.attention; tokens past the table are left out, and a row that sees none gives zeros."""
    B, T, Hq, d = q.shape
    Hk, n = cache.shape[1], table.shape[1] * 32
    out = [torch.zeros(q.shape, dtype=torch.float64, device="cuda") for _ in range(3)]
    for b, before in enumerate(lens):
        k, v = ref.tokens(cache, table[b], n)
        p, j = before + torch.arange(T, device="cuda")[:, None], torch.arange(n, device="cuda")
        seen = j <= p
        if window:
            seen &= (p - j < window) | (j < sinks)
        s = torch.einsum("thgd,jhd->thgj", q[b].double().unflatten(1, (Hk, -1)), k) * d ** -0.5
        w = torch.softmax(torch.where(seen[:, None, None], s, -torch.inf), -1).nan_to_num(0)
        out[0][b] = torch.einsum("thgj,jhd->thgd", w, v).flatten(1, 2)
        out[1][b] = torch.einsum("thgj,jhd->thgd", w, v.abs()).flatten(1, 2)
        out[2][b] = v.abs().max() * n
    return out


@pytest.mark.parametrize("d,T,G", INSTANCES)
@pytest.mark.parametrize("pages", [4, 5])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 0), (50, 4), (300, 40), (1 << 30, 1)])
def test_sequences_longer_than_their_table(sv, d, T, G, pages, window, sinks):  # noqa: F811
    """Rows past the table's end are reported and see what it holds of their window, not of another one."""
    gen = rng_of(d + T + pages)
    lens = [100, 32 * pages - 1, 32 * pages, 200, 5000, (1 << 30) - 1, 1 << 30, (1 << 30) + 100, (1 << 31) - 1]
    cache = ref.filled(gen, pages * len(lens), 2, d)
    table = ref.shuffled(gen, [pages] * len(lens), slack=0)
    q = (2 * randn(gen, len(lens), T, 2 * G, d)).bfloat16()
    o = sv.kv4_attention(q, cache, table, ints(lens), window=window, sinks=sinks)
    assert sv.last_device_error() == sv.DEVERR_BAD_PAGE
    want = within_table(q, cache, table, lens, window, sinks)
    ref.check_attention(o, want)
    nothing = want[1].sum(-1) == 0
    assert not o[nothing].any() and (sinks > 0 or window == 0 or bool(nothing.any()))


@pytest.mark.parametrize("d,T,G", INSTANCES)
@pytest.mark.parametrize("ragged", [False, True])
def test_workspace_of_just_the_size(sv, d, T, G, ragged):  # noqa: F811
    """As many bytes as asked for give the same bits, and none behind them is written; with one fewer the call is
    refused."""
    gen = rng_of(d + T)
    lens = [1500, 0, 333]
    need = [-(-(n + T) // 32) for n in lens]
    cache, table = ref.filled(gen, sum(need), 2, d), ref.shuffled(gen, need)
    q = randn(gen, 3, T, 2 * G, d).bfloat16()
    cu = None
    if ragged:
        q, cu = q.flatten(0, 1), ints([0, T, 2 * T, 3 * T])
    n = sv.kv4_attention_bytes(q, cache, table, cu)
    want = sv.kv4_attention(q, cache, table, ints(lens), cu)
    whole = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    assert torch.equal(sv.kv4_attention(q, cache, table, ints(lens), cu, workspace=whole[:n]), want)
    assert bool((whole[n:] == 0xA5).all())
    with pytest.raises(sv.SpecVerifyError):
        sv.kv4_attention(q, cache, table, ints(lens), cu, workspace=whole[:n - 1])
    ref.check_attention(want, ref.attention(q, cache, table, ints(lens), cu))
    assert sv.last_device_error() == 0


@pytest.mark.parametrize("d,T,G", INSTANCES)
def test_slices(sv, d, T, G):  # noqa: F811
    """A page table and outputs that are slices of wider ones: the same bits, and nothing beside them is written."""
    gen = rng_of(d + G)
    lens = [700, 31, 2000]
    need = [-(-(n + T) // 32) for n in lens]
    cache, table = ref.filled(gen, sum(need), 2, d), ref.shuffled(gen, need)
    wide = torch.full((3, table.shape[1] + 9), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, 4:-5] = table
    q = randn(gen, 3, T, 2 * G + 3, d).bfloat16()[:, :, 1:-2]
    want = sv.kv4_attention(q.contiguous(), cache, table, ints(lens))
    ref.check_attention(want, ref.attention(q, cache, table, ints(lens)))
    out = torch.full((3, T, 2 * G + 2, d), 7.0, device="cuda").bfloat16()
    o = out[:, :, 1:-1]
    assert sv.kv4_attention(q, cache, wide[:, 4:-5], ints(lens), o=o) is o
    assert torch.equal(o, want) and bool((out[:, :, 0] == 7).all()) and bool((out[:, :, -1] == 7).all())
    k, v = (randn(gen, 3, T, 2, d).bfloat16() for _ in range(2))
    same = cache.clone()
    sv.kv4_append(k, v, cache, table, ints(lens))
    sv.kv4_append(k, v, same, wide[:, 4:-5], ints(lens))
    assert torch.equal(cache, same)
    for a, b in zip(sv.kv4_gather(cache, table, ints(lens), T), sv.kv4_gather(cache, wide[:, 4:-5], ints(lens), T)):
        assert torch.equal(a, b)
    assert sv.last_device_error() == 0
