"""Rotary positions, the 4-bit cache and the attention over it against their
definitions in 64 bits (tolerances: check_attention of kv4_reference, and
beside each test)."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import kv4_reference as ref  # noqa: E402


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_verify_gb300 as m
    from speculative_verify_gb300 import build
    build.build()
    m.load()
    assert m.last_device_error() == 0
    return m


def rng_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *s):
    return torch.randn(*s, device="cuda", generator=g)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------- rotary


def rotary64(x, positions, inv_freq, axes, interleaved, factor):
    h = len(inv_freq)
    y = x.double().clone()
    for i in range(h):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        t = positions[axes[i]].double() * inv_freq[i].double()
        c, s = factor * torch.cos(t)[..., None], factor * torch.sin(t)[..., None]
        u, v = x[..., a].double(), x[..., b].double()
        y[..., a], y[..., b] = u * c - v * s, v * c + u * s
    return y


def check_rotary(y, x, want, factor=1.0):
    """Half a bf16 step, and angles within 2^-24 of a turn with fp32 products: 2e-6 of the pair."""
    err = (y.double() - want).abs()
    pair = x.double().abs().amax(-1, keepdim=True) * 2 * abs(factor)
    assert bool((err <= 2.0 ** -8 * want.abs() + 2e-6 * pair + 1e-38).all()), float(err.max())


@pytest.mark.parametrize("rows", [1, 2, 7, 333, 5000])
@pytest.mark.parametrize("Hq,Hk,d,rot", [(24, 4, 256, 64), (4, 2, 128, 128), (7, 1, 64, 16), (1, 0, 16, 16), (3, 5, 1024, 512),
                                         (2, 2, 72, 48)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary(sv, rows, Hq, Hk, d, rot, interleaved):
    g = rng_of(rows + d)
    qkv = randn(g, rows, (Hq + Hk + 1) * d).bfloat16()
    q = qkv[:, :Hq * d].unflatten(1, (Hq, d))
    k = qkv[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d)) if Hk else None
    axes = ints([i % 3 for i in range(rot // 2)])
    positions = torch.randint(-1000, 1 << 20, (3, rows), device="cuda", generator=g).to(torch.int32)
    inv_freq = 10000.0 ** (-torch.arange(rot // 2, device="cuda") * 2 / rot)
    yq, yk = sv.rotary(q, k, positions, inv_freq, axes=axes, interleaved=interleaved, factor=1.25)
    for x, y in ((q, yq), (k, yk)):
        if x is None:
            assert y is None
            continue
        check_rotary(y, x, rotary64(x, positions, inv_freq, axes.tolist(), interleaved, 1.25), 1.25)
        assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_in_place_and_batched(sv, interleaved):
    """[B][T] rows, one axis, in place: the same bits as out of place, nothing else written."""
    g = rng_of(5)
    qkv = randn(g, 3, 5, 7 * 64).bfloat16()
    keep = qkv.clone()
    q, k = qkv[..., :4 * 64].unflatten(-1, (4, 64)), qkv[..., 4 * 64:6 * 64].unflatten(-1, (2, 64))
    positions = torch.randint(0, 300000, (3, 5), device="cuda", generator=g).to(torch.int32)
    f = 1e6 ** (-torch.arange(16, device="cuda") / 16)
    yq, yk = sv.rotary(q, k, positions, f, interleaved=interleaved)
    check_rotary(yq, q, rotary64(q, positions[None], f, [0] * 16, interleaved, 1.0))
    rq, rk = sv.rotary(q, k, positions[None].contiguous(), f, interleaved=interleaved, q_out=q, k_out=k)
    assert rq is q and rk is k and torch.equal(q, yq) and torch.equal(k, yk)
    assert torch.equal(qkv[..., 6 * 64:], keep[..., 6 * 64:])


def test_rotary_far_positions(sv):
    """The smallest and largest positions, and a frequency above one step: angles reduced without loss."""
    g = rng_of(6)
    positions = ints([0, 1, -1, 2**31 - 1, -2**31, 123456789, 2**24 + 1])
    f = torch.tensor([1.0, 0.7310585786, 1e-7, 0.0, -0.25, 0.999999, 2.5, 3.0], device="cuda")
    x = randn(g, 7, 2, 16).bfloat16()
    y, _ = sv.rotary(x, None, positions, f)
    check_rotary(y, x, rotary64(x, positions[None], f, [0] * 8, False, 1.0))


def test_rotary_special(sv):
    """A NaN or infinite frequency reaches its own pair only; an axis out of range is axis 0, and reported; no rows."""
    g = rng_of(7)
    x = randn(g, 3, 2, 32).bfloat16()
    f = torch.tensor([1.0, math.nan, 0.5, math.inf] + [0.1] * 12, device="cuda")
    y, _ = sv.rotary(x, None, ints([1, 2, 3]), f)
    bad = torch.zeros(32, dtype=torch.bool, device="cuda")
    bad[[1, 3, 17, 19]] = True
    assert bool(y[..., bad].isnan().all()) and bool(y[..., ~bad].isfinite().all())
    f = torch.rand(16, device="cuda", generator=g)
    positions = ints([[5, 6, 7], [0, 0, 0]])
    y, _ = sv.rotary(x, None, positions, f, axes=ints([0, 2, -1] + [1] * 13))
    assert sv.last_device_error() == sv.DEVERR_BAD_AXIS
    check_rotary(y, x, rotary64(x, positions, f, [0, 0, 0] + [1] * 13, False, 1.0))
    y, k = sv.rotary(x[:0], x[:0], ints([]), f)
    assert y.shape == (0, 2, 32) and k.shape == (0, 2, 32)


# -------------------------------------------------------------------- cache


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Hk", [1, 3, 8])
@pytest.mark.parametrize("T,lens", [(1, [0]), (1, [31, 32, 63, 5]), (5, [30, -1, 0, 77]), (33, [1, 95])])
def test_append_rows(sv, d, Hk, T, lens):
    """Every byte of the cache: the rows' codes and scales, and nothing else.  Power-of-two scales: a quotient of an
    8-bit by a 4-bit number (or by six) is either exactly between two codes or 2^-14 away, so 64 and 32 bits agree."""
    g = rng_of(d + Hk + T)
    B = len(lens)
    kv = (randn(g, B, T, 3 * Hk * d) * torch.exp(2 * randn(g, B, T, 1))).bfloat16()
    k, v = kv[..., :Hk * d].unflatten(-1, (Hk, d)), kv[..., 2 * Hk * d:].unflatten(-1, (Hk, d))
    k[0, 0, 0, :16] = 0
    v[0, 0, 0, 16:32] *= 1e-4                   # scales below the smallest
    k[-1, 0, 0, 32:48] *= 1e5                   # and above the largest
    need = [max(0, (n + T + 31) // 32) for n in lens]
    table = ref.shuffled(g, need, sum(need) + 3)
    cache = torch.randint(0, 256, (sum(need) + 3, Hk, 36 * d), device="cuda", generator=g).to(torch.uint8)
    want = cache.clone()
    for x, codes, scales, scale in zip((k, v), ref.pieces(want)[:2], ref.pieces(want)[2:], (0.5, 2.0)):
        c, s = ref.quantise(x, scale)
        for b, n in enumerate(lens):
            for t in range(T if n >= 0 else 0):
                page = int(table[b, (n + t) // 32])
                codes[page, :, (n + t) % 32] = (c[b, t, :, ::2] + 16 * c[b, t, :, 1::2]).to(torch.uint8)
                scales[page, :, (n + t) % 32] = s[b, t]
    sv.kv4_append(k, v, cache, table, ints(lens), k_scale=0.5, v_scale=2.0)
    assert torch.equal(cache, want)
    assert sv.last_device_error() == 0
    gk, gv = sv.kv4_gather(cache, table, ints(lens), T, k_scale=0.5, v_scale=2.0)
    for got, codes, scales, scale in zip((gk, gv), ref.pieces(want)[:2], ref.pieces(want)[2:], (0.5, 2.0)):
        for b, n in enumerate(lens):
            if n < 0:
                assert not got[b].any()
                continue
            at = torch.arange(n, n + T, device="cuda")
            page = table[b, at // 32].long()
            x = ref.read(codes[page, :, at % 32], scales[page, :, at % 32]) * scale
            assert torch.equal(got[b].double(), x)              # six bits: exact in bf16


def test_append_ragged(sv):
    """cu_seqlens with an empty sequence, an inactive one and rows of no sequence; a scale that is no power of two: the
    restored value is off by at most the largest half step, 1 of the scale, plus the output's rounding."""
    g = rng_of(8)
    lens, cu, R, Hk, d = [40, 0, -1, 7], [2, 35, 35, 40, 139], 150, 2, 128
    k, v = (randn(g, R, Hk, d).bfloat16() for _ in range(2))
    table = ref.shuffled(g, [4, 0, 0, 4])
    cache = torch.zeros(8, Hk, 36 * d, dtype=torch.uint8, device="cuda")
    sv.kv4_append(k, v, cache, table, ints(lens), cu_seqlens=ints(cu), k_scale=0.05, v_scale=0.3)
    out = [torch.full((R, Hk, d), 7.0, device="cuda").bfloat16() for _ in range(2)]
    got = sv.kv4_gather(cache, table, ints(lens), R, cu_seqlens=ints(cu), k_scale=0.05, v_scale=0.3, k=out[0], v=out[1])
    assert got[0] is out[0] and got[1] is out[1]
    for x, y in ((k, got[0]), (v, got[1])):
        assert bool((y[:2] == 7).all()) and bool((y[139:] == 7).all()) and not y[35:40].any()
        for a, b in ((2, 35), (40, 139)):
            u, w = x[a:b].double().unflatten(-1, (-1, 16)), y[a:b].double().unflatten(-1, (-1, 16))
            step = u.abs().amax(-1, keepdim=True) / 6 * (1 + 2.0 ** -4)
            assert bool(((w - u).abs() <= step + 2.0 ** -8 * w.abs() + 1e-6).all())
    assert sv.last_device_error() == 0


def test_append_not_a_number(sv):
    """NaN and infinity: a NaN scale of their 16 dimensions, and the token's first K scale of that head."""
    g = rng_of(9)
    k, v = (randn(g, 1, 4, 2, 64).bfloat16() for _ in range(2))
    k[0, 1, 0, 20] = math.nan
    v[0, 2, 1, 63] = -math.inf
    cache, table = torch.zeros(1, 2, 36 * 64, dtype=torch.uint8, device="cuda"), ints([[0]])
    sv.kv4_append(k, v, cache, table, ints([3]))
    ks, vs = ref.pieces(cache)[2:]
    bad_k, bad_v = (ks[0] & 0x7F) == 0x7F, (vs[0] & 0x7F) == 0x7F
    assert bad_k.nonzero().tolist() == [[0, 4, 0], [0, 4, 1], [1, 5, 0]]
    assert bad_v.nonzero().tolist() == [[1, 5, 3]]
    gk, gv = sv.kv4_gather(cache, table, ints([3]), 4)
    assert gk.isnan().sum() == 48 and gv.isnan().sum() == 16


def test_cache_without_pages(sv):
    """Tokens past the table, on entries out of range: reported, not written, read as zeros."""
    g = rng_of(10)
    k, v = (randn(g, 2, 40, 1, 64).bfloat16() for _ in range(2))
    cache = torch.zeros(3, 1, 36 * 64, dtype=torch.uint8, device="cuda")
    table = ints([[0, 3], [-1, 2]])
    sv.kv4_append(k, v, cache, table, ints([10, 30]))
    assert sv.last_device_error() == sv.DEVERR_BAD_PAGE
    assert not cache[1].any()
    gk, gv = sv.kv4_gather(cache, table, ints([10, 30]), 40)
    assert sv.last_device_error() == sv.DEVERR_BAD_PAGE
    assert gk[0, :22].any() and not gk[0, 22:].any() and not gk[1, :2].any() and gk[1, 2:34].any() and not gk[1, 34:].any()
    assert not gv[0, 22:].any() and not gv[1, 34:].any()
    q = randn(g, 2, 40, 1, 64).bfloat16()
    o = sv.kv4_attention(q, cache, table, ints([10, 30]))
    assert sv.last_device_error() == sv.DEVERR_BAD_PAGE and bool(o.isfinite().all())
    # sequence 1's first rows (positions 30, 31) see no token that has a page
    assert not o[1, :2].any()


# ---------------------------------------------------------------- attention


def run(sv, seed, lens, rows, Hq, Hk, d, window=0, sinks=0, ragged=False, scale=None, g=(1.0, 1.0), peak=2.0, n_pages=None):
    """q and the result of a call on a filled cache, and the reference."""
    gen = rng_of(seed)
    need = [max(0, -(-(n + r) // 32)) for n, r in zip(lens, rows)]
    table = ref.shuffled(gen, need, n_pages)
    cache = ref.filled(gen, max(1, n_pages or sum(need)), Hk, d)
    q = peak * randn(gen, sum(rows), Hq + 1, d).bfloat16()
    cu = None
    if ragged:
        cu = ints([sum(rows[:b]) for b in range(len(rows) + 1)])
    else:
        q = q.unflatten(0, (len(rows), rows[0]))
    q = q[..., :Hq, :]                          # rows with something behind them
    kw = dict(scale=scale, window=window, sinks=sinks)
    o = sv.kv4_attention(q, cache, table, ints(lens), cu_seqlens=cu, k_scale=g[0], v_scale=g[1], **kw)
    assert o.shape == q.shape and sv.last_device_error() == 0
    want = ref.attention(q, cache, table, ints(lens), cu, g=g, **kw)
    ref.check_attention(o, want)
    return q, cache, table, o


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (6, 1), (6, 2), (16, 2), (40, 2), (3, 3)])
@pytest.mark.parametrize("T", [1, 2, 5, 8, 32])
def test_decode_and_verify_rows(sv, d, Hq, Hk, T):
    run(sv, d + T + Hq, [0, 1, 30, 31, 32, 33, 64, 500, -1, 1029], [T] * 10, Hq, Hk, d)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hk,T", [(6, 2, 1), (6, 2, 4), (20, 1, 7)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (32, 0), (33, 32), (100, 40), (257, 1000), (5000, 7)])
def test_window_and_sinks(sv, d, Hq, Hk, T, window, sinks):
    run(sv, d + T + window, [0, 3, 31, 40, 132, 133, 700, 1500], [T] * 8, Hq, Hk, d, window, sinks)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,G", [(1, 4), (4, 4), (9, 3), (150, 2)])
@pytest.mark.parametrize("before", [300, 320, 345, 363])
@pytest.mark.parametrize("window,sinks", [(70, 0), (33, 7), (96, 40), (64, 70)])
def test_pages_before_the_windows_may_be_gone(sv, d, T, G, before, window, sinks):
    """Table entries of pages that no row sees are no pages: not reported, and the same bits."""
    gen = rng_of(17)
    n = (before + T + 31) // 32
    cache, table = ref.filled(gen, n, 1, d), ref.shuffled(gen, [n])
    q = randn(gen, 1, T, G, d).bfloat16()
    kw = dict(window=window, sinks=sinks)
    want = sv.kv4_attention(q, cache, table, ints([before]), **kw)
    first = max(0, before - window + 1)         # that the first row sees, besides the sinks
    for i in range((min(sinks, first) + 31) // 32, first // 32):
        table[0, i] = -1
    assert bool((table < 0).any())
    got = sv.kv4_attention(q, cache, table, ints([before]), **kw)
    assert sv.last_device_error() == 0 and torch.equal(got, want)
    ref.check_attention(got, ref.attention(q, cache, table.clamp(min=0), ints([before]), **kw))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 5)])
@pytest.mark.parametrize("Hq,Hk", [(4, 1), (8, 8), (24, 4), (7, 1)])
def test_prompts(sv, d, window, sinks, Hq, Hk):
    run(sv, d + Hq, [0, 0, 17, 64, -1, 333, 5], [1, 129, 0, 40, 9, 300, 64], Hq, Hk, d, window, sinks, ragged=True)


@pytest.mark.parametrize("d,Hq,Hk", [(64, 8, 2), (128, 32, 8), (256, 12, 2)])
def test_long_prompt(sv, d, Hq, Hk):
    run(sv, d, [100], [2100], Hq, Hk, d, ragged=True)
    run(sv, d + 1, [1000, 0], [1111, 700], Hq, Hk, d, window=512, sinks=64, ragged=True)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,B", [(1, 1), (4, 1), (1, 3), (8, 2)])
def test_long_contexts(sv, d, T, B):
    """Sequences spread over many blocks and joined; a long cache beside short ones."""
    run(sv, d + T + B, [33000 // B, 5, 12345][:B], [T] * B, 12, 2, d)


def test_many_sequences(sv):
    run(sv, 1, [(37 * b) % 300 - (b % 9 == 0) for b in range(260)], [1] * 260, 16, 8, 128)
    run(sv, 2, [(11 * b) % 90 for b in range(70)], [b % 5 for b in range(70)], 8, 2, 64, ragged=True)


def test_more_sequences_than_the_warps_share_out(sv):
    """Beyond 64 groups of 32 sequences: rows everywhere, and a few among thousands that have none."""
    run(sv, 3, [(7 * b) % 70 for b in range(2100)], [1] * 2100, 2, 1, 64)
    rows = [0] * 2300
    for b, n in ((0, 3), (31, 1), (1000, 40), (2047, 2), (2048, 17), (2299, 5)):
        rows[b] = n
    run(sv, 4, [(13 * b) % 200 - 1 for b in range(2300)], rows, 4, 2, 128, ragged=True)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("many,long,G", [(40, 700, 4), (60, 300, 2), (3, 2000, 1)])
def test_decode_rows_beside_a_prompt(sv, d, many, long, G):
    """Single rows and a long prompt in a call, whichever kernel their average picks; some sequences inactive."""
    lens = [(97 * b) % 900 - (b % 7 == 3) * 1000 for b in range(many)]
    run(sv, 5, lens[:many // 2] + [130] + lens[many // 2:], [1] * (many // 2) + [long] + [1] * (many - many // 2), 2 * G, 2, d,
        ragged=True)


def test_nothing_active(sv):
    q, cache, table, o = run(sv, 6, [-1, -5, -1], [4] * 3, 8, 2, 128)
    assert not o.any()


def test_scales(sv):
    """A scale of the scores, and scales of the cache that are no powers of two."""
    run(sv, 3, [100, 700], [3, 3], 6, 2, 128, scale=0.3, g=(0.05, 3.7), peak=1.0)
    run(sv, 4, [100, 700], [3, 3], 6, 2, 256, scale=-0.02, g=(1.0, 1e-3))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rising_scores(sv, d):
    """Maxima that move on every page, scores far apart (p from 1 to below the smallest fp16)."""
    gen = rng_of(d)
    cache, table = ref.filled(gen, 12, 1, d), ref.shuffled(gen, [12])
    ks = ref.pieces(cache)[2]
    for i in range(12):
        ks[table[0, i].long()] = 0x30 + 2 * i   # larger keys page by page
    q = (3 * randn(gen, 1, 5, 4, d)).bfloat16()
    for t in (1.0, -1.0):
        o = sv.kv4_attention((t * q).bfloat16(), cache, table, ints([379]))
        ref.check_attention(o, ref.attention((t * q).bfloat16(), cache, table, ints([379])))


@pytest.mark.parametrize("d,T", [(64, 3), (128, 3), (256, 3), (128, 150)])
def test_not_a_number_stays_with_rows_that_see_it(sv, d, T):
    """NaN tokens: ahead of a row, out of its window, behind the sequence's end, in the place of another row of the
    call; query rows that hold a NaN or an infinity."""
    gen = rng_of(d)
    lens, window = [50, 200], 20
    cache, table = ref.filled(gen, 40, 1, d), ref.shuffled(gen, [12, 12], 40)
    for p in ref.pieces(cache)[2:]:
        p[table[0, 50 // 32].long(), :, 50 % 32 + 1] = 0x7F     # the second row's own token
        p[table[1, 0].long(), :, 9] = 0xFF                      # out of every window (with sinks)
    for b, n in enumerate(lens):                                # behind the end
        at = n + T
        while at % 32:
            for p in ref.pieces(cache)[2:]:
                p[table[b, at // 32].long(), :, at % 32] = 0x7F
            at += 1
    q = randn(gen, 2, T, 8, d).bfloat16()
    q[1, 1, 2, 5] = math.nan
    q[1, 1, 4, 6] = math.inf
    o = sv.kv4_attention(q, cache, table, ints(lens), window=window, sinks=4)
    bad = o.isnan().any(-1)
    want = torch.zeros(2, T, 8, dtype=torch.bool, device="cuda")
    want[0, 1:1 + window] = True
    want[1, 1, 2] = want[1, 1, 4] = True
    assert torch.equal(bad, want) and bool(o[~want].isfinite().all())
    clean = q.clone()
    clean[1, 1, 2] = clean[1, 1, 4] = 0         # (their rows are left out below)
    for p in ref.pieces(cache)[2:]:
        p[(p & 0x7F) == 0x7F] = 0x30
    r = ref.attention(clean, cache, table, ints(lens), window=window, sinks=4)
    ref.check_attention(torch.where(want[..., None], 0, o), [torch.where(want[..., None], 0, x) for x in r])


@pytest.mark.parametrize("d,T", [(64, 3), (128, 3), (256, 3), (64, 150), (128, 150), (256, 150)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_queries_that_are_no_numbers(sv, d, T, bad):
    """A row and head with a NaN or an infinity gives NaNs, the others what they give without it."""
    gen = rng_of(18)
    cache, table = ref.filled(gen, 12, 1, d), ref.shuffled(gen, [12])
    q = randn(gen, 1, T, 4, d).bfloat16()
    want = ref.attention(q, cache, table, ints([200]))
    q[0, T // 2, 1, 5] = q[0, T // 2, 1, d - 1] = bad
    o = sv.kv4_attention(q, cache, table, ints([200]))
    assert bool(o[0, T // 2, 1].isnan().all()) and int(o.isnan().sum()) == d
    o[0, T // 2, 1] = want[0][0, T // 2, 1].bfloat16()
    ref.check_attention(o, want)


def test_large_values(sv):
    """The largest scales and queries of every magnitude: no overflow on the way."""
    gen = rng_of(11)
    cache, table = ref.filled(gen, 8, 1, 128), ref.shuffled(gen, [8])
    for p in ref.pieces(cache)[2:]:
        p.fill_(0x7E)
    q = randn(gen, 1, 6, 2, 128).bfloat16()
    q *= torch.tensor([1e-38, 1e-20, 1e-6, 1.0, 1e4, 3e38], device="cuda").view(1, 6, 1, 1) / 4
    for scale in (1.0, 2e-4):
        o = sv.kv4_attention(q.bfloat16()[:, :5], cache, table, ints([200]), scale=scale * 1e-4)
        ref.check_attention(o, ref.attention(q.bfloat16()[:, :5], cache, table, ints([200]), scale=scale * 1e-4))
    o = sv.kv4_attention(q.bfloat16(), cache, table, ints([200]), scale=1e-38)
    ref.check_attention(o, ref.attention(q.bfloat16(), cache, table, ints([200]), scale=1e-38))


def test_far_pages(sv):
    """Offsets past 32 bits: a pool of 2.4 GB, pages from its end."""
    gen = rng_of(12)
    d, Hk, n = 256, 8, 33000
    cache = torch.zeros(n, Hk, 36 * d, dtype=torch.uint8, device="cuda")
    small = ref.filled(gen, 6, Hk, d)
    where = ints([n - 1, 0, n - 7, 31000, n - 2, 30001])
    cache[where.long()] = small
    q = randn(gen, 1, 2, 16, d).bfloat16()
    o = sv.kv4_attention(q, cache, where[None].contiguous(), ints([180]))
    want = ref.attention(q, small, torch.arange(6, device="cuda")[None].int(), ints([180]))
    ref.check_attention(o, want)
    k, v = (randn(gen, 1, 40, Hk, d).bfloat16() for _ in range(2))
    sv.kv4_append(k, v, cache, where[None].contiguous(), ints([10]))
    gk, _ = sv.kv4_gather(cache, where[None].contiguous(), ints([10]), 40)
    c, s = ref.quantise(k, 1.0)
    assert torch.equal(gk.double(), ref.read((c[..., ::2] + 16 * c[..., 1::2]).to(torch.uint8), s))


def test_same_bits_every_time(sv):
    """Results do not depend on timing, nor on a workspace's contents; rows of no sequence are not written."""
    gen = rng_of(13)
    cache, table = ref.filled(gen, 700, 2, 128), ref.shuffled(gen, [600, 90], 700)
    q = randn(gen, 300, 12, 128).bfloat16()
    cu, lens = ints([3, 40, 290]), ints([19000, 2000])
    o = torch.full_like(q, 5)
    sv.kv4_attention(q, cache, table, lens, cu_seqlens=cu, o=o)
    assert bool((o[:3] == 5).all()) and bool((o[290:] == 5).all())
    for fill in (0, 255):
        ws = torch.full((1 << 28,), fill, dtype=torch.uint8, device="cuda")
        again = sv.kv4_attention(q, cache, table, lens, cu_seqlens=cu, workspace=ws)
        assert torch.equal(again[3:290], o[3:290])


def test_bad_seqlens(sv):
    """cu_seqlens that decrease and claim more rows than there are: nothing is written, and reported."""
    gen = rng_of(14)
    cache, table = ref.filled(gen, 8, 1, 64), ref.shuffled(gen, [2, 2, 2, 2])
    q = randn(gen, 40, 2, 64).bfloat16()
    o = torch.full_like(q, 3)
    sv.kv4_attention(q, cache, table, ints([0, 0, 0, 0]), cu_seqlens=ints([0, 40, 0, 40, 40]), o=o)
    assert sv.last_device_error() == sv.DEVERR_BAD_SEQLENS and bool((o == 3).all())


def test_empty_calls(sv):
    cache = torch.zeros(1, 2, 36 * 64, dtype=torch.uint8, device="cuda")
    q = torch.zeros(0, 3, 4, 64, device="cuda").bfloat16()
    none = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    assert sv.kv4_attention(q, cache, none, ints([])).shape == q.shape
    q = torch.zeros(2, 0, 4, 64, device="cuda").bfloat16()
    two = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    assert sv.kv4_attention(q, cache, two, ints([0, 0])).shape == q.shape
    sv.kv4_append(q[:, :, :2], q[:, :, :2], cache, two, ints([0, 0]))
    assert sv.kv4_gather(cache, two, ints([0, 0]), 0)[0].shape == (2, 0, 2, 64)


def test_graphs_and_streams(sv):
    """A cycle (rotary, append, attention) captured twice, replayed on two streams at once, against eager calls; new
    lengths and tables are read at replay."""
    gen = rng_of(15)
    Hq, Hk, d, T = 12, 2, 128, 3
    cases = []
    for i in range(2):
        cache, table = ref.filled(gen, 800, Hk, d), ref.shuffled(gen, [700, 90], 800)
        qkv = randn(gen, 2, T, (Hq + 2 * Hk) * d).bfloat16()
        f = 1e6 ** (-torch.arange(d // 2, device="cuda") * 2 / d)
        cases.append((cache, table, qkv, f, ints([0, 0])))

    def cycle(cache, table, qkv, f, lens):
        q, k, v = (t.unflatten(-1, (-1, d)) for t in qkv.split((Hq * d, Hk * d, Hk * d), -1))
        pos = lens[:, None] + torch.arange(T, device="cuda", dtype=torch.int32)
        q, k = sv.rotary(q, k, pos, f)
        sv.kv4_append(k, v, cache, table, lens)
        return sv.kv4_attention(q, cache, table, lens)

    eager = []
    for i, c in enumerate(cases):
        c[-1].copy_(ints([20000 + i, 1000]))
        eager.append((cycle(*c).clone(), c[0].clone()))
    graphs, outs = [], []
    for c in cases:
        c[-1].copy_(ints([0, 0]))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(cycle(*c))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in cases]
    for i, c in enumerate(cases):
        c[-1].copy_(ints([20000 + i, 1000]))
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (o, cache), got, c in zip(eager, outs, cases):
        assert torch.equal(o, got) and torch.equal(cache, c[0])
    # a stream argument: the work is ordered on it
    c = cases[0]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    q = randn(gen, 2, T, Hq, d).bfloat16()
    torch.cuda.synchronize()
    o = sv.kv4_attention(q, c[0], c[1], c[-1], stream=s)
    s.synchronize()
    assert torch.equal(o, sv.kv4_attention(q, c[0], c[1], c[-1]))


@pytest.mark.parametrize("d,Hq", [(64, 16), (128, 16), (256, 16), (128, 40), (256, 6)])
def test_outputs_follow_the_last_products(sv, d, Hq):
    """Items of a few units, many at a time and again and again: a block's outputs are read when its last products are
    done, however late they come."""
    gen = rng_of(16)
    for n, B in ((200, 40), (500, 50), (300, 50), (2000, 30)):
        need = [(n + 39) // 32] * B
        table, cache = ref.shuffled(gen, need), ref.filled(gen, sum(need), 1, d)
        q = randn(gen, B, 8, Hq, d).bfloat16()
        lens = ints([n] * B)
        want = ref.attention(q, cache, table, lens)
        first = sv.kv4_attention(q, cache, table, lens)
        ref.check_attention(first, want)
        for _ in range(8):
            assert torch.equal(sv.kv4_attention(q, cache, table, lens), first)
