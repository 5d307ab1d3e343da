"""Scales of the scores and of the cache on every instance of the attention
kernels: packed rows (tokens times query heads of a key head) choose it."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import kv4_reference as ref  # noqa: E402
from test_kv4_gpu import ints, randn, rng_of, run, sv  # noqa: E402,F401

# (d, rows a sequence, query heads a key head): items of 8 and of 16 packed
# rows, one tile of 128 and two
INSTANCES = [(d, T, G) for d in (64, 128, 256) for T, G in ((2, 3), (8, 2), (60, 2), (250, 2))]


@pytest.mark.parametrize("d,T,G", INSTANCES)
@pytest.mark.parametrize("scale,g", [(0.3, (0.05, 3.7)), (-0.02, (1.0, 1e-3)), (0.0, (1.0, 1.0)), (-0.0, (0.5, 2.0)),
                                     (1e-44, (1e-3, 1.0))])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 5)])
def test_scales(sv, d, T, G, scale, g, window, sinks):  # noqa: F811
    """Of either sign, none (the mean of what a row sees), and one that fp32 has only as zero with the cache's."""
    run(sv, d + T, [0, 100, -1, 700], [T] * 4, 2 * G, 2, d, window, sinks, scale=scale, g=g, peak=1.0)


@pytest.mark.parametrize("d,T,G", INSTANCES)
def test_queries_of_every_magnitude(sv, d, T, G):  # noqa: F811
    """Rows from fp32's smallest to its largest, under scales that keep the scores of the latter in range: a row's own
    factor may be below any fp32 number."""
    gen = rng_of(d + G)
    cache, table = ref.filled(gen, 10, 1, d), ref.shuffled(gen, [10])
    size = torch.tensor([1e-38, 1e-32, 1e-20, 1e-6, 1.0, 1e4], device="cuda")[torch.arange(T, device="cuda") % 6]
    q = (randn(gen, 1, T, G, d) * size[:, None, None]).bfloat16()
    before = ints([310 - T])
    for scale in (1e-4, 1e-12):
        o = sv.kv4_attention(q, cache, table, before, scale=scale)
        ref.check_attention(o, ref.attention(q, cache, table, before, scale=scale))
    q = (q.float() * 1e34).clamp(-3e38, 3e38).bfloat16()
    o = sv.kv4_attention(q, cache, table, before, scale=1e-38)
    ref.check_attention(o, ref.attention(q, cache, table, before, scale=1e-38))
    assert sv.last_device_error() == 0


@pytest.mark.parametrize("d,T,G", INSTANCES)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_maxima_that_move(sv, d, T, G, sign):  # noqa: F811
    """Keys that grow page by page: sums rescaled again and again, rows of a warp by different factors."""
    gen = rng_of(d + T)
    cache, table = ref.filled(gen, 20, 1, d), ref.shuffled(gen, [20])
    ks = ref.pieces(cache)[2]
    for i in range(20):
        ks[table[0, i].long()] = 0x28 + 2 * i
    q = (sign * 3 * randn(gen, 1, T, G, d) * torch.linspace(0.1, 1, T, device="cuda")[:, None, None]).bfloat16()
    before = ints([640 - T])
    for scale in (None, -0.03):
        o = sv.kv4_attention(q, cache, table, before, scale=scale)
        ref.check_attention(o, ref.attention(q, cache, table, before, scale=scale))
    assert sv.last_device_error() == 0
