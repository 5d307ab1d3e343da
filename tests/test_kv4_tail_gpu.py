"""Attention where one token outweighs each of very many others: their weights,
each far below it, count together."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import kv4_reference as ref  # noqa: E402
from test_kv4_gpu import ints, randn, rng_of, sv  # noqa: E402,F401

BELOW = [17.0, 24.5, 25.25, 28.0]               # log2 of the first token's weight over one of the others'


def tail(sv, d, T, G, n, B, spread=0.004, below=BELOW, values=range(1, 8)):  # noqa: F811
    """o of T rows of B sequences of n tokens, the last row's position n - 1, and the same from the definition.

    The first page holds the token that outweighs the others; all later pages of all sequences are one page, so that
    the sums over them have a closed form.  Query head h is below[h % 4] above the others' mean."""
    gen = rng_of(d + T)
    pages = -(-n // 32)
    cache = torch.zeros(2, 1, 36 * d, dtype=torch.uint8, device="cuda")
    kc, vc, ks, vs = ref.pieces(cache)
    for p in (ks, vs):
        p.fill_(0x38)                           # e4m3 1.0
    # keys: dimension 0 tells the first token, dimension 1 makes the others differ a little; values: the first token
    # has zeros in the even dimensions, the others are positive
    kc[..., 0] = torch.randint(0, 16, kc.shape[:-1], device="cuda", generator=gen).to(torch.uint8) << 4
    kc[0, 0, 0, 0] = 6                          # 4.0 and 0
    some = torch.tensor(list(values), dtype=torch.uint8, device="cuda")
    vc[:] = some[torch.randint(0, len(values), vc.shape, device="cuda", generator=gen)] * 17
    vc[0, 0, 0] = 2 << 4
    q = torch.zeros(B, T, G, d, device="cuda")
    q[..., 0] = torch.tensor(below, device="cuda").repeat(-(-G // 4))[:G] / 32
    q[..., 1] = spread * randn(gen, T, G)        # (the same rows in every sequence)
    q = q.bfloat16()
    scale = 8 * math.log(2)                     # 4 * BELOW / 32 * scale = BELOW ln 2
    table = torch.ones(B, pages, dtype=torch.int32, device="cuda")
    table[:, 0] = 0
    o = sv.kv4_attention(q, cache, table, ints([n - T] * B), scale=scale)
    assert sv.last_device_error() == 0

    k, v = (ref.read(c[:, 0], s[:, 0]) for c, s in ((kc, ks), (vc, vs)))        # [2][32][d]
    e = torch.exp(torch.einsum("tgd,pjd->tgpj", q[0].double(), k) * scale)
    seen = torch.arange(n - T, n, device="cuda")[:, None, None] + 1 - 32 - torch.arange(32, device="cuda")
    times = (seen.clamp(min=0) + 31) // 32      # how often a row sees token j of the second page
    w = torch.stack((e[:, :, 0], e[:, :, 1] * times), 2)
    want = torch.einsum("tgpj,pjd->tgd", w / w.sum((-1, -2), keepdim=True), v)
    return o, want


def check(o, want, n):
    """Rounding of the output, 2^-8 of it.  A weight is off by 2^-11 of itself as an fp16 number, by 2^-12 from its
    score; and as fp16 has them to 2^-25 and the largest is 2^7 at least, by 2^-32 of that one, of each of the n
    tokens (values are at most 6).  A product that the tensor cores add to an fp32 sum is aligned to it and may lose
    what is below its last place, 2^-23 of the sum at most, and there are n of them.  All values are positive, so the sum
    of the weighted magnitudes is the output itself."""
    bound = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12 + n * 2.0 ** -23) * want + 2.0 ** -32 * 6 * n
    ratio = (o.double() - want).abs() / bound
    assert float(ratio.max()) <= 1, (float(ratio.max()), ratio.amax((0, 1, 3)).tolist())


INSTANCES = [(d, T, G) for d in (64, 128, 256) for T, G in ((1, 4), (4, 4), (25, 4), (130, 4))]


@pytest.mark.parametrize("d,T,G", INSTANCES)
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("n", [131072, (1 << 20) + 7])
def test_long_tail(sv, d, T, G, many, n):  # noqa: F811
    """One sequence, spread over the GPU, and so many that a block has a whole one, whose weights are all relative to
    the first token's."""
    B = 1 if not many else 800 if T * G <= 16 else 160
    o, want = tail(sv, d, T, G, n, B)
    check(o, want, n)


@pytest.mark.parametrize("d,T,G", INSTANCES)
@pytest.mark.parametrize("scale", [1e4, 3e5, 1e7, -1e8, 1e12])
def test_scores_that_fp32_tells_apart_by_more_than_the_slack(sv, d, T, G, scale):  # noqa: F811
    """Which token wins is then a matter of rounding, but the output lies among the values: off by the roundings of
    `check`, and by fp16's largest number where a weight is up to 2^16 (2^-11)."""
    gen = rng_of(d)
    cache, table = ref.filled(gen, 12, 1, d), ref.shuffled(gen, [12])
    q = (20 * randn(gen, 1, T, G, d)).bfloat16()
    o = sv.kv4_attention(q, cache, table, ints([384 - T]), scale=scale)
    assert sv.last_device_error() == 0
    _, v = ref.tokens(cache, table[0], 384)
    most = v[:, 0].abs().amax(0) * (1 + 2.0 ** -8 + 2 * 2.0 ** -11 + 2.0 ** -12)
    assert bool((o.double().abs() <= most).all())


@pytest.mark.parametrize("d,T,G", INSTANCES)
def test_sums_of_weights(sv, d, T, G):  # noqa: F811
    """The others at 2^-25 of the first token, each, their values 1 and 2: a sum of products of an even dimension is a
    multiple of 2^-18 below 2^24 of them, and exact.  What is left is the output's rounding, 2^-8; the
    score's, 2^-12; and the sum of the weights, each addition off by 2^-24 of the total: a unit's 64 weights at most and
    n / 64 units in kv4_attn_tc_kernel, a thread's n / 32 weights in kv4_attn_kernel."""
    n = 1 << 22
    o, want = tail(sv, d, T, G, n, 800 if T * G <= 16 else 160, 0.0, [25.0] * 4, [2, 4])
    err = ((o.double() - want) / want)[..., ::2].abs()
    assert float(err.max()) <= 2.0 ** -8 + 2.0 ** -12 + (64 + n // 32) * 2.0 ** -24, float(err.max())
