"""The 4-bit cache and the attention over it from their definitions, in 64
bits, a token and a sequence at a time."""
import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
PAGE = 32


def nearest(x, levels):
    """Numbers of the nearest of the rising levels, of two as near the even one."""
    hi = torch.searchsorted(levels, x.contiguous()).clamp(1, len(levels) - 1)
    a, b = x - levels[hi - 1], levels[hi] - x
    return torch.where((a < b) | ((a == b) & (hi % 2 == 1)), hi - 1, hi)


def quantise(x, g):
    """(codes, scales) of rows x [..., d]: numbers 0 .. 15 [..., d] and e4m3 bytes [..., d / 16]."""
    x = x.double().unflatten(-1, (-1, 16))
    fp8 = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
    fp4 = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    bad = ~x.isfinite().all(-1)
    scale = nearest(torch.where(bad, 0, x.abs().amax(-1)) / (6 * g), fp8)
    s = (fp8[scale] * g)[..., None]
    codes = nearest(torch.where(s > 0, x.abs() / s, 0).nan_to_num(0, 0, 0), fp4) + 8 * torch.signbit(x)
    codes = torch.where((s > 0) & ~bad[..., None], codes, 0)
    return codes.flatten(-2), torch.where(bad, 0x7F, scale).to(torch.uint8)


def pieces(cache):
    """K codes, V codes, K scales, V scales: views [pages][Hk][32][...] of the bytes."""
    d = cache.shape[-1] // 36
    return [cache[..., a * d:b * d].unflatten(-1, (PAGE, -1)) for a, b in ((0, 16), (16, 32), (32, 34), (34, 36))]


def read(codes, scales):
    """64-bit values of codes [..., d / 2] and scales [..., d / 16] bytes."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    level = torch.tensor(E2M1, dtype=torch.float64, device=codes.device)
    x = torch.cat((level, -level))[n]
    return x * scales.contiguous().view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)


def tokens(cache, row, n, g=(1.0, 1.0)):
    """(k, v) [n][Hk][d] of the first n tokens of the sequence with that row of the page table."""
    used = cache[row[:-(-n // PAGE)].long()].transpose(0, 1)                    # [Hk][pages][36 d]
    kc, vc, ks, vs = (p.flatten(1, 2)[:, :n].transpose(0, 1) for p in pieces(used))
    return read(kc, ks) * g[0], read(vc, vs) * g[1]


def attention(q, cache, table, lens, cu=None, scale=None, window=0, sinks=0, g=(1.0, 1.0)):
    """(o, sum of p |v|, largest |v| times the tokens): 64 bits, of q's shape; NaN for rows of no sequence."""
    B = len(lens)
    flat = q.flatten(0, -3).double()
    T = 0 if cu is not None else q.shape[1]
    cu = [b * T for b in range(B + 1)] if cu is None else cu.tolist()
    Hk, d = cache.shape[1], cache.shape[2] // 36
    G = flat.shape[1] // Hk
    scale = d ** -0.5 if scale is None else scale
    out = [torch.full_like(flat, float("nan")) for _ in range(3)]
    for b, before in enumerate(lens.tolist()):
        first, n = cu[b], cu[b + 1] - cu[b]
        if not n:
            continue
        if before < 0:
            for o in out:
                o[first:first + n] = 0
            continue
        k, v = tokens(cache, table[b], before + n, g)
        p, j = torch.arange(before, before + n, device=q.device)[:, None], torch.arange(before + n, device=q.device)
        seen = j <= p
        if window:
            seen &= (p - j < window) | (j < sinks)
        for h in range(Hk):
            x = flat[first:first + n, h * G:(h + 1) * G]
            s = torch.einsum("tgd,jd->gtj", x, k[:, h]) * scale
            w = torch.softmax(torch.where(seen, s, -torch.inf), -1)
            vh = torch.where(seen.any(0)[:, None], v[:, h], 0)
            at = (slice(first, first + n), slice(h * G, (h + 1) * G))
            out[0][at] = torch.einsum("gtj,jd->tgd", w, vh)
            out[1][at] = torch.einsum("gtj,jd->tgd", w, vh.abs())
            out[2][at] = vh.abs().max() * (before + n)
    return [o.view(q.shape) for o in out]


def check_attention(o, ref):
    """Rounding of the output, 2^-8 of it; of the probabilities, 2^-11 of each (fp16) or 2^-25 of the largest where
    fp16 has no more bits; fp32 scores of up to a few hundred, 2^-12 of each probability at most."""
    want, mass, most = ref
    bound = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -12) * mass + 2.0 ** -25 * most + 1e-30
    err = (o.double() - want).abs()
    ok = want.isnan() | (err <= bound)
    assert bool(ok.all()), (float((err / bound).nan_to_num().max()), int((~ok).sum()), (~ok).nonzero()[:3].tolist())


def filled(gen, n_pages, Hk, d, g=1.0):
    """A cache of normal keys and values, codes and scales as appending them gives."""
    cache = torch.zeros(n_pages, Hk, 36 * d, dtype=torch.uint8, device="cuda")
    x = [torch.randn(n_pages, Hk, PAGE, d, device="cuda", generator=gen).bfloat16() for _ in range(2)]
    got = [quantise(t, g) for t in x]
    for view, (codes, _) in zip(pieces(cache)[:2], got):
        view.copy_(codes[..., ::2] + 16 * codes[..., 1::2])
    for view, (_, scales) in zip(pieces(cache)[2:], got):
        view.copy_(scales)
    return cache


def shuffled(gen, need, n_pages=None, slack=2):
    """Page table [B][most + slack] of shuffled pages, -1 behind each sequence's."""
    order = torch.randperm(n_pages or sum(need), device="cuda", generator=gen).to(torch.int32)
    table = torch.full((len(need), max(need + [0]) + slack), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table
