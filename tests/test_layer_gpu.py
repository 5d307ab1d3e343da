"""The operators between a layer's weight reads against their definitions in
64 bits: residual norm, gated delta rule (decode, verify and prompt rows) and
gated feed-forward.

Tolerances (derived from the formats, not from runs):
  * a bf16 output carries half a unit in the last place, at most 2^-8 of its
    value, on top of the fp32 arithmetic before it (1e-5 of the magnitudes
    that are added);
  * e4m3 carries 2^-4 of the value or 2^-10 of the scale;
  * an fp32 state: 2e-5 of its norm -- the class of fp32 products whose
    operands keep 16 or more bits;
  * prompt outputs may also round an operand of their products to bf16, 2^-9
    relative and independent, so that a value is off by a few times 2^-9 of
    its head's spread: 2^-7 of the rms is over five standard deviations.
"""
import numpy as np
import pytest

import gen

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -8


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


# --------------------------------------------------------------------- norm


def norm64(s, w, eps, off):
    f = s.double()
    return f / torch.sqrt((f * f).mean(-1, keepdim=True) + eps) * (w.double() + off)


def check_bf16(y, ref):
    err = (y.double() - ref).abs()
    assert bool((err <= (U + 1e-5) * ref.abs() + 1e-38).all()), float((err / ref.abs().clamp_min(1e-30)).max())


def strided(t, pad, off=0):
    """The values of t in rows `pad` elements further apart, `off` elements into their buffer."""
    T, D = t.shape
    buf = torch.zeros(T * (D + pad) + off + 8, dtype=t.dtype, device=t.device)
    v = buf[off:off + T * (D + pad)].view(T, D + pad)[:, :D]
    v.copy_(t)
    return v


@pytest.mark.parametrize("T", [1, 3, 33])
@pytest.mark.parametrize("D", [1, 7, 8, 127, 128, 129, 1000, 5120, 5121, 17408, 17411])
@pytest.mark.parametrize("residual,off", [(False, 0), (True, 1)])
def test_rmsnorm(sv, T, D, residual, off):
    g = rng_of(T * 100003 + D)
    x, w = randn(g, T, D).bfloat16(), randn(g, D).bfloat16()
    r = (3 * randn(g, T, D)).bfloat16() if residual else None
    y, s = sv.rmsnorm(x, w, r, unit_offset=bool(off))
    ref = (x.float() + r.float()).bfloat16() if residual else x
    if residual:
        assert torch.equal(s, ref)
    else:
        assert s is None
    check_bf16(y, norm64(ref, w, 1e-6, off))


@pytest.mark.parametrize("D,pad,off", [(256, 8, 0), (256, 8, 8), (256, 3, 0), (256, 0, 1), (250, 6, 2), (65536, 0, 0),
                                       (65535, 1, 0), (40000, 0, 0)])
def test_rmsnorm_strides_and_alignment(sv, D, pad, off):
    g = rng_of(D + pad + off)
    T = 5
    x, r = strided(randn(g, T, D).bfloat16(), pad, off), strided(randn(g, T, D).bfloat16(), pad, off)
    w = randn(g, D).bfloat16()
    y = strided(torch.zeros(T, D, device="cuda").bfloat16(), pad, off)
    guard = y._base if y._base is not None else y
    sv.rmsnorm(x, w, r, eps=1e-5, y=y, residual_out=r if pad == 8 else None)
    torch.cuda.synchronize()
    check_bf16(y, norm64((x.float() + r.float()).bfloat16() if pad != 8 else r, w, 1e-5, 0))
    if pad:                                     # nothing is written between the rows
        full = guard.flatten()
        keep = torch.ones_like(full, dtype=torch.bool)
        for t in range(T):
            a = off + t * (D + pad)
            keep[a:a + D] = False
        assert bool((full[keep] == 0).all())


def test_rmsnorm_in_place(sv):
    g = rng_of(3)
    x, r, w = randn(g, 9, 5120).bfloat16(), randn(g, 9, 5120).bfloat16(), randn(g, 5120).bfloat16()
    y0, s0 = sv.rmsnorm(x, w, r)
    x1, r1 = x.clone(), r.clone()
    sv.rmsnorm(x1, w, r1, y=x1, residual_out=r1)
    assert torch.equal(x1, y0) and torch.equal(r1, s0)


@pytest.mark.parametrize("group", [128, 0])
@pytest.mark.parametrize("T,D,pad", [(1, 5120, 0), (32, 5120, 0), (3, 1, 0), (4, 129, 0), (4, 136, 0), (2, 1000, 8),
                                     (3, 777, 5), (2, 17411, 0), (2, 40000, 0)])
def test_rmsnorm_fp8(sv, T, D, pad, group):
    g = rng_of(D + group)
    x, r = strided(randn(g, T, D).bfloat16(), pad), randn(g, T, D).bfloat16()
    w = randn(g, D).bfloat16()
    y, sc, s = sv.rmsnorm_fp8(x, w, r, group=group, unit_offset=True)
    assert torch.equal(s, (x.float() + r.float()).bfloat16())
    ref = norm64(s, w, 1e-6, 1)
    n = group or D
    cols = torch.arange(D, device="cuda") // n
    want = torch.stack([ref[:, cols == i].abs().amax(1) for i in range(sc.shape[1])], 1) / 448
    assert bool(((sc.double() - want).abs() <= 1e-5 * want).all())
    per = sc.double()[:, cols]
    err = (y.float().double() * per - ref).abs()
    assert bool((err <= (2.0 ** -4) * (1 + 1e-4) * ref.abs() + (2.0 ** -10) * (1 + 1e-4) * per).all())


def test_norm_special_rows(sv):
    """A zero row, a row of tiny values, rows with a NaN and an infinity: what the formula gives."""
    D = 256
    x = torch.ones(5, D, device="cuda").bfloat16()
    x[0] = 0
    x[1] = 1e-38
    x[2, 7] = float("nan")
    x[3, 9] = float("inf")
    w = torch.ones(D, device="cuda").bfloat16()
    y, _ = sv.rmsnorm(x, w)
    assert bool((y[0] == 0).all())
    check_bf16(y[1:2], norm64(x[1:2], w, 1e-6, 0))
    assert bool(y[2].isnan().all())
    assert bool(y[3, 9].isnan()) and bool((y[3, :9] == 0).all())
    check_bf16(y[4:], norm64(x[4:], w, 1e-6, 0))
    y8, sc, _ = sv.rmsnorm_fp8(x, w)
    v = y8.float() * sc.repeat_interleave(128, 1)
    assert bool((v[0] == 0).all()) and bool(torch.isfinite(sc[0]).all()) and bool((sc[0] > 0).all())
    assert bool(((v[1] - y[1].float()).abs() <= 2.0 ** -3 * y[1].float().abs() + 2.0 ** -10 * sc[1, 0]).all())
    assert bool(v[2].isnan().all())
    assert bool(sc[3, 0].isnan()) and bool((v[3, 128:] == 0).all())


def test_norm_no_rows_and_refusals(sv):
    w = torch.ones(64, device="cuda").bfloat16()
    e = torch.empty(0, 64, device="cuda").bfloat16()
    y, s = sv.rmsnorm(e, w, e)
    assert y.shape == (0, 64) and s.shape == (0, 64)
    x = torch.ones(2, 64, device="cuda").bfloat16()
    with pytest.raises(TypeError):
        sv.rmsnorm(x.float(), w)
    with pytest.raises(ValueError):
        sv.rmsnorm(x, w[:32])
    with pytest.raises(ValueError):
        sv.rmsnorm(x, w, x[:1])
    with pytest.raises(ValueError):
        sv.rmsnorm_fp8(x, w, group=64)
    with pytest.raises(ValueError):
        sv.rmsnorm(x.t().contiguous().t(), w)
    with pytest.raises(sv.SpecVerifyError):
        sv.rmsnorm(x, w, eps=-1.0)


# --------------------------------------------------------- gated delta rule


def delta_rows(g, lead, Hk, Hv, dk, dv, decay=1.0, fused=True):
    """q, k, v as slices of one projection's output, and the gates."""
    n = int(np.prod(lead))
    x = randn(g, n, 2 * Hk * dk + Hv * dv)
    x = (x * torch.sigmoid(x)).bfloat16()
    q, k, v = x.split([Hk * dk, Hk * dk, Hv * dv], 1)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    q, k = (t.unflatten(1, (Hk, dk)).unflatten(0, lead) for t in (q, k))
    v = v.unflatten(1, (Hv, dv)).unflatten(0, lead)
    gate = -decay * torch.rand(*lead, Hv, device="cuda", generator=g)
    beta = torch.sigmoid(randn(g, *lead, Hv))
    return q, k, v, gate, beta


def rule64(S, q, k, v, gate, beta, scale, l2norm):
    """The recurrence on rows [n][heads][d] with S [Hv][dv][dk]; (o, S)."""
    rep = v.shape[1] // k.shape[1]
    out = []
    for t in range(k.shape[0]):
        kt, qt = k[t].double(), q[t].double()
        if l2norm:
            kt, qt = (a / torch.sqrt((a * a).sum(-1, keepdim=True) + 1e-6) for a in (kt, qt))
        kt, qt = kt.repeat_interleave(rep, 0), qt.repeat_interleave(rep, 0)
        S = S * torch.exp(gate[t].double())[:, None, None]
        u = beta[t].double()[:, None] * (v[t].double() - torch.einsum("hvk,hk->hv", S, kt))
        S = S + u[:, :, None] * kt[:, None, :]
        out.append(scale * torch.einsum("hvk,hk->hv", S, qt))
    o = torch.stack(out) if out else v.new_zeros(v.shape, dtype=torch.float64)
    return o, S


def check_state(got, ref):
    got, ref = got.double().flatten(1), ref.flatten(1)
    err, norm = (got - ref).norm(dim=1), ref.norm(dim=1)
    assert bool((err <= 2e-5 * norm + 1e-30).all()), float((err / norm.clamp_min(1e-30)).max())


def check_out(o, ref, spread):
    """o, ref [n][Hv][dv]; spread: the allowance in the head's rms."""
    if not ref.numel():
        return
    rms = (ref ** 2).mean((0, 2), keepdim=True).sqrt()
    err = (o.double() - ref).abs()
    assert bool((err <= U * ref.abs() + spread * rms + 1e-30).all()), float((err / rms.clamp_min(1e-30)).max())


SHAPES = [(2, 6, 128, 128), (1, 1, 64, 64), (3, 3, 128, 64), (2, 8, 64, 128)]


@pytest.mark.parametrize("Hk,Hv,dk,dv", SHAPES)
@pytest.mark.parametrize("B,T,P", [(1, 1, 0), (3, 4, 0), (2, 1, 5), (4, 8, 8), (3, 32, 32), (2, 0, 4)])
@pytest.mark.parametrize("l2norm", [True, False])
def test_step_follows_the_recurrence(sv, Hk, Hv, dk, dv, B, T, P, l2norm):
    g = rng_of(B * 1000 + T * 37 + P + dk)
    rows, prev = delta_rows(g, (B, T), Hk, Hv, dk, dv), delta_rows(g, (B, P), Hk, Hv, dk, dv)[1:]
    if not l2norm:                              # unnormalised keys need small ones to stay bounded
        rows[0].mul_(0.1), rows[1].mul_(0.1), prev[0].mul_(0.1)
    state = randn(g, B + 2, Hv, dv, dk)
    idx = torch.randperm(B + 2, device="cuda", generator=g)[:B].to(torch.int32)
    accept = torch.tensor([-1, 0, P - 1, P + 3][:B], dtype=torch.int32, device="cuda")
    for commit in (False, True):
        got = state.clone()
        o = sv.gated_delta_step(*rows, got, state_idx=idx, prev=prev if P else None,
                                accept_len=accept if P else None, commit=commit, l2norm=l2norm)
        want = state.double()
        for b in range(B):
            S = want[int(idx[b])]
            if P:
                n = min(P, max(0, int(accept[b]) + 1))
                k, v, gt, be = (t[b][:n] for t in prev)
                S = kept = rule64(S, k, k, v, gt, be, 1.0, l2norm)[1]
            ref, S = rule64(S, *(t[b] for t in rows), dk ** -0.5, l2norm)
            check_out(o[b], ref, 1e-5)
            if commit:
                want[int(idx[b])] = S
            elif P:
                want[int(idx[b])] = kept
        for s in range(B + 2):
            check_state(got[s], want[s])
        untouched = [s for s in range(B + 2) if s not in idx.tolist()]
        assert torch.equal(got[untouched], state[untouched])
    assert sv.last_device_error() == 0


@pytest.mark.parametrize("gate", [0.0, -1e-4, -5.0, -60.0, float("-inf"), 0.2])
def test_step_decays(sv, gate):
    """Decays from none to a wiped state; the running product is left where it would over- or underflow."""
    g = rng_of(17)
    B, T, Hk, Hv, d = 2, 12, 1, 2, 128
    q, k, v, gt, beta = delta_rows(g, (B, T), Hk, Hv, d, d)
    gt = torch.full_like(gt, gate)
    gt[0, 5] = -0.5
    state = randn(g, B, Hv, d, d)
    got = state.clone()
    o = sv.gated_delta_step(q, k, v, gt, beta, got, l2norm=True)
    for b in range(B):
        ref, S = rule64(state[b].double(), q[b], k[b], v[b], gt[b], beta[b], d ** -0.5, True)
        check_out(o[b], ref, 1e-5)
        check_state(got[b], S)


def test_step_beta_extremes(sv):
    """beta = 0 leaves the decayed state, beta = 1 with one key stores its value exactly in place."""
    d = 64
    k = torch.zeros(1, 2, 1, d, device="cuda").bfloat16()
    k[..., 3] = 1
    v = torch.arange(2 * d, device="cuda").float().view(1, 2, 1, d).bfloat16()
    zero = torch.zeros(1, 2, 1, device="cuda")
    state = randn(rng_of(1), 1, 1, d, d)
    got = state.clone()
    sv.gated_delta_step(k, k, v, zero, zero, got)
    assert torch.equal(got, state)
    o = sv.gated_delta_step(k, k, v, zero, zero + 1, got, scale=1.0)
    # S - S k k^T + v k^T to fp32 rounding
    assert bool(((got[0, 0, :, 3] - v[0, 1, 0].float()).abs() <= 1e-5 * (1 + v[0, 1, 0].float().abs())).all())
    assert torch.equal(got[0, 0, :, :3], state[0, 0, :, :3])
    check_out(o[0], v[0].double(), 1e-5)


def test_verify_and_replay_is_decode(sv):
    """Cycles of provisional rows, replayed by their accepted prefix, leave the state of decoding those rows one by one."""
    g = rng_of(99)
    B, T, Hk, Hv, d, cycles = 3, 5, 2, 4, 128, 4
    state = randn(g, B, Hv, d, d)
    a, b = state.clone(), state.clone()
    prev = accept = None
    for c in range(cycles):
        rows = delta_rows(g, (B, T), Hk, Hv, d, d)
        new_accept = torch.randint(-1, T, (B,), device="cuda", generator=g).to(torch.int32)
        o = sv.gated_delta_step(*rows, a, prev=prev, accept_len=accept, commit=False, l2norm=True)
        for s in range(B):
            for t in range(int(new_accept[s]) + 1):
                one = [x[s:s + 1, t:t + 1] for x in rows]
                od = sv.gated_delta_step(*one, b, state_idx=torch.tensor([s], dtype=torch.int32, device="cuda"),
                                         l2norm=True)
                check_out(o[s, t:t + 1], od[0].double(), 2 * U + 1e-5)
        prev, accept = rows[1:], new_accept
    empty = [x[:, :0] for x in rows]
    sv.gated_delta_step(*empty, a, prev=prev, accept_len=accept, commit=False, l2norm=True)
    check_state(a.flatten(0, 1), b.double().flatten(0, 1))


def test_step_slots(sv):
    """A negative slot is inactive; one past the pool is skipped and reported."""
    g = rng_of(5)
    rows = delta_rows(g, (3, 2), 1, 2, 64, 64)
    state = randn(g, 2, 2, 64, 64)
    got = state.clone()
    idx = torch.tensor([-1, 1, -7], dtype=torch.int32, device="cuda")
    o = sv.gated_delta_step(*rows, got, state_idx=idx, l2norm=True)
    assert bool((o[0] == 0).all()) and bool((o[2] == 0).all()) and torch.equal(got[0], state[0])
    assert not torch.equal(got[1], state[1])
    assert sv.last_device_error() == 0
    idx[0] = 2
    o = sv.gated_delta_step(*rows, got, state_idx=idx, l2norm=True)
    assert bool((o[0] == 0).all()) and torch.equal(got[0], state[0])
    assert sv.last_device_error() == sv.DEVERR_BAD_SLOT
    assert sv.last_device_error() == 0


def test_step_refusals(sv):
    g = rng_of(6)
    q, k, v, gt, be = delta_rows(g, (2, 3), 2, 4, 64, 64)
    state = randn(g, 2, 4, 64, 64)
    with pytest.raises(ValueError):
        sv.gated_delta_step(q, k, v[:, :2], gt, be, state)
    with pytest.raises(ValueError):
        sv.gated_delta_step(q, k, v, gt, be, state[:, :, :, :32].contiguous())
    with pytest.raises(TypeError):
        sv.gated_delta_step(q.float(), k, v, gt, be, state)
    with pytest.raises(TypeError):
        sv.gated_delta_step(q, k, v, gt.double(), be, state)
    with pytest.raises(ValueError):
        sv.gated_delta_step(q, k, v, gt, be, state, accept_len=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(sv.SpecVerifyError):     # two sequences, one slot in the pool
        sv.gated_delta_step(q, k, v, gt, be, state[:1])
    long = delta_rows(g, (1, 33), 2, 4, 64, 64)
    with pytest.raises(sv.SpecVerifyError):
        sv.gated_delta_step(*long, state)
    wide = delta_rows(g, (1, 1), 1, 1, 32, 64)
    with pytest.raises(sv.SpecVerifyError):
        sv.gated_delta_step(*wide, torch.zeros(1, 1, 64, 32, device="cuda"))


def chunk64(rows, lens, state, idx, zero, scale, l2norm):
    outs, want, at = [], state.double(), 0
    for b, n in enumerate(lens):
        s = int(idx[b])
        S = torch.zeros_like(want[s]) if zero else want[s]
        o, S = rule64(S, *(t[at:at + n] for t in rows), scale, l2norm)
        outs.append(o)
        want[s] = S
        at += n
    return outs, want


def run_chunk(sv, rows, lens, state, idx, zero=False, l2norm=True, **kw):
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32), device="cuda")
    return sv.gated_delta_chunk(*rows, cu, state, state_idx=idx, zero_init=zero, l2norm=l2norm, **kw)


@pytest.mark.parametrize("Hk,Hv,dk,dv", SHAPES)
@pytest.mark.parametrize("lens", [[1], [63], [64], [65], [130], [0, 1, 200, 64, 0, 17], [31, 32, 33, 127, 128, 129]])
@pytest.mark.parametrize("zero,decay", [(False, 1.0), (True, 0.05), (False, 12.0)])
def test_chunk_follows_the_recurrence(sv, Hk, Hv, dk, dv, lens, zero, decay):
    g = rng_of(sum(lens) * 7 + dk + dv + int(decay * 100))
    rows = delta_rows(g, (sum(lens),), Hk, Hv, dk, dv, decay)
    B = len(lens)
    state = randn(g, B + 1, Hv, dv, dk)
    idx = torch.randperm(B + 1, device="cuda", generator=g)[:B].to(torch.int32)
    got = state.clone()
    o = run_chunk(sv, rows, lens, got, idx, zero)
    outs, want = chunk64(rows, lens, state, idx, zero, dk ** -0.5, True)
    for b, part in enumerate(o.split(lens)):
        check_out(part, outs[b], 2.0 ** -7)
    for s in range(B + 1):
        check_state(got[s], want[s])
    assert sv.last_device_error() == 0


@pytest.mark.parametrize("gate", [0.0, -20.0, -300.0, float("-inf"), 0.01])
def test_chunk_decays(sv, gate):
    g = rng_of(23)
    n, Hk, Hv, d = 150, 1, 2, 128
    q, k, v, gt, beta = delta_rows(g, (n,), Hk, Hv, d, d)
    gt = torch.where(torch.rand(n, Hv, device="cuda", generator=g) < 0.3, gate, gt)
    if gate == 0.01:
        gt = torch.full_like(gt, gate)
    state = randn(g, 1, Hv, d, d)
    got = state.clone()
    idx = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = run_chunk(sv, (q, k, v, gt, beta), [n], got, idx)
    outs, want = chunk64((q, k, v, gt, beta), [n], state, idx, False, d ** -0.5, True)
    check_out(o, outs[0], 2.0 ** -7)
    check_state(got[0], want[0])


def test_chunk_equal_keys(sv):
    """One key in every row: the rows' triangular system is as far from the identity as it gets."""
    g = rng_of(29)
    n, d = 192, 128
    q, k, v, gt, beta = delta_rows(g, (n,), 1, 1, d, d, 0.01)
    k = k[:1].expand(n, 1, d).contiguous()
    beta = torch.full_like(beta, 0.97)
    state = randn(g, 1, 1, d, d)
    got = state.clone()
    idx = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = run_chunk(sv, (q, k, v, gt, beta), [n], got, idx)
    outs, want = chunk64((q, k, v, gt, beta), [n], state, idx, False, d ** -0.5, True)
    check_out(o, outs[0], 2.0 ** -7)
    check_state(got[0], want[0])


def test_chunk_magnitudes(sv):
    """Values and states of 2^40 and 2^-40: nothing in between is kept in a format that they leave."""
    g = rng_of(31)
    n, d = 100, 128
    for e in (40, -40):
        q, k, v, gt, beta = delta_rows(g, (n,), 1, 2, d, d)
        v = v * 2.0 ** e
        state = randn(g, 1, 2, d, d) * 2.0 ** e
        got = state.clone()
        idx = torch.zeros(1, dtype=torch.int32, device="cuda")
        o = run_chunk(sv, (q, k, v, gt, beta), [n], got, idx)
        outs, want = chunk64((q, k, v, gt, beta), [n], state, idx, False, d ** -0.5, True)
        check_out(o, outs[0], 2.0 ** -7)
        check_state(got[0], want[0])


def test_chunk_without_normalisation_and_with_scale(sv):
    g = rng_of(37)
    n, d = 140, 64
    q, k, v, gt, beta = delta_rows(g, (n,), 2, 2, d, d, fused=False)
    k = (k.float() / k.float().norm(dim=-1, keepdim=True)).bfloat16()
    state = randn(g, 1, 2, d, d)
    got = state.clone()
    idx = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = run_chunk(sv, (q, k, v, gt, beta), [n], got, idx, l2norm=False, scale=0.3)
    outs, want = chunk64((q, k, v, gt, beta), [n], state, idx, False, 0.3, False)
    check_out(o, outs[0], 2.0 ** -7)
    check_state(got[0], want[0])


def test_chunk_continues_and_meets_step(sv):
    """A prompt in two calls gives the state of one call, and decode goes on from it."""
    g = rng_of(41)
    n, cut, d = 333, 150, 128
    rows = delta_rows(g, (n,), 1, 2, d, d)
    idx = torch.zeros(1, dtype=torch.int32, device="cuda")
    one, two = torch.zeros(1, 2, d, d, device="cuda"), torch.zeros(1, 2, d, d, device="cuda")
    run_chunk(sv, rows, [n], one, idx, zero=True)
    run_chunk(sv, [t[:cut] for t in rows], [cut], two, idx, zero=True)
    run_chunk(sv, [t[cut:300] for t in rows], [300 - cut], two, idx)
    for a in range(300, n, 32):
        sv.gated_delta_step(*(t[None, a:min(n, a + 32)] for t in rows), two, l2norm=True)
    err = (one - two).double().flatten(1).norm(dim=1)
    assert bool((err <= 4e-5 * one.double().flatten(1).norm(dim=1)).all())


def test_chunk_uncovered_rows_and_slots(sv):
    """Rows of no sequence keep their outputs; inactive and bad slots are skipped; cu_seqlens is kept in range."""
    g = rng_of(43)
    rows = delta_rows(g, (200,), 1, 1, 64, 64)
    state = randn(g, 3, 1, 64, 64)
    got = state.clone()
    o = torch.full((200, 1, 64), 7.0, device="cuda").bfloat16()
    cu = torch.tensor([10, 80, 120, 100, 5000], dtype=torch.int32, device="cuda")
    idx = torch.tensor([0, -1, 2, 9], dtype=torch.int32, device="cuda")
    sv.gated_delta_chunk(*rows, cu, got, state_idx=idx, l2norm=True, o=o)
    assert bool((o[:10] == 7).all()) and bool((o[80:120] == 0).all())
    ref, S = rule64(state[0].double(), *(t[10:80] for t in rows), 64 ** -0.5, True)
    check_out(o[10:80], ref, 2.0 ** -7)
    check_state(got[0], S)
    assert torch.equal(got[1], state[1])
    assert torch.equal(got[2], state[2])        # sequence 2 ends before it begins: empty
    assert bool((o[100:] == 0).all())           # sequence 3 (100 .. 200) has no slot
    assert sv.last_device_error() == sv.DEVERR_BAD_SLOT


def test_chunk_empty(sv):
    state = randn(rng_of(1), 2, 1, 64, 64)
    rows = delta_rows(rng_of(2), (0,), 1, 1, 64, 64)
    got = state.clone()
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert sv.gated_delta_chunk(*rows, cu, got).shape == (0, 1, 64)
    assert torch.equal(got, state)
    sv.gated_delta_chunk(*rows, cu, got, zero_init=True)
    assert bool((got == 0).all())
    sv.gated_delta_chunk(*rows, cu[:1], got)
    with pytest.raises(TypeError):
        sv.gated_delta_chunk(*rows, cu.long(), got)
    with pytest.raises(sv.SpecVerifyError):
        sv.gated_delta_chunk(*rows, cu, got, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------- gated feed-forward


def gate_up64(oracle, x, W, s, T, K, F, act):
    """Sums of the library's own CPU oracle (fp32 group sums), activation and product in 64 bits."""
    y, _ = oracle.w4a16_gemm(x, W, s, T, K, 2 * F)
    y = y.astype(np.float64)
    gt, up = y[:, :F], y[:, F:]
    if act == "silu":
        a = gt / (1 + np.exp(-gt))
    else:
        a = 0.5 * gt * (1 + np.tanh(np.sqrt(2 / np.pi) * (gt + 0.044715 * gt ** 3)))
    return gt, up, a * up


def check_gate_up(h, gt, up, ref, mag):
    """mag [T][2F]: fp32 rounding of a sum of K products is below 1e-6 of the magnitudes added (2^-24 times a
    tree of at most 17 levels); a gate error moves act by at most 1.13 times itself."""
    F = ref.shape[1]
    eg, eu = 1e-6 * mag[:, :F], 1e-6 * mag[:, F:]
    tol = U * np.abs(ref) + 1.13 * eg * np.abs(up) + (np.abs(gt) + eg) * eu + 2e-6 * np.abs(ref) + 1e-30
    err = np.abs(h.float().cpu().numpy().astype(np.float64) - ref)
    assert np.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 31, 32])
@pytest.mark.parametrize("K,F", [(128, 1), (128, 8), (640, 77), (1024, 1300), (2176, 4001)])
def test_gate_up(sv, oracle, T, K, F):
    rng = np.random.default_rng(T * 7919 + K + F)
    W, s = gen.weights(rng, 2 * F, K)
    x = gen.f32_to_bf16_bits(rng.standard_normal((T, K)).astype(np.float32) * 0.3)
    dx, dW = torch.from_numpy(x.view(np.int16)).cuda(), torch.from_numpy(W.view(np.int32)).cuda()
    ds = torch.from_numpy(s.view(np.int16)).cuda()
    levels = np.abs(((W[:, :, None] >> (4 * np.arange(8, dtype=np.uint32))) & 15).astype(np.float64) - 8)
    w = levels.reshape(2 * F, K) * np.repeat(gen.bf16_bits_to_f32(s).astype(np.float64), 128, axis=1)
    mag = np.abs(gen.bf16_bits_to_f32(x).astype(np.float64)) @ w.T
    for act in ("silu", "gelu"):
        h = sv.w4a16_gate_up(dx, dW, ds, act=act)
        gt, up, ref = gate_up64(oracle, x, W, s, T, K, F, act)
        check_gate_up(h, gt, up, ref, mag)
    assert sv.last_device_error() == 0


def test_gate_up_one_hot(sv):
    """One activation of 1 at column k: gate and up are level * scale exactly, for every nibble position."""
    rng = np.random.default_rng(5)
    K, F = 256, 48
    W, s = gen.weights(rng, 2 * F, K)
    lv = ((W[:, :, None] >> (4 * np.arange(8, dtype=np.uint32))) & 15).astype(np.float64).reshape(2 * F, K) - 8
    sc = gen.bf16_bits_to_f32(s).astype(np.float64)
    dW, ds = torch.from_numpy(W.view(np.int32)).cuda(), torch.from_numpy(s.view(np.int16)).cuda()
    for k0 in range(0, K, 32):
        x = torch.zeros(32, K, device="cuda")
        x[torch.arange(32), k0 + torch.arange(32)] = 1000.0     # large: silu(g) = g or 0 where |g| > 40
        h = sv.w4a16_gate_up(x.bfloat16(), dW, ds).float().cpu().numpy().astype(np.float64)
        for t in range(32):
            y = 1000.0 * lv[:, k0 + t] * sc[:, (k0 + t) // 128]
            ref = y[:F] / (1 + np.exp(-y[:F])) * y[F:]
            assert np.all(np.abs(h[t] - ref) <= (U + 1e-5) * np.abs(ref) + 1e-12)


def test_gate_up_large_and_nan(sv):
    """A saturated gate gives 0 or the gate itself, a NaN activation NaNs in its row alone."""
    rng = np.random.default_rng(6)
    K, F = 512, 40
    W, s = gen.weights(rng, 2 * F, K)
    dW, ds = torch.from_numpy(W.view(np.int32)).cuda(), torch.from_numpy(s.view(np.int16)).cuda()
    x = torch.randn(3, K, device="cuda").bfloat16()
    x[0] *= 1e6
    x[1, 7] = float("nan")
    for act in ("silu", "gelu"):
        h = sv.w4a16_gate_up(x, dW, ds, act=act)
        assert bool(torch.isfinite(h[0]).all()) and bool(h[1].isnan().all()) and bool(torch.isfinite(h[2]).all())


def test_gate_up_refusals(sv):
    rng = np.random.default_rng(7)
    W, s = gen.weights(rng, 32, 256)
    dW, ds = torch.from_numpy(W.view(np.int32)).cuda(), torch.from_numpy(s.view(np.int16)).cuda()
    x = torch.ones(2, 256, device="cuda").bfloat16()
    with pytest.raises(ValueError):
        sv.w4a16_gate_up(x, dW, ds, act="relu")
    with pytest.raises(ValueError):
        sv.w4a16_gate_up(x, dW[:31], ds[:31])
    with pytest.raises(ValueError):
        sv.w4a16_gate_up(x[:, :128].contiguous(), dW, ds)
    with pytest.raises(sv.SpecVerifyError):
        sv.w4a16_gate_up(torch.ones(33, 256, device="cuda").bfloat16(), dW, ds)


# ------------------------------------------------- streams and captured graphs


def test_side_stream_and_graph(sv):
    """Every operator on a stream of its own and inside a captured graph, replayed on new inputs."""
    g = rng_of(77)
    rng = np.random.default_rng(77)
    Hk, Hv, d, D, F = 1, 2, 128, 512, 256
    W, s = gen.weights(rng, 2 * F, D)
    dW, ds = torch.from_numpy(W.view(np.int32)).cuda(), torch.from_numpy(s.view(np.int16)).cuda()
    w = randn(g, D).bfloat16()
    x, r = torch.zeros(4, D, device="cuda").bfloat16(), torch.zeros(4, D, device="cuda").bfloat16()
    y, ro, h = torch.empty_like(x), torch.empty_like(x), torch.empty(4, F, device="cuda").bfloat16()
    rows = delta_rows(g, (1, 4), Hk, Hv, d, d)
    state = torch.zeros(1, Hv, d, d, device="cuda")
    o = torch.empty(1, 4, Hv, d, device="cuda").bfloat16()

    def work(stream):
        sv.rmsnorm(x, w, r, y=y, residual_out=ro, stream=stream)
        sv.w4a16_gate_up(y, dW, ds, h=h, stream=stream)
        sv.gated_delta_step(*rows, state, l2norm=True, o=o, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    work(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            work(side)
    torch.cuda.synchronize()
    for _ in range(2):
        x.copy_(randn(g, 4, D))
        r.copy_(randn(g, 4, D))
        state.copy_(randn(g, 1, Hv, d, d))
        before = state.clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        y1, r1 = sv.rmsnorm(x, w, r)
        assert torch.equal(y, y1) and torch.equal(ro, r1)
        assert torch.equal(h, sv.w4a16_gate_up(y1, dW, ds))
        ref, S = rule64(before[0].double(), *(t[0] for t in rows), d ** -0.5, True)
        check_out(o[0], ref, 1e-5)
        check_state(state[0], S)


def test_repeat_calls_are_bit_identical(sv):
    g = rng_of(55)
    lens = [150, 3, 70]
    rows = delta_rows(g, (sum(lens),), 2, 4, 128, 128)
    state = randn(g, 3, 4, 128, 128)
    idx = torch.arange(3, dtype=torch.int32, device="cuda")
    a, b = state.clone(), state.clone()
    oa, ob = run_chunk(sv, rows, lens, a, idx), run_chunk(sv, rows, lens, b, idx)
    assert torch.equal(oa, ob) and torch.equal(a, b)


@pytest.mark.parametrize("lens", [[16], [31], [3, 0, 20, 1], [16, 15, 17], [64, 0, 0], [1] * 40])
@pytest.mark.parametrize("zero", [False, True])
def test_chunk_of_few_rows(sv, lens, zero):
    """Prompts of a few rows in all, one of them inactive."""
    g = rng_of(sum(lens) + len(lens))
    Hk, Hv, d, B = 2, 4, 128, len(lens)
    rows = delta_rows(g, (sum(lens),), Hk, Hv, d, d)
    state = randn(g, B + 2, Hv, d, d)
    idx = torch.randperm(B + 2, device="cuda", generator=g)[:B].to(torch.int32)
    own = idx.clone()                           # (the reference's place for the inactive one's state)
    if B > 2:
        idx[1] = -1
    got = state.clone()
    o = run_chunk(sv, rows, lens, got, idx, zero)
    outs, want = chunk64(rows, lens, state, own, zero, d ** -0.5, True)
    live = [b for b in range(B) if int(idx[b]) >= 0]
    for b, part in enumerate(o.split(lens)):
        if b in live:
            check_out(part, outs[b], 2.0 ** -7)
            check_state(got[int(idx[b])], want[int(idx[b])])
        else:
            assert bool((part == 0).all())
    untouched = [s for s in range(B + 2) if s not in idx.tolist()]
    assert torch.equal(got[untouched], state[untouched])
    assert sv.last_device_error() == 0


@pytest.mark.parametrize("T,D,pad,off", [(300, 5119, 0, 0), (64, 1003, 0, 0), (40, 2049, 0, 3), (33, 9001, 6, 1), (700, 67, 0, 5),
                                         (9, 65519, 0, 0), (5, 40001, 2, 7)])
@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm_unaligned_rows(sv, T, D, pad, off, residual):
    """Rows at every 2-byte offset, the same in all tensors; in place; nothing written between or past them."""
    g = rng_of(T + D + off)
    x, r = strided(randn(g, T, D).bfloat16(), pad, off), strided((2 * randn(g, T, D)).bfloat16(), pad, off)
    w = randn(g, D + 1).bfloat16()[1:]
    y = strided(torch.zeros(T, D, device="cuda").bfloat16(), pad, off)
    want = (x.float() + r.float()).bfloat16() if residual else x.clone()
    sv.rmsnorm(x, w, r if residual else None, y=y, residual_out=r if residual else None)
    if residual:
        assert torch.equal(r, want)
    check_bf16(y, norm64(want, w, 1e-6, 0))
    for t in (y, r):
        full = t._base if t._base is not None else t
        keep = torch.ones_like(full.flatten(), dtype=torch.bool)
        for i in range(T):
            a = off + i * (D + pad)
            keep[a:a + D] = False
        assert bool((full.flatten()[keep] == 0).all())
    assert sv.last_device_error() == 0


@pytest.mark.parametrize("group", [128, 0])
@pytest.mark.parametrize("T,D,pad,off", [(40, 5119, 0, 0), (300, 1003, 0, 0), (64, 9001, 6, 3), (33, 129, 0, 0), (50, 127, 2, 1),
                                         (7, 65519, 0, 0)])
def test_rmsnorm_fp8_unaligned_rows(sv, T, D, pad, off, group):
    """8-bit rows at every offset: groups of 128 columns that straddle the 16-byte pieces."""
    g = rng_of(D + group + T)
    x, r = strided(randn(g, T, D).bfloat16(), pad, off), strided(randn(g, T, D).bfloat16(), pad, off)
    w = randn(g, D).bfloat16()
    y8 = strided(torch.zeros(T, D, device="cuda").to(torch.float8_e4m3fn), pad, off)
    y, sc, s = sv.rmsnorm_fp8(x, w, r, group=group, unit_offset=True, y=y8, residual_out=r)
    ref = norm64(s, w, 1e-6, 1)
    n = group or D
    cols = torch.arange(D, device="cuda") // n
    most = torch.stack([ref[:, cols == i].abs().amax(1) for i in range(sc.shape[1])], 1)
    want = most.clamp_min(448 * 2.0 ** -126) / 448      # (a group of one column may hold a zero alone)
    assert bool(((sc.double() - want).abs() <= 1e-5 * want).all())
    per = sc.double()[:, cols]
    err = (y.float().double() * per - ref).abs()
    assert bool((err <= (2.0 ** -4) * (1 + 1e-4) * ref.abs() + (2.0 ** -10) * (1 + 1e-4) * per).all())
    full = y8._base if y8._base is not None else y8
    keep = torch.ones(full.numel(), dtype=torch.bool, device="cuda")
    for i in range(T):
        a = off + i * (D + pad)
        keep[a:a + D] = False
    assert bool((full.flatten().view(torch.uint8)[keep] == 0).all())
    assert sv.last_device_error() == 0
