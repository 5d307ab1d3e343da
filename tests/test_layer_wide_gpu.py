"""The gated feed-forward at widths that take the tcgen05 kernel -- tiles that
do not divide the result, an odd number of 128-column groups, two rounds of
tiles -- steps of as many heads as give a multiprocessor two or three blocks,
and rows with a NaN among a step's rows."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import gen

U = 2.0 ** -8                           # bf16: half a unit is 2^-9 of the value; the sums' error may cross a rounding point


@pytest.fixture(scope="module")
def sv():
    import speculative_verify_gb300 as m
    m.load()
    return m


def dense64(W, s):
    """(levels * scales, their magnitudes) in 64 bits, on the device."""
    shifts = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    lv = ((W[:, :, None] >> shifts) & 15).flatten(1).double() - 8
    return lv * s.double().repeat_interleave(128, dim=1)


def act64(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    return 0.5 * g * (1 + torch.tanh((2 / np.pi) ** 0.5 * (g + 0.044715 * g ** 3)))


@pytest.fixture(scope="module")
def layers():
    """Weights by (K, F), drawn once."""
    made = {}

    def get(K, F):
        if (K, F) not in made:
            made.clear()
            g = torch.Generator(device="cuda")
            g.manual_seed(K + F)
            W = torch.randint(-2 ** 31, 2 ** 31, (2 * F, K // 8), device="cuda", generator=g, dtype=torch.int64).to(torch.int32)
            s = (0.005 + 0.015 * torch.rand(2 * F, K // 128, device="cuda", generator=g)).bfloat16()
            made[K, F] = W, s, dense64(W, s)
        return made[K, F]

    return get


@pytest.mark.parametrize("K,F,T", [(K, F, T) for K, F in ((1024, 19456), (2048, 14001), (1920, 19455), (1152, 38000))
                                   for T in (1, 8, 9, 16, 17, 31, 32)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gate_up_wide(sv, layers, K, F, T, act):
    """The sums' bound: fp32 rounding of K products is below 1e-6 of the magnitudes added (2^-24 times a tree of
    at most 17 levels); a gate error moves act by at most 1.13 times itself."""
    W, s, w = layers(K, F)
    x = (0.3 * torch.randn(T, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(T))).bfloat16()
    h = torch.full((T + 1, F), 7.0, device="cuda").bfloat16()
    sv.w4a16_gate_up(x, W, s, act=act, h=h[:T])
    y, mag = x.double() @ w.T, x.double().abs() @ w.abs().T
    gt, up, eg, eu = y[:, :F], y[:, F:], 1e-6 * mag[:, :F], 1e-6 * mag[:, F:]
    ref = act64(gt, act) * up
    tol = U * ref.abs() + 1.13 * eg * up.abs() + (gt.abs() + eg) * eu + 2e-6 * ref.abs() + 1e-30
    err = (h[:T].double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    assert bool((h[T] == 7).all())              # nothing past the last token
    assert sv.last_device_error() == 0


@pytest.mark.parametrize("T", [3, 8, 16, 32])
def test_gate_up_wide_nan_stays_in_its_row(sv, layers, T):
    W, s, _ = layers(2048, 14001)
    x = torch.randn(T, 2048, device="cuda").bfloat16()
    want = sv.w4a16_gate_up(x, W, s)
    x[1, 77] = float("nan")
    x[2, 5] = float("inf")
    h = sv.w4a16_gate_up(x, W, s)
    keep = [t for t in range(T) if t not in (1, 2)]
    assert torch.equal(h[keep], want[keep]) and bool(h[1].isnan().all())
    assert not bool(torch.isfinite(h[2]).any())


@pytest.mark.parametrize("Hk,Hv", [(2, 4), (16, 96)])
@pytest.mark.parametrize("T,P,bad", [(2, 0, 1), (4, 0, 2), (8, 8, 3), (12, 0, 11), (9, 9, 1), (20, 4, 13), (32, 32, 30)])
def test_step_nan_stays_with_later_rows(sv, T, P, bad, Hk, Hv):
    """A draft with a NaN in its key, query, value or gates changes no earlier row's output, no other sequence, and
    not the state, which holds the rows before the drafts."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    B, d = 2, 128

    def rows(n):
        r = lambda *a: torch.randn(B, n, *a, device="cuda", generator=g)                   # noqa: E731
        return [r(Hk, d).bfloat16(), r(Hk, d).bfloat16(), r(Hv, d).bfloat16(), -r(Hv).abs(), torch.sigmoid(r(Hv))]

    new, old = rows(T), rows(P)
    prev = tuple(old[1:]) if P else None
    acc = torch.tensor([P // 2, P - 1], dtype=torch.int32, device="cuda") if P else None
    start = torch.randn(B, Hv, d, d, device="cuda", generator=g)
    want_s = start.clone()
    want = sv.gated_delta_step(*new, want_s, prev=prev, accept_len=acc, commit=False, l2norm=True)
    for which in range(5):
        hurt = [t.clone() for t in new]
        hurt[which][0, bad] = float("nan")
        got_s = start.clone()
        got = sv.gated_delta_step(*hurt, got_s, prev=prev, accept_len=acc, commit=False, l2norm=True)
        assert torch.equal(got[0, :bad], want[0, :bad]) and torch.equal(got[1], want[1])
        assert bool(got[0, bad].isnan().all())
        assert torch.equal(got_s, want_s)
    if P:                                       # a rejected draft's NaN goes nowhere
        hurt = [t.clone() for t in old[1:]]
        for t in hurt:
            t[0, P // 2 + 1:] = float("nan")
        got_s = start.clone()
        got = sv.gated_delta_step(*new, got_s, prev=tuple(hurt), accept_len=acc, commit=False, l2norm=True)
        assert torch.equal(got, want) and torch.equal(got_s, want_s)


def rule64(S, q, k, v, gate, beta, scale):
    """The recurrence on rows [B][n][heads][d] with S [B][Hv][dv][dk], keys and queries normalised; (o, S)."""
    rep, out = v.shape[2] // k.shape[2], []
    for t in range(k.shape[1]):
        kt, qt = (a[:, t].double() for a in (k, q))
        kt, qt = ((a / torch.sqrt((a * a).sum(-1, keepdim=True) + 1e-6)).repeat_interleave(rep, 1) for a in (kt, qt))
        S = S * torch.exp(gate[:, t].double())[..., None, None]
        u = beta[:, t].double()[..., None] * (v[:, t].double() - torch.einsum("bhvk,bhk->bhv", S, kt))
        S = S + u[..., None] * kt[:, :, None, :]
        out.append(scale * torch.einsum("bhvk,bhk->bhv", S, qt))
    return torch.stack(out, 1) if out else None, S


@pytest.mark.parametrize("Hk,Hv,dk,dv,B", [(16, 48, 128, 128, 4), (32, 96, 64, 64, 3), (16, 48, 128, 64, 5),
                                           (8, 40, 64, 128, 4)])
@pytest.mark.parametrize("T,P", [(3, 0), (5, 0), (4, 4), (8, 8), (8, 5), (1, 7), (0, 6)])
@pytest.mark.parametrize("commit", [False, True])
def test_step_of_many_heads(sv, Hk, Hv, dk, dv, B, T, P, commit):
    """The state to 2e-6 of a head's norm (22-bit factors; fp32 sums of at most 17 terms), outputs to bf16's
    rounding and 1e-5 of the head's rms."""
    g = torch.Generator(device="cuda")
    g.manual_seed(Hk + Hv + dk + dv + 31 * T + P)

    def rows(n):
        r = lambda *a: torch.randn(B, n, *a, device="cuda", generator=g)                   # noqa: E731
        return [r(Hk, dk).bfloat16(), r(Hk, dk).bfloat16(), r(Hv, dv).bfloat16(), -r(Hv).abs(), torch.sigmoid(r(Hv))]

    new, old = rows(T), rows(P)
    state = torch.randn(B, Hv, dv, dk, device="cuda", generator=g)
    acc = torch.tensor([(3 * b + 1) % (P + 2) - 1 for b in range(B)], dtype=torch.int32, device="cuda") if P else None
    got = state.clone()
    o = sv.gated_delta_step(*new, got, prev=tuple(old[1:]) if P else None, accept_len=acc, commit=commit, l2norm=True)
    scale = dk ** -0.5
    for b in range(B):
        S = state[b:b + 1].double()
        n = min(max(int(acc[b]) + 1, 0), P) if P else 0
        if n:
            _, S = rule64(S, *(t[b:b + 1, :n] for t in old), scale)
        ref, after = rule64(S, *(t[b:b + 1] for t in new), scale)
        want = (after if commit else S)[0].flatten(1)
        err = (got[b].double().flatten(1) - want).norm(dim=1)
        assert bool((err <= 2e-6 * want.norm(dim=1)).all()), float((err / want.norm(dim=1)).max())
        if T:
            rms = (ref ** 2).mean((1, 3), keepdim=True).sqrt()
            bad = (o[b:b + 1].double() - ref).abs() - (U * ref.abs() + 1e-5 * rms)
            assert bool((bad <= 0).all()), float(bad.max())
    assert sv.last_device_error() == 0
