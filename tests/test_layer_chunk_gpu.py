"""Gated delta prompts closer than test_layer_gpu.py looks: outputs as exact as
their rounding allows, rows beside a prompt that hold anything, many value
heads per key head, long ragged prompts.

Tolerances (from the formats): a bf16 output carries half a unit, 2^-8 of its
value, and the products' operands 16 bits, errors of 2^-17 each: a handful of
products in a row and a sum over independent errors stay below 1e-4 of the
head's rms (six times 2^-16).  The state: 2e-5 of its norm, as there.
"""
import numpy as np
import pytest

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


def prompt_rows(g, n, Hk, Hv, dk, dv, decay):
    """q, k, v as slices of one projection's output after its activation, and the gates."""
    x = randn(g, n, 2 * Hk * dk + Hv * dv)
    x = (x * torch.sigmoid(x)).bfloat16()
    q, k, v = x.split([Hk * dk, Hk * dk, Hv * dv], 1)
    return [q.unflatten(1, (Hk, dk)), k.unflatten(1, (Hk, dk)), v.unflatten(1, (Hv, dv)),
            -decay * torch.rand(n, Hv, device="cuda", generator=g), torch.sigmoid(randn(g, n, Hv))]


def rule64(S, q, k, v, gate, beta):
    """The recurrence with normalised keys and queries in 64 bits, all rows of [n][heads][d]; (o, S)."""
    rep, scale = v.shape[1] // k.shape[1], k.shape[2] ** -0.5
    q, k = (t.double() / torch.sqrt((t.double() ** 2).sum(-1, keepdim=True) + 1e-6) for t in (q, k))
    q, k = q.repeat_interleave(rep, 1)[..., None], k.repeat_interleave(rep, 1)[..., None]
    v, decay, beta = v.double()[..., None], torch.exp(gate.double())[..., None, None], beta.double()[..., None, None]
    out = torch.empty(v.shape[:3], dtype=torch.float64, device=v.device)
    for t in range(v.shape[0]):
        S = S * decay[t]
        S = S + (beta[t] * (v[t] - S @ k[t])) * k[t].transpose(-1, -2)
        out[t] = scale * (S @ q[t])[..., 0]
    return out, S


def check(o, S, ref, ref_S):
    if ref.numel():
        rms = (ref ** 2).mean((0, 2), keepdim=True).sqrt()
        err = (o.double() - ref).abs() - U * ref.abs()
        assert bool((err <= 1e-4 * rms + 1e-30).all()), float((err / rms.clamp_min(1e-30)).max())
    err = (S.double() - ref_S).flatten(1).norm(dim=1)
    norm = ref_S.flatten(1).norm(dim=1)
    assert bool((err <= 2e-5 * norm + 1e-30).all()), float((err / norm.clamp_min(1e-30)).max())


def cu_of(lens, first=0):
    return torch.from_numpy((first + np.concatenate([[0], np.cumsum(lens)])).astype(np.int32)).cuda()


def run(sv, lens, Hk, Hv, dk, dv, decay, seed, change=None):
    g = rng_of(seed)
    rows = prompt_rows(g, sum(lens), Hk, Hv, dk, dv, decay)
    if change:
        change(rows)
    state = randn(g, len(lens), Hv, dv, dk)
    got = state.clone()
    o = sv.gated_delta_chunk(*rows, cu_of(lens), got, l2norm=True)
    at = 0
    for b, n in enumerate(lens):
        ref, S = rule64(state[b].double(), *(t[at:at + n] for t in rows))
        check(o[at:at + n], got[b], ref, S)
        at += n
    assert sv.last_device_error() == 0


@pytest.mark.parametrize("Hk,Hv,dk,dv", [(2, 6, 128, 128), (1, 1, 64, 64), (3, 3, 128, 64), (2, 8, 64, 128)])
@pytest.mark.parametrize("lens", [[65], [130, 0, 1, 64], [200, 333], [64] * 5])
@pytest.mark.parametrize("decay", [0.02, 1.0, 12.0])
def test_outputs_are_exact_to_their_rounding(sv, Hk, Hv, dk, dv, lens, decay):
    run(sv, lens, Hk, Hv, dk, dv, decay, sum(lens) + dk + dv)


@pytest.mark.parametrize("Hk,Hv", [(1, 5), (2, 16), (1, 9)])
def test_many_value_heads_per_key_head(sv, Hk, Hv):
    """The gates of the value heads of a key head are staged four at a time."""
    run(sv, [150, 20], Hk, Hv, 128, 128, 1.0, Hv)


@pytest.mark.parametrize("decay", [0.05, 1.0])
def test_long_ragged_prompts(sv, decay):
    """Chains longer than a CTA's share and shorter, 16 key and 48 value heads."""
    run(sv, [1, 700, 63, 0, 2049, 129], 16, 48, 128, 128, decay, 7)


def test_near_equal_keys(sv):
    """Keys within 5 % of one another: a row's update takes most of the last one's back."""
    def change(rows):
        k = rows[1].float()
        rows[1] = (k[:1] + 0.05 * k).bfloat16()
        rows[4].fill_(0.95)

    run(sv, [300], 1, 2, 128, 128, 0.01, 5, change)


BAD = [float("nan"), float("inf"), -float("inf"), 3e38]


@pytest.mark.parametrize("lens", [[70, 33, 130, 1, 64, 5], [5, 9, 3, 11], [640, 3, 200, 190]])
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("dv", [128, 64])
def test_rows_beside_a_prompt_may_hold_anything(sv, lens, bad, dv):
    """NaNs, infinities and huge values in every other prompt, its state and the rows of no prompt: the others
    come out bit for bit as without them."""
    g = rng_of(sum(lens))
    Hk, Hv, dk, before, after = 2, 4, 128, 7, 90
    R = before + sum(lens) + after
    rows = prompt_rows(g, R, Hk, Hv, dk, dv, 1.0)
    rows = [t.contiguous() for t in rows]
    state = randn(g, len(lens), Hv, dv, dk)
    cu = cu_of(lens, before)
    edges = cu.tolist()
    clean = torch.zeros(R, dtype=torch.bool, device="cuda")
    for b in range(0, len(lens), 2):
        clean[edges[b]:edges[b + 1]] = True
    want = state.clone()
    ref = sv.gated_delta_chunk(*rows, cu, want, l2norm=True)
    for t in rows:
        t[~clean] = bad
    got = state.clone()
    got[1::2] = bad
    o = sv.gated_delta_chunk(*rows, cu, got, l2norm=True)
    assert torch.equal(o[clean], ref[clean]) and torch.equal(got[0::2], want[0::2])
    assert sv.last_device_error() == 0
