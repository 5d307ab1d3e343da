"""How the layer operators are called: who owns the tensors of a call, and what
its operands may be.  The definitions' checks are in test_layer_gpu.py."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


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


def delta_rows(g, lead, Hk, Hv, dk, dv):
    q, k = randn(g, *lead, Hk, dk).bfloat16(), randn(g, *lead, Hk, dk).bfloat16()
    v = randn(g, *lead, Hv, dv).bfloat16()
    return q, k, v, -torch.rand(*lead, Hv, device="cuda", generator=g), torch.sigmoid(randn(g, *lead, Hv))


def test_prev_from_an_iterator(sv):
    """prev may be any iterable; tensors that only it owns are held until the launch (an output of the size of
    prev's values would otherwise be given their memory)."""
    g = rng_of(3)
    B, T, Hk, Hv, d = 8, 8, 16, 48, 128
    rows, prev = delta_rows(g, (B, T), Hk, Hv, d, d), delta_rows(g, (B, T), Hk, Hv, d, d)[1:]
    state = randn(g, B, Hv, d, d)
    want = state.clone()
    o = sv.gated_delta_step(*rows, want, prev=prev, commit=False, l2norm=True)
    for it in (lambda: (t.clone() for t in prev), lambda: map(torch.Tensor.clone, prev), lambda: list(prev)):
        got = state.clone()
        torch.cuda.synchronize()
        o2 = sv.gated_delta_step(*rows, got, prev=it(), commit=False, l2norm=True)
        assert torch.equal(o, o2) and torch.equal(want, got)
    with pytest.raises(TypeError):
        sv.gated_delta_step(*rows, got, prev=3, commit=False)
    with pytest.raises(ValueError):
        sv.gated_delta_step(*rows, got, prev=(t for t in prev[:3]), commit=False)


@pytest.mark.parametrize("D", [512, 5120, 5119, 30000])
def test_norm_weight_from_the_kernel_before(sv, D):
    """The weight may be what the kernel just before wrote (here the last row of a long norm's output)."""
    g = rng_of(D)
    T = 4096 if D < 10000 else 512
    x, w = randn(g, 2, D).bfloat16(), randn(g, D).bfloat16()
    y = torch.zeros(T, D, device="cuda").bfloat16()
    for _ in range(8):
        a = randn(g, T, D).bfloat16()
        torch.cuda.synchronize()
        sv.rmsnorm(a, w, y=y)
        got, _ = sv.rmsnorm(x, y[-1])
        got8, sc, _ = sv.rmsnorm_fp8(x, y[-1])
        torch.cuda.synchronize()
        last = y[-1].clone()
        torch.cuda.synchronize()
        assert torch.equal(got, sv.rmsnorm(x, last)[0])
        want8, wsc, _ = sv.rmsnorm_fp8(x, last)
        assert torch.equal(got8.view(torch.uint8), want8.view(torch.uint8)) and torch.equal(sc, wsc)


@pytest.mark.parametrize("T,K,F", [(1, 256, 200), (8, 2048, 640), (17, 256, 77), (32, 2048, 14000)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_negative_gates(sv, T, K, F, act):
    """Gates down to -8, exact in fp32 (one activation of 1): a small output is as exact as a large one.

    The bound is relative: half a bf16 unit, 2^-8; and of the activation's exponential, whose argument (50 at most)
    is rounded a few times, 4 * 50 * 2^-24 < 2e-5."""
    g = rng_of(T + F)
    lv = torch.randint(0, 16, (2 * F, K), device="cuda", generator=g)
    shift = 4 * torch.arange(8, device="cuda")
    W = (lv.view(2 * F, K // 8, 8) << shift).sum(-1)
    W = torch.where(W >= 2 ** 31, W - 2 ** 32, W).to(torch.int32)
    s = (0.5 + 0.5 * torch.rand(2 * F, K // 128, device="cuda", generator=g)).bfloat16()
    at = torch.randint(0, K, (T,), device="cuda", generator=g)
    x = torch.zeros(T, K, device="cuda").bfloat16()
    x[torch.arange(T, device="cuda"), at] = 1
    h = sv.w4a16_gate_up(x, W, s, act=act).double()
    y = ((lv[:, at] - 8).double() * s.double()[:, at // 128]).t()
    gate, up = y[:, :F], y[:, F:]
    z = gate if act == "silu" else 2 * (2 / torch.pi) ** 0.5 * (gate + 0.044715 * gate ** 3)
    ref = gate / (1 + torch.exp(-z)) * up
    err = (h - ref).abs()
    assert bool((err <= (2.0 ** -8 + 2e-5) * ref.abs()).all()), float((err / ref.abs().clamp_min(1e-300)).max())
    assert sv.last_device_error() == 0


def test_chunk_rows_claimed_too_often(sv):
    """cu_seqlens that go back and forth claim the rows many times over: nothing is run, and the error word says so."""
    g = rng_of(8)
    R, B, Hk, Hv, d = 6400, 9, 1, 2, 64
    rows = delta_rows(g, (R,), Hk, Hv, d, d)
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[1::2] = R
    state = randn(g, B, Hv, d, d)
    got, o = state.clone(), torch.full((R, Hv, d), 7.0, device="cuda").bfloat16()
    sv.gated_delta_chunk(*rows, cu, got, l2norm=True, o=o)
    assert sv.last_device_error() == sv.DEVERR_BAD_SEQLENS
    assert torch.equal(got, state) and bool((o == 7).all())
    cu[:2], cu[2:] = torch.tensor([0, R]), R        # once: as always
    sv.gated_delta_chunk(*rows, cu, got, l2norm=True, o=o)
    assert sv.last_device_error() == 0
    assert not torch.equal(got[0], state[0]) and torch.equal(got[1:], state[1:])


def operands(g):
    """{operator: its tensors}, small."""
    q, k, v, gt, be = delta_rows(g, (2, 3), 1, 2, 64, 64)
    state = randn(g, 2, 2, 64, 64)
    cu = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    x, w = randn(g, 4, 256).bfloat16(), randn(g, 256).bfloat16()
    W = torch.randint(-2 ** 31, 2 ** 31, (64, 32), device="cuda", generator=g).to(torch.int32)
    return {"rmsnorm": dict(x=x, weight=w, residual=x.clone()), "rmsnorm_fp8": dict(x=x, weight=w, residual=x.clone()),
            "gated_delta_step": dict(q=q, k=k, v=v, g=gt, beta=be, state=state, prev=(k, v, gt, be)),
            "gated_delta_chunk": dict(q=q.flatten(0, 1), k=k.flatten(0, 1), v=v.flatten(0, 1), g=gt.flatten(0, 1),
                                      beta=be.flatten(0, 1), cu_seqlens=cu, state=state),
            "w4a16_gate_up": dict(x=x, Wq=W, scales=randn(g, 64, 2).bfloat16())}


@pytest.mark.parametrize("op", ["rmsnorm", "rmsnorm_fp8", "gated_delta_step", "gated_delta_chunk", "w4a16_gate_up"])
def test_no_gradient_is_lost(sv, op):
    """A tensor that requires a gradient is refused, unless gradients are off."""
    args = operands(rng_of(4))[op]
    call = getattr(sv, op)
    call(**args)
    for name, t in args.items():
        if name == "prev":
            wants = tuple(a.detach().requires_grad_() for a in t)
        elif t.is_floating_point():
            wants = t.detach().requires_grad_()
        else:
            continue
        with pytest.raises(RuntimeError, match="gradient"):
            call(**dict(args, **{name: wants}))
        with torch.no_grad():
            call(**dict(args, **{name: wants}))
