"""The operators between the weight reads of a verify cycle, as measured cases.

Four entry points of ``speculative_verify_gb300`` that a hybrid decoder layer
(gated delta rule + gated feed-forward) runs between ``w4a16_gemm`` and
``lmhead_verify``:

  norm     rmsnorm / rmsnorm_fp8   residual addition and root-mean-square norm
  step     gated_delta_step        gated delta rule, decode and verify rows
  chunk    gated_delta_chunk       gated delta rule, whole prompts
  gate_up  w4a16_gate_up           act(x Wg^T) * (x Wu^T) from int4 weights

``run`` computes them in plain 32-bit torch operations where ``own`` is false
and calls the library where it is true.  ``exact`` evaluates the definitions
in 64 bits.  Sizes are those of the repository's workload (hidden 5,120; fused
QKV 10,240 = 2 x 16 key heads of 128 + 48 value heads of 128; fused gate+up
2 x 17,408; up to 32 verify rows, four streams of eight) and generic ones
around them.
"""
import math

import torch

own = False

FP8_MAX = 448.0
L2_EPS = 1e-6
BLOCK = 64          # rows of the plain form's blocks


# --------------------------------------------------------------------------
# cases


def _norm(T, D, residual=True, fp8=False, group=128, unit_offset=False):
    return dict(op="norm", T=T, D=D, residual=residual, fp8=fp8, group=group, unit_offset=unit_offset)


def _step(B, T, prev, commit, Hk=16, Hv=48, dk=128, dv=128, l2norm=True, slots=0):
    return dict(op="step", B=B, T=T, prev=prev, commit=commit, Hk=Hk, Hv=Hv, dk=dk, dv=dv, l2norm=l2norm,
                slots=slots or B)


def _chunk(lens, Hk=16, Hv=48, dk=128, dv=128, l2norm=True, zero_init=False):
    return dict(op="chunk", lens=",".join(str(n) for n in lens), Hk=Hk, Hv=Hv, dk=dk, dv=dv, l2norm=l2norm,
                zero_init=zero_init)


def _gate_up(T, K, F, act="silu"):
    return dict(op="gate_up", T=T, K=K, F=F, act=act)


def listed():
    return [
        # the norm before a projection of single-stream decode: one row
        dict(_norm(1, 5120), name="norm T1 D5120"),
        # four streams of eight verify rows, 8-bit output with a scale per 128 columns
        dict(_norm(32, 5120, fp8=True), name="norm fp8 T32 D5120"),
        # the norm of a long prompt
        dict(_norm(16384, 5120, unit_offset=True), name="norm T16384 D5120"),
        # plain decode of one stream: every row is kept
        dict(_step(1, 1, 0, True), name="step 1x1"),
        # a verify cycle of four streams of eight rows: the accepted rows of the last cycle, then the new ones
        dict(_step(4, 8, 8, False, slots=6), name="step 4x8 replay 8"),
        # a large serving batch with three drafts a stream
        dict(_step(256, 4, 4, False), name="step 256x4 replay 4"),
        # one prompt of an odd length
        dict(_chunk([3847]), name="chunk 1x3847"),
        # prompts of mixed lengths, an empty one and a single token among them
        dict(_chunk([1, 700, 63, 0, 2049, 129, 1500, 64, 311]), name="chunk ragged 9"),
        # four long prompts
        dict(_chunk([8192, 8192, 8192, 8192], zero_init=True), name="chunk 4x8192"),
        # the feed-forward block of single-stream decode
        dict(_gate_up(1, 5120, 17408), name="gate_up T1"),
        # a smaller block with a column count that no tile divides, one verify block of four rows
        dict(_gate_up(4, 1280, 3331, "gelu"), name="gate_up T4 odd"),
        # four streams of eight verify rows
        dict(_gate_up(32, 5120, 17408), name="gate_up T32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "step", "chunk", "gate_up"])
    if op == "norm":
        T, D = _log(rng, 1, 16384), _log(rng, 65, 17408)
        D = rng.choice([D, D - D % 8 or 8, 5120])
        T = max(1, min(T, 16384 * 5120 // D))
        fp8 = rng.random() < 0.5
        return _norm(T, D, residual=rng.random() < 0.8, fp8=fp8, group=rng.choice([128, 0]) if fp8 else 128,
                     unit_offset=rng.random() < 0.5)
    if op == "gate_up":
        K, F = 128 * _log(rng, 1, 40), _log(rng, 65, 17408)
        return _gate_up(rng.choice([1, 2, 3, 4, 5, 8, 11, 16, 17, 24, 32]), K, F, rng.choice(["silu", "silu", "gelu"]))
    Hk, Hv = rng.choice([(16, 48), (16, 32), (16, 16), (4, 12), (2, 8), (1, 3)])
    dk, dv = rng.choice([(128, 128), (128, 128), (128, 64), (64, 64), (64, 128)])
    l2 = rng.random() < 0.7
    if op == "step":
        B, T = _log(rng, 1, 256), rng.choice([1, 2, 3, 4, 5, 8])
        prev = rng.choice([0, T, T, rng.randint(1, 8)])
        return _step(B, T, prev, prev == 0 or rng.random() < 0.2, Hk, Hv, dk, dv, l2, slots=B + rng.randint(0, 3))
    rows, B = _log(rng, 65, 16384), rng.randint(1, 8)
    cuts = sorted(rng.randint(0, rows) for _ in range(B - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [rows])]
    return _chunk(lens, Hk, Hv, dk, dv, l2, zero_init=rng.random() < 0.3)


def _lens(case):
    return [int(n) for n in case["lens"].split(",")]


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * c["D"]
        b = 2 * n + (4 * n if c["residual"] else 0) + 2 * c["D"] + (n if c["fp8"] else 2 * n)
        if c["fp8"]:
            b += 4 * c["T"] * (-(-c["D"] // c["group"]) if c["group"] else 1)
        return {"bytes": b, "flops": 4 * n}
    if c["op"] == "gate_up":
        T, K, F = c["T"], c["K"], c["F"]
        return {"bytes": 2 * F * (K // 2 + K // 128 * 2) + 2 * T * K + 2 * T * F, "flops": 4 * T * K * F}
    Hk, Hv, dk, dv = c["Hk"], c["Hv"], c["dk"], c["dv"]
    state, kv, qo = 4 * Hv * dk * dv, 2 * Hk * dk + 2 * Hv * dv + 8 * Hv, 2 * Hk * dk + 2 * Hv * dv
    if c["op"] == "step":
        B, rows = c["B"], c["T"] + c["prev"]
        writes = 1 if c["prev"] or c["commit"] else 0
        return {"bytes": B * (state * (1 + writes) + rows * kv + c["T"] * qo), "flops": 6 * B * rows * Hv * dk * dv}
    lens = _lens(c)
    R, B = sum(lens), len(lens)
    return {"bytes": R * (kv + qo) + B * state * (1 if c["zero_init"] else 2), "flops": 6 * R * Hv * dk * dv}


# --------------------------------------------------------------------------
# inputs


def _silu(x):
    return x * torch.sigmoid(x)


def _delta_rows(gen, n, c, decay, bias):
    """n rows of the fused QKV projection after its activation, and their gates:
    q, k, v are slices of one [n][2 Hk dk + Hv dv] matrix, as the projection writes it."""
    Hk, Hv, dk, dv = c["Hk"], c["Hv"], c["dk"], c["dv"]
    x = _silu(torch.randn(n, 2 * Hk * dk + Hv * dv, device="cuda", generator=gen))
    if not c["l2norm"]:           # keys and queries that their producer has normalised
        qk = x[:, :2 * Hk * dk].view(n, 2 * Hk, dk)
        qk /= (qk * qk).sum(-1, keepdim=True).add(L2_EPS).sqrt()
    x = x.bfloat16()
    q, k, v = x[:, :Hk * dk], x[:, Hk * dk:2 * Hk * dk], x[:, 2 * Hk * dk:]
    dt = torch.randn(n, Hv, device="cuda", generator=gen) * 0.5 + bias
    g = -decay * torch.log1p(torch.exp(dt))
    beta = torch.sigmoid(torch.randn(n, Hv, device="cuda", generator=gen))
    return q.view(n, Hk, dk), k.view(n, Hk, dk), v.view(n, Hv, dv), g, beta


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rand = lambda *s: torch.rand(*s, device="cuda", generator=gen)                       # noqa: E731
    randn = lambda *s: torch.randn(*s, device="cuda", generator=gen)                     # noqa: E731
    st = {"case": c}
    if c["op"] == "norm":
        T, D = c["T"], c["D"]
        st["x"] = randn(T, D).bfloat16()
        st["residual"] = (4 * randn(T, D)).bfloat16() if c["residual"] else None
        w = 0.3 * randn(D)
        st["weight"] = (w if c["unit_offset"] else w + 1).bfloat16()
        return st
    if c["op"] == "gate_up":
        T, K, F = c["T"], c["K"], c["F"]
        st["x"] = randn(T, K).bfloat16()
        st["Wq"] = torch.randint(-2**31, 2**31, (2 * F, K // 8), dtype=torch.int64, device="cuda",
                                 generator=gen).to(torch.int32)
        # levels of -8..7 at 0.005..0.02 a step; scaled so that the gates' spread is a few units
        st["scales"] = ((0.005 + 0.015 * rand(2 * F, K // 128)) * (512 / K) ** 0.5).bfloat16()
        return st
    Hv, dk, dv = c["Hv"], c["dk"], c["dv"]
    decay = 1 + 15 * rand(Hv)
    dt = torch.exp(rand(Hv) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
    bias = dt + torch.log(-torch.expm1(-dt))            # softplus(bias) = dt
    if c["op"] == "step":
        B, T, P = c["B"], c["T"], c["prev"]
        shape = lambda r, n: [t.view(B, n, *t.shape[1:]) if t.dim() == 2 else                # noqa: E731
                              t.unflatten(0, (B, n)) for t in r]
        st["rows"] = shape(_delta_rows(gen, B * T, c, decay, bias), T)
        st["prev"] = st["accept"] = None
        if P:
            st["prev"] = shape(_delta_rows(gen, B * P, c, decay, bias), P)[1:]
            # accepted drafts of the last cycle, -1 for a stream that starts
            st["accept"] = torch.randint(-1, P, (B,), device="cuda", generator=gen).to(torch.int32)
        st["idx"] = torch.randperm(c["slots"], device="cuda", generator=gen)[:B].to(torch.int32)
        st["state"] = 0.1 * randn(c["slots"], Hv, dv, dk)
        return st
    lens = _lens(c)
    st["rows"] = _delta_rows(gen, sum(lens), c, decay, bias)
    ends = torch.tensor(lens).cumsum(0)
    st["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64), ends]).to(torch.int32).cuda()
    st["state"] = 0.1 * randn(len(lens), Hv, dv, dk)
    return st


# --------------------------------------------------------------------------
# plain forms, 32 bits


def _act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _plain_norm(st):
    c = st["case"]
    s = st["x"]
    if c["residual"]:
        s = (s.float() + st["residual"].float()).bfloat16()
    f = s.float()
    w = st["weight"].float() + (1 if c["unit_offset"] else 0)
    y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + 1e-6) * w
    if not c["fp8"]:
        return (y.bfloat16(), s) if c["residual"] else (y.bfloat16(),)
    T, D = y.shape
    group = c["group"] or D
    n = -(-D // group)
    z = y.new_zeros(T, n * group)
    z[:, :D] = y
    scales = (z.view(T, n, group).abs().amax(-1) / FP8_MAX).clamp_min(2.0 ** -126)
    q = (y / scales.repeat_interleave(group, 1)[:, :D]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return (q, scales, s) if c["residual"] else (q, scales)


def _plain_gate_up(st):
    x, Wq, sc = st["x"].float(), st["Wq"], st["scales"].float()
    shifts = torch.arange(0, 32, 4, device=Wq.device, dtype=torch.int32)
    w = ((Wq[:, :, None] >> shifts) & 15).float().sub_(8).view(Wq.shape[0], -1, 128)
    w = w.mul_(sc[:, :, None]).view(Wq.shape[0], -1)
    y = x @ w.t()
    F = y.shape[1] // 2
    return (_act(y[:, :F], st["case"]["act"]) * y[:, F:]).bfloat16()


def _plain_heads(q, k, v, g, beta, l2norm, Hv):
    """[B][n][heads][d] rows -> 32-bit [B][Hv][n][d], keys shared by Hv / Hk value heads."""
    q, k, v = q.float(), k.float(), v.float()
    if l2norm:
        q = q * torch.rsqrt((q * q).sum(-1, keepdim=True) + L2_EPS)
        k = k * torch.rsqrt((k * k).sum(-1, keepdim=True) + L2_EPS)
    rep = Hv // q.shape[2]
    q, k = (t.repeat_interleave(rep, 2).transpose(1, 2) for t in (q, k))
    return q, k, v.transpose(1, 2), g.transpose(1, 2), beta.transpose(1, 2)


def _plain_block(q, k, v, g, beta, S):
    """One block of rows at once: with G the running sum of g,
    u = (I + tril(beta_i e^(G_i - G_j) k_i k_j, -1))^-1 beta (v - e^G S k),
    o = d^-1/2 (e^G S q + tril(e^(G_i - G_j) q_i k_j) u), S' = e^G_n S + u^T (e^(G_n - G) k)."""
    n = k.shape[2]
    G = g.cumsum(-1)
    diff = G[..., :, None] - G[..., None, :]
    low = torch.ones(n, n, dtype=torch.bool, device=k.device).tril()
    D = torch.exp(torch.where(low, diff, -math.inf))
    A = (beta[..., None] * D * (k @ k.transpose(-1, -2))).tril(-1)
    eG = torch.exp(G)[..., None]
    rhs = beta[..., None] * (v - eG * (k @ S.transpose(-1, -2)))
    u = torch.linalg.solve_triangular(A, rhs, upper=False, unitriangular=True)
    o = (eG * (q @ S.transpose(-1, -2)) + (D * (q @ k.transpose(-1, -2))) @ u) * k.shape[-1] ** -0.5
    last = G[..., -1:]
    S = torch.exp(last)[..., None] * S + u.transpose(-1, -2) @ (torch.exp(last - G)[..., None] * k)
    return o, S


def _plain_step(st):
    c = st["case"]
    idx = st["idx"].long()
    S = st["state"][idx]
    if c["prev"]:
        k, v, g, beta = st["prev"]
        keep = torch.arange(c["prev"], device=k.device) < (st["accept"].long() + 1)[:, None]
        _, k, v, g, beta = _plain_heads(k, k, v, g * keep[..., None], beta * keep[..., None], c["l2norm"], c["Hv"])
        S = kept = _plain_block(k, k, v, g, beta, S)[1]
    o, S = _plain_block(*_plain_heads(*st["rows"], c["l2norm"], c["Hv"]), S)
    if c["commit"]:
        st["state"][idx] = S
    elif c["prev"]:
        st["state"][idx] = kept
    return o.transpose(1, 2).bfloat16(), st["state"]


def _plain_chunk(st):
    c = st["case"]
    q, k, v, g, beta = st["rows"]
    start, end = st["cu"][:-1].long(), st["cu"][1:].long()
    S = torch.zeros_like(st["state"]) if c["zero_init"] else st["state"]
    o = torch.empty(v.shape, dtype=torch.bfloat16, device=v.device)
    at = torch.arange(BLOCK, device=v.device)
    for first in range(0, max(_lens(c)), BLOCK):
        rows = (start + first)[:, None] + at
        real = rows < end[:, None]
        rows = rows.clamp_max(q.shape[0] - 1)
        gate = real[..., None].float()
        out, S = _plain_block(*_plain_heads(q[rows], k[rows], v[rows], g[rows] * gate, beta[rows] * gate,
                                            c["l2norm"], c["Hv"]), S)
        o[rows[real]] = out.transpose(1, 2)[real].bfloat16()
    st["state"].copy_(S)
    return o, st["state"]


def _own(st):
    import speculative_verify_gb300 as sv
    c = st["case"]
    if c["op"] == "norm":
        if c["fp8"]:
            y, scales, s = sv.rmsnorm_fp8(st["x"], st["weight"], st["residual"], group=c["group"],
                                          unit_offset=c["unit_offset"])
            return (y, scales, s) if c["residual"] else (y, scales)
        y, s = sv.rmsnorm(st["x"], st["weight"], st["residual"], unit_offset=c["unit_offset"])
        return (y, s) if c["residual"] else (y,)
    if c["op"] == "gate_up":
        return sv.w4a16_gate_up(st["x"], st["Wq"], st["scales"], act=c["act"])
    if c["op"] == "step":
        o = sv.gated_delta_step(*st["rows"], st["state"], state_idx=st["idx"], prev=st["prev"],
                                accept_len=st["accept"], commit=c["commit"], l2norm=c["l2norm"])
    else:
        o = sv.gated_delta_chunk(*st["rows"], st["cu"], st["state"], zero_init=c["zero_init"], l2norm=c["l2norm"])
    return o, st["state"]


PLAIN = {"norm": _plain_norm, "gate_up": _plain_gate_up, "step": _plain_step, "chunk": _plain_chunk}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------------------
# definitions in 64 bits


def _exact_rule(S, q, k, v, g, beta, real, l2norm):
    """The recurrence itself, a row at a time: S <- e^g S; u = beta (v - S k); S <- S + u k^T; o = d^-1/2 S q.
    Rows [B][n][heads][d]; rows that are not real change nothing and give no output."""
    rep = v.shape[2] // k.shape[2]
    out = torch.zeros(v.shape, dtype=torch.float64, device=v.device)
    for t in range(k.shape[1]):
        kt, qt, vt = k[:, t].double(), q[:, t].double(), v[:, t].double()
        if l2norm:
            kt = kt / torch.sqrt((kt ** 2).sum(-1, keepdim=True) + L2_EPS)
            qt = qt / torch.sqrt((qt ** 2).sum(-1, keepdim=True) + L2_EPS)
        kt, qt = kt.repeat_interleave(rep, 1)[..., None], qt.repeat_interleave(rep, 1)[..., None]
        on = real[:, t, None].double()
        S = S * torch.exp(g[:, t].double() * on)[..., None, None]
        u = (beta[:, t].double() * on)[..., None, None] * (vt[..., None] - S @ kt)
        S = S + u * kt.transpose(-1, -2)
        out[:, t] = (S @ qt)[..., 0] * k.shape[-1] ** -0.5
    return out, S


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "norm":
        s = st["x"]
        if c["residual"]:
            s = (s.double() + st["residual"].double()).bfloat16()
        f = s.double()
        y = f / torch.sqrt(torch.mean(f ** 2, -1, keepdim=True) + 1e-6) * (st["weight"].double() + c["unit_offset"])
        if not c["fp8"]:
            return (y, s.double()) if c["residual"] else (y,)
        T, D = y.shape
        group = c["group"] or D
        parts = y.split(group, 1)
        scales = torch.stack([p.abs().amax(1) / FP8_MAX for p in parts], 1)
        q = torch.cat([(p / scales[:, i:i + 1]).float().to(torch.float8_e4m3fn).double()
                       for i, p in enumerate(parts)], 1)
        return (q, scales, s.double()) if c["residual"] else (q, scales)
    if c["op"] == "gate_up":
        x, F, K = st["x"].double(), c["F"], c["K"]
        out = torch.empty(c["T"], F, dtype=torch.float64, device="cuda")
        for a in range(0, F, 4096):          # a slice of columns at a time
            b = min(F, a + 4096)
            y = []
            for r0, r1 in ((a, b), (F + a, F + b)):
                words = st["Wq"][r0:r1].long()
                lv = torch.stack([(words >> (4 * i)) % 16 - 8 for i in range(8)], -1).reshape(r1 - r0, K).double()
                y.append(x @ (lv * st["scales"][r0:r1].double().repeat_interleave(128, 1)).t())
            g, up = y
            if c["act"] == "silu":
                a_g = g * torch.sigmoid(g)
            else:
                a_g = g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))
            out[:, a:b] = a_g * up
        return out
    if c["op"] == "step":
        B, T, P = c["B"], c["T"], c["prev"]
        full = st["state"].double()
        idx = st["idx"].long()
        S = full[idx]
        if P:
            k, v, g, beta = st["prev"]
            real = torch.arange(P, device="cuda")[None] <= st["accept"].long()[:, None]
            S = kept = _exact_rule(S, k, k, v, g, beta, real, c["l2norm"])[1]
        o, S = _exact_rule(S, *st["rows"], torch.ones(B, T, dtype=torch.bool, device="cuda"), c["l2norm"])
        if c["commit"]:
            full[idx] = S
        elif P:
            full[idx] = kept
        return o, full
    lens = _lens(c)
    n, B = max(lens), len(lens)
    q, k, v, g, beta = st["rows"]
    pad = lambda t: torch.stack([torch.cat([p, p.new_zeros(n - p.shape[0], *p.shape[1:])])    # noqa: E731
                                 for p in t.split(lens)])
    real = torch.arange(n, device="cuda")[None] < torch.tensor(lens, device="cuda")[:, None]
    S = torch.zeros_like(st["state"]).double() if c["zero_init"] else st["state"].double()
    o, S = _exact_rule(S, *(pad(t) for t in (q, k, v, g, beta)), real, c["l2norm"])
    return o[real], S
