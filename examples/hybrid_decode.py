"""Greedy speculative decoding of a small hybrid decoder from the library's
operators: whole prompts through gated_delta_chunk, then verify cycles in which
every layer runs

    rmsnorm -> w4a16_gemm (QKV) -> gated_delta_step -> w4a16_gemm (out)
    -> rmsnorm -> w4a16_gate_up -> w4a16_gemm (down)

and lmhead_verify_batched tells how many drafts hold.  The recurrent states are
never advanced past unverified drafts: a cycle hands its rows to the next one
as ``prev`` with the accept_len that the head wrote, on the device, and the
accepted ones are replayed there.

Weights are random (seeded), so the text means nothing and no cheap drafter
could guess it: the drafts are the text of a run without drafts, with every
fifth token wrong.  Run: python examples/hybrid_decode.py
"""
import os
import sys
from dataclasses import dataclass

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gen
import speculative_verify_gb300 as sv

MAX_ROWS = 32                           # rows of one weight pass


@dataclass
class Config:
    layers: int = 2
    hidden: int = 512
    key_heads: int = 2
    value_heads: int = 4
    dk: int = 128
    dv: int = 128
    ffn: int = 1408
    vocab: int = 4096


class Model:
    def __init__(self, cfg, seed=0):
        self.cfg, rng = cfg, np.random.default_rng(seed)
        dev = "cuda"

        def packed(rows, K):            # levels of +-8 at U(0.005, 0.02): scaled to keep activations of order one
            W, s = gen.weights(rng, rows, K)
            s = torch.from_numpy(gen.bf16_bits_to_f32(s).copy()) * (16 / K) ** 0.5
            return torch.from_numpy(W.view(np.int32)).to(dev), s.bfloat16().to(dev)

        def dense(*shape, scale=1.0):
            return torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * scale).to(dev)

        c, nv = cfg, cfg.value_heads * cfg.dv
        self.embed = dense(c.vocab, c.hidden).bfloat16()
        self.layers = [dict(norm1=(1 + 0.1 * dense(c.hidden)).bfloat16(), norm2=(1 + 0.1 * dense(c.hidden)).bfloat16(),
                            qkv=packed(2 * c.key_heads * c.dk + nv, c.hidden), out=packed(c.hidden, nv),
                            gates=dense(c.hidden, 2 * c.value_heads, scale=c.hidden ** -0.5).bfloat16(),
                            rate=torch.from_numpy(rng.uniform(0.02, 0.5, c.value_heads).astype(np.float32)).to(dev),
                            gate_up=packed(2 * c.ffn, c.hidden), down=packed(c.hidden, c.ffn))
                       for _ in range(c.layers)]
        self.norm = (1 + 0.1 * dense(c.hidden)).bfloat16()
        self.head = packed(c.vocab, c.hidden)

    def states(self, B):
        """Zero states of B sequences, one tensor a layer."""
        c = self.cfg
        return [torch.zeros(B, c.value_heads, c.dv, c.dk, device="cuda") for _ in range(c.layers)]

    def forward(self, tokens, delta):
        """The last norm's rows [n][hidden] for tokens [n]; delta(layer, q, k,
        v, g, beta) runs the gated delta rule on the n rows."""
        c, n, nk = self.cfg, tokens.numel(), self.cfg.key_heads * self.cfg.dk

        def by_slices(f, x, *w):        # a weight pass takes up to 32 rows
            if n <= MAX_ROWS:
                return f(x, *w)
            return torch.cat([f(x[i:i + MAX_ROWS], *w) for i in range(0, n, MAX_ROWS)])

        res = self.embed[tokens]
        y, _ = sv.rmsnorm(res, self.layers[0]["norm1"])
        for i, w in enumerate(self.layers):
            qkv = torch.nn.functional.silu(by_slices(sv.w4a16_gemm, y, *w["qkv"]))
            gates = (y @ w["gates"]).float()
            g = -w["rate"] * torch.nn.functional.softplus(gates[:, :c.value_heads])
            beta = torch.sigmoid(gates[:, c.value_heads:]).contiguous()
            o = delta(i, qkv[:, :nk].unflatten(1, (c.key_heads, c.dk)), qkv[:, nk:2 * nk].unflatten(1, (c.key_heads, c.dk)),
                      qkv[:, 2 * nk:].unflatten(1, (c.value_heads, c.dv)), g, beta)
            a = by_slices(sv.w4a16_gemm, o.reshape(n, -1), *w["out"])
            y, res = sv.rmsnorm(a, w["norm2"], residual=res)
            h = by_slices(sv.w4a16_gate_up, y, *w["gate_up"])
            d = by_slices(sv.w4a16_gemm, h, *w["down"])
            last = i + 1 == len(self.layers)
            y, res = sv.rmsnorm(d, self.norm if last else self.layers[i + 1]["norm1"], residual=res)
        return y

    def prompt(self, prompts, states):
        """Whole prompts into the states; the first new token of each sequence."""
        lens = [len(p) for p in prompts]
        cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
        tokens = torch.tensor(sum(prompts, []), device="cuda")
        y = self.forward(tokens, lambda i, q, k, v, g, beta: sv.gated_delta_chunk(
            q, k, v, g, beta, cu, states[i], zero_init=True, l2norm=True))
        ends = y[(cu[1:] - 1).long()].contiguous()
        return sv.lmhead_argmax(ends, *self.head)[0]

    def verify(self, tokens, states, prev=None, accept_len=None, commit=False):
        """One cycle over tokens [B][1 + drafts]: (accept_len, next_token, rows
        for the next cycle's prev)."""
        B, T = tokens.shape
        rows = []

        def delta(i, q, k, v, g, beta):
            q, k, v, g, beta = (t.unflatten(0, (B, T)) for t in (q, k, v, g, beta))
            rows.append((k, v, g, beta))
            return sv.gated_delta_step(q, k, v, g, beta, states[i], prev=prev and prev[i], accept_len=accept_len,
                                       commit=commit, l2norm=True)

        y = self.forward(tokens.reshape(-1).long(), delta)
        acc, nxt = sv.lmhead_verify_batched(y, *self.head, tokens[:, 1:].contiguous())
        return acc, nxt, rows

    def replay(self, states, prev, accept_len):
        """The last cycle's accepted rows into the states, no new rows."""
        for i, (k, v, g, beta) in enumerate(prev):
            q = k[:, :0]
            sv.gated_delta_step(q, q, v[:, :0], g[:, :0], beta[:, :0], states[i], prev=(k, v, g, beta),
                                accept_len=accept_len, l2norm=True)


def drafter(texts):
    """Drafts n tokens of a sequence from known texts, every fifth wrong."""
    def draft(history, n):
        known = next((t for t in texts if t[:len(history)] == history), None)
        if known is None:
            return [history[-1]] * n
        return [(x ^ 1 if (len(history) + i) % 5 == 4 else x)
                for i, x in enumerate((known[len(history):] + [0] * n)[:n])]
    return draft


def generate(model, prompts, n_tokens, n_draft=0, draft=None):
    """Greedy decoding: (new tokens of each prompt, cycles, states after all
    but the newest token of each)."""
    states = model.states(len(prompts))
    first = model.prompt(prompts, states).tolist()
    text = [p + [t] for p, t in zip(prompts, first)]
    prev = acc = None
    cycles = 0
    while min(len(t) - len(p) for t, p in zip(text, prompts)) < n_tokens:
        drafts = [draft(t, n_draft) if n_draft else [] for t in text]
        tokens = torch.tensor([[t[-1]] + d for t, d in zip(text, drafts)], dtype=torch.int32, device="cuda")
        acc, nxt, prev = model.verify(tokens, states, prev, acc)
        for t, d, a, x in zip(text, drafts, acc.tolist(), nxt.tolist()):
            t += d[:a] + [x]
        cycles += 1
    if prev:
        model.replay(states, prev, acc)
    return [t[len(p):] for t, p in zip(text, prompts)], cycles, states


def main():
    rng = np.random.default_rng(1)
    cfg = Config()
    model = Model(cfg)
    prompts = [rng.integers(0, cfg.vocab, n).tolist() for n in (300, 41)]
    new, cycles, _ = generate(model, prompts, 48)
    print("no drafts: %d cycles for %s tokens" % (cycles, " and ".join(str(len(t)) for t in new)))
    fast, cycles, _ = generate(model, prompts, 48, 3, drafter([p + t for p, t in zip(prompts, new)]))
    print("3 drafts: %d cycles for %s tokens" % (cycles, " and ".join(str(len(t)) for t in fast)))
    for t in fast:
        print(*t[:16], "...")


if __name__ == "__main__":
    main()
