"""Greedy speculative decoding of a small hybrid decoder from the library's
operators: whole prompts through gated_delta_chunk, then verify cycles in which
every layer runs

    rmsnorm -> w4a16_gemm (QKV) -> gated_delta_step -> w4a16_gemm (out)
    -> rmsnorm -> w4a16_gate_up -> w4a16_gemm (down)

and lmhead_verify_batched tells how many drafts hold.  The recurrent states are
never advanced past unverified drafts: a cycle hands its rows to the next one
as ``prev`` with the accept_len that the head wrote, on the device, and the
accepted ones are replayed there.

With Config(attention_every=n) every n-th layer is an attention layer instead:

    rmsnorm -> w4a16_gemm (QKV) -> rotary -> kv4_append -> kv4_attention -> w4a16_gemm (out) ...

over a cache of 4-bit pages.  Its rows are appended before they are verified: a
cycle moves the sequences' lengths on by the accepted rows alone, on the
device, and the next one writes over the others.

Weights are random (seeded), so the text means nothing and no cheap drafter
could guess it: the drafts are the text of a run without drafts, with every
fifth token wrong.  Run: python examples/hybrid_decode.py
[attention_every]
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
    attention_every: int = 0            # every n-th layer attends; 0: none
    heads: int = 8                      # of its queries
    kv_heads: int = 2
    head_dim: int = 128
    window: int = 0                     # tokens that it sees besides the first `sinks`; 0: all
    sinks: int = 4
    max_tokens: int = 1024              # of a sequence

    def attends(self, i):
        return self.attention_every > 0 and (i + 1) % self.attention_every == 0


class Cache:
    """An attention layer's pages and the sequences' tables of them."""
    def __init__(self, cfg, B):
        n = -(-cfg.max_tokens // sv.KV4_PAGE)
        self.pages = sv.kv4_cache(B * n, cfg.kv_heads, cfg.head_dim)
        self.table = torch.arange(B * n, dtype=torch.int32, device="cuda").view(B, n)


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

        c = cfg
        self.embed = dense(c.vocab, c.hidden).bfloat16()
        self.layers = [dict(norm1=(1 + 0.1 * dense(c.hidden)).bfloat16(), norm2=(1 + 0.1 * dense(c.hidden)).bfloat16(),
                            qkv=packed(self.widths(i)[0], c.hidden), out=packed(c.hidden, self.widths(i)[1]),
                            gates=dense(c.hidden, 2 * c.value_heads, scale=c.hidden ** -0.5).bfloat16(),
                            rate=torch.from_numpy(rng.uniform(0.02, 0.5, c.value_heads).astype(np.float32)).to(dev),
                            gate_up=packed(2 * c.ffn, c.hidden), down=packed(c.hidden, c.ffn))
                       for i in range(c.layers)]
        self.norm = (1 + 0.1 * dense(c.hidden)).bfloat16()
        self.head = packed(c.vocab, c.hidden)
        half = c.head_dim // 2
        self.inv_freq = 1e4 ** (-torch.arange(half, device=dev) / half)

    def widths(self, i):
        """Columns of layer i's fused QKV projection and of its heads' outputs."""
        c = self.cfg
        if c.attends(i):
            return (c.heads + 2 * c.kv_heads) * c.head_dim, c.heads * c.head_dim
        return 2 * c.key_heads * c.dk + c.value_heads * c.dv, c.value_heads * c.dv

    def states(self, B):
        """Zero states of B sequences, one tensor a layer; attention layers' caches."""
        c = self.cfg
        return [Cache(c, B) if c.attends(i) else torch.zeros(B, c.value_heads, c.dv, c.dk, device="cuda")
                for i in range(c.layers)]

    def attend(self, cache, qkv, positions, lens, cu=None):
        """An attention layer: qkv [B][T] or, with cu, [R] rows of queries, keys
        and values, whose sequences have lens tokens before them."""
        c = self.cfg
        nq, nk = c.heads * c.head_dim, c.kv_heads * c.head_dim
        q, k, v = (t.unflatten(-1, (-1, c.head_dim)) for t in qkv.split((nq, nk, nk), -1))
        q, k = sv.rotary(q, k, positions, self.inv_freq)
        sv.kv4_append(k, v, cache.pages, cache.table, lens, cu)
        return sv.kv4_attention(q, cache.pages, cache.table, lens, cu, window=c.window, sinks=c.sinks if c.window else 0)

    def forward(self, tokens, delta, attend=None):
        """The last norm's rows [n][hidden] for tokens [n]; delta(layer, q, k,
        v, g, beta) runs the gated delta rule on the n rows, attend(layer, qkv)
        an attention layer."""
        c, n, nk = self.cfg, tokens.numel(), self.cfg.key_heads * self.cfg.dk

        def by_slices(f, x, *w):        # a weight pass takes up to 32 rows
            if n <= MAX_ROWS:
                return f(x, *w)
            return torch.cat([f(x[i:i + MAX_ROWS], *w) for i in range(0, n, MAX_ROWS)])

        res = self.embed[tokens]
        y, _ = sv.rmsnorm(res, self.layers[0]["norm1"])
        for i, w in enumerate(self.layers):
            qkv = by_slices(sv.w4a16_gemm, y, *w["qkv"])
            if c.attends(i):
                o = attend(i, qkv)
            else:
                qkv = torch.nn.functional.silu(qkv)
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
        positions = torch.cat([torch.arange(n, dtype=torch.int32, device="cuda") for n in lens])
        y = self.forward(tokens, lambda i, q, k, v, g, beta: sv.gated_delta_chunk(
            q, k, v, g, beta, cu, states[i], zero_init=True, l2norm=True),
            lambda i, qkv: self.attend(states[i], qkv, positions, torch.zeros_like(cu[1:]), cu))
        ends = y[(cu[1:] - 1).long()].contiguous()
        return sv.lmhead_argmax(ends, *self.head)[0]

    def verify(self, tokens, states, prev=None, accept_len=None, commit=False, lens=None):
        """One cycle over tokens [B][1 + drafts]: (accept_len, next_token, rows
        for the next cycle's prev).  lens [B] (with attention layers): the tokens
        before them."""
        B, T = tokens.shape
        rows = [None] * self.cfg.layers

        def delta(i, q, k, v, g, beta):
            q, k, v, g, beta = (t.unflatten(0, (B, T)) for t in (q, k, v, g, beta))
            rows[i] = (k, v, g, beta)
            return sv.gated_delta_step(q, k, v, g, beta, states[i], prev=prev and prev[i], accept_len=accept_len,
                                       commit=commit, l2norm=True)

        def attend(i, qkv):
            positions = lens[:, None] + torch.arange(T, dtype=torch.int32, device="cuda")
            return self.attend(states[i], qkv.unflatten(0, (B, T)), positions, lens)

        y = self.forward(tokens.reshape(-1).long(), delta, attend)
        acc, nxt = sv.lmhead_verify_batched(y, *self.head, tokens[:, 1:].contiguous())
        return acc, nxt, rows

    def replay(self, states, prev, accept_len):
        """The last cycle's accepted rows into the states, no new rows."""
        for i, rows in enumerate(prev):
            if rows is None:            # (an attention layer)
                continue
            k, v, g, beta = rows
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
    lens = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
    while min(len(t) - len(p) for t, p in zip(text, prompts)) < n_tokens:
        drafts = [draft(t, n_draft) if n_draft else [] for t in text]
        tokens = torch.tensor([[t[-1]] + d for t, d in zip(text, drafts)], dtype=torch.int32, device="cuda")
        acc, nxt, prev = model.verify(tokens, states, prev, acc, lens=lens)
        lens = lens + acc + 1
        for t, d, a, x in zip(text, drafts, acc.tolist(), nxt.tolist()):
            t += d[:a] + [x]
        cycles += 1
    if prev:
        model.replay(states, prev, acc)
    return [t[len(p):] for t, p in zip(text, prompts)], cycles, states


def main():
    rng = np.random.default_rng(1)
    cfg = Config(attention_every=int(sys.argv[1]) if len(sys.argv) > 1 else 0)
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
