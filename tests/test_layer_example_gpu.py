"""The operators together, as examples/hybrid_decode.py runs them: speculative
cycles leave the recurrent states where one-token decoding of the same tokens
leaves them, and emit what that decoding would."""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("hybrid_decode", os.path.join(ROOT, "examples", "hybrid_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("n_draft", [0, 1, 3, 7])
def test_cycles_match_single_token_decoding(ex, n_draft):
    """A row's activations are rounded to bf16 (2^-9) at each of a dozen places
    a layer, in sums that the row count may order differently: the states of
    two layers are held to 2^-5 of their norm, and the logit of an emitted
    token to 2^-5 of the largest logit below the largest."""
    cfg = ex.Config()
    model = ex.Model(cfg, seed=3)
    rng = np.random.default_rng(4)
    prompts = [rng.integers(0, cfg.vocab, n).tolist() for n in (131, 1, 70)]
    plain, cycles, states = ex.generate(model, prompts, 20)
    assert cycles == 19 and all(len(t) == 20 for t in plain)
    new = plain
    if n_draft:
        texts = [p + t for p, t in zip(prompts, plain)]
        new, cycles, states = ex.generate(model, prompts, 20, n_draft, ex.drafter(texts))
        assert all(len(t) >= 20 for t in new) and cycles < 19    # some drafts held

    levels = (model.head[0].view(torch.uint8).cpu().numpy().reshape(cfg.vocab, -1))
    levels = np.stack([levels & 15, levels >> 4], -1).reshape(cfg.vocab, cfg.hidden).astype(np.float64) - 8
    head = levels * np.repeat(model.head[1].float().cpu().numpy().astype(np.float64), 128, axis=1)
    for b, (p, t) in enumerate(zip(prompts, new)):
        one = model.states(1)
        model.prompt([p], one)
        for i, x in enumerate(t[:-1]):
            tokens = torch.tensor([[x]], dtype=torch.int32, device="cuda")

            def delta(j, *a):
                q, k, v, g, beta = (s.unflatten(0, (1, 1)) for s in a)
                return ex.sv.gated_delta_step(q, k, v, g, beta, one[j], l2norm=True)

            y = model.forward(tokens.reshape(-1).long(), delta)
            logits = head @ y[0].double().cpu().numpy()
            assert logits.max() - logits[t[i + 1]] <= 2 ** -5 * np.abs(logits).max(), (b, i)
        for j in range(cfg.layers):
            a, want = states[j][b].double(), one[j][0].double()
            assert ((a - want).norm() <= 2 ** -5 * want.norm()).item(), (b, j)
