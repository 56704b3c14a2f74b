"""The paged-cache operators and the verifier together: the tokens of
draft-then-verify rounds are those of plain greedy decoding."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


def dense_logits(target, tokens, window, sinks):
    """Logits [n, V] after each token of one sequence, in 64 bits, without a cache."""
    x = target.qkv[tokens].double()
    h, k = target.heads, target.kv_heads
    q, ks, vs = x[:, :h], x[:, h:h + k], x[:, h + k:]
    n = len(tokens)
    i, j = torch.arange(n, device=x.device)[:, None], torch.arange(n, device=x.device)
    hidden = j > i
    if window:
        hidden = hidden | ((i - j >= window) & (j >= sinks))
    rows = []
    for head in range(h):
        s = (q[:, head] @ ks[:, head // (h // k)].T) * target.dim ** -0.5
        rows.append(torch.softmax(s.masked_fill(hidden, -torch.inf), 1)
                    @ vs[:, head // (h // k)])
    flat = torch.stack(rows, 1).reshape(n, -1)
    return flat @ target.out.double() + target.bigram[tokens].double()


@pytest.mark.parametrize("window,sinks,gamma,page", [(0, 0, 4, 16), (24, 3, 3, 8), (0, 0, 7, 64)])
def test_rounds_decode_as_the_target_alone(window, sinks, gamma, page):
    import paged_rounds
    target = paged_rounds.Target(V=256, seed=3)
    g = torch.Generator().manual_seed(gamma)
    prompts = [torch.randint(0, 256, (n,), generator=g).tolist() for n in (1, 2, 15, 16, 17, 90)]
    tokens, accepted = paged_rounds.decode(target, prompts, rounds=8, gamma=gamma, page=page,
                                           window=window, sinks=sinks)
    counts = [sum(a[r] for a in accepted) for r in range(len(prompts))]
    assert 0 < sum(counts) < 8 * gamma * len(prompts)  # drafts were accepted and rejected
    for r, (prompt, out) in enumerate(zip(prompts, tokens)):
        assert len(out) == counts[r] + 8
        logits = dense_logits(target, torch.tensor(prompt + out[:-1], device="cuda:0"), window,
                              sinks)[len(prompt) - 1:]
        best = logits.max(1).values
        chosen = logits.gather(1, torch.tensor(out, device="cuda:0")[:, None])[:, 0]
        # Both logits were rounded to bf16 (half a spacing of at most 2^-8 of the largest,
        # twice), after an attention in bf16 (2^-8 of its values, which the output matrix
        # takes with a factor of about 0.7 * 8 / sqrt(512) * sqrt(512) = 5.6).
        slack = 2 * 2.0 ** -8 * logits.abs().max() + 2 * 2.0 ** -8 * 5.6 * 3
        assert ((best - chosen) <= slack).all()
