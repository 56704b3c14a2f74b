"""Draft-then-verify rounds over a paged cache, end to end on one GPU.

A toy target (one attention layer between random embeddings and an output
matrix, with a bigram term that a greedy bigram draft guesses well) decodes a
batch of prompts. Every round is

    cache_step    drop what the last round rejected, make room for the last
                  token and the new drafts of every request
    cache_append  their keys and values into the pages
    cache_attend  the target's attention, the drafts of a request in one pass
    Verifier      accept drafts, emit one token more

and no length is read back before the end. Run: python examples/paged_rounds.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import speculative_decoding_rejection_02_gb300 as sv  # noqa: E402


class Target:
    """Random weights: x = E[token]; logits = attention(x Wq, x Wk, x Wv) Wo + bigram[token]."""

    def __init__(self, V=512, heads=8, kv_heads=2, dim=64, seed=0, device="cuda:0"):
        g = torch.Generator().manual_seed(seed)
        self.V, self.heads, self.kv_heads, self.dim = V, heads, kv_heads, dim
        width = (heads + 2 * kv_heads) * dim

        def randn(*shape, scale):
            return (torch.randn(shape, generator=g) * scale).to(device, torch.bfloat16)
        # the projected token is all that q, k and v depend on
        self.qkv = randn(V, heads + 2 * kv_heads, dim, scale=1.0)
        self.out = randn(heads * dim, V, scale=0.7 * (heads * dim) ** -0.5 * 8)
        self.bigram = randn(V, V, scale=3.0)
        self.width = width

    def project(self, tokens):
        x = self.qkv[tokens]
        h, k = self.heads, self.kv_heads
        return x[:, :h], x[:, h:h + k], x[:, h + k:]

    def logits(self, attended, tokens):
        flat = attended.reshape(attended.shape[0], -1)
        return (flat @ self.out + self.bigram[tokens]).contiguous()

    def draft(self, last, gamma):
        """[B, gamma] tokens, each the bigram's favourite after the one before."""
        favourite = self.bigram.argmax(1)
        out = []
        for _ in range(gamma):
            last = favourite[last]
            out.append(last)
        return torch.stack(out, 1)


def decode(target, prompts, rounds=6, gamma=4, page=16, window=0, sinks=0):
    """Greedy decoding of `prompts` (lists of tokens) for some rounds. Returns
    the emitted tokens of each request and the accepted drafts [rounds, B]."""
    dev, B = target.qkv.device, len(prompts)
    most = max(map(len, prompts)) + rounds * (gamma + 1)
    width = -(-most // page)
    pages = B * width
    shape = (pages, page, target.kv_heads, target.dim)
    k_pages = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    v_pages = torch.empty_like(k_pages)
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    free = torch.arange(pages, dtype=torch.int32, device=dev)
    count = torch.full((1,), pages, dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)

    def target_pass(step, tokens, max_q):
        q, k, v = target.project(tokens)
        sv.cache_append(k, v, step.slots, k_pages, v_pages, status=status)
        o = sv.cache_attend(q, k_pages, v_pages, table, step.lens, step.cu_new, max_q=max_q,
                            window=window, sinks=sinks, status=status)
        return target.logits(o, tokens)

    # The prompts but for their last tokens, which the first round takes.
    fed = torch.tensor([len(p) - 1 for p in prompts], dtype=torch.int32, device=dev)
    chunk = torch.tensor([t for p in prompts for t in p[:-1]], device=dev)
    last = torch.tensor([p[-1] for p in prompts], device=dev)
    step = sv.cache_step(torch.zeros_like(fed), fed, table, free, count, page_size=page,
                         num_tokens=chunk.numel(), status=status)
    if chunk.numel():
        target_pass(step, chunk, max(map(len, prompts)))

    verifier = sv.Verifier(max_batch=B, max_rows=B * (gamma + 1), max_vocab=target.V)
    cu_draft = torch.arange(B + 1, dtype=torch.int32, device=dev) * gamma
    new = torch.full((B,), gamma + 1, dtype=torch.int32, device=dev)
    greedy = torch.zeros(B, device=dev)
    emitted, accepted = [], []
    drafts_before = None
    for _ in range(rounds):
        drafts = target.draft(last, gamma)
        step = sv.cache_step(step.lens, new, table, free, step.free_count, page_size=page,
                             num_tokens=B * (gamma + 1), cu_num_draft=drafts_before,
                             num_accepted=accepted[-1] if accepted else None, status=status)
        tokens = torch.cat([last[:, None], drafts], 1).reshape(-1)
        batch = sv.DeviceBatch(cu_num_draft=cu_draft,
                               draft_token_ids=drafts.reshape(-1).to(torch.int32),
                               target_logits=target_pass(step, tokens, gamma + 1),
                               draft_probs=None, temperature=greedy)
        verifier.run(batch)
        emitted.append(batch.out_tokens.view(B, gamma + 1))
        accepted.append(batch.num_accepted)
        last = emitted[-1].gather(1, accepted[-1].long()[:, None])[:, 0].long()
        drafts_before = cu_draft
    bits = int(status) | verifier.status()
    verifier.close()
    if bits:
        raise RuntimeError(f"device status {bits:#x}")
    emitted, accepted = [e.tolist() for e in emitted], [a.tolist() for a in accepted]
    tokens = [[t for e, a in zip(emitted, accepted) for t in e[r][: a[r] + 1]] for r in range(B)]
    return tokens, accepted


def main():
    g = torch.Generator().manual_seed(1)
    target = Target()
    prompts = [torch.randint(0, target.V, (n,), generator=g).tolist()
               for n in (1, 5, 40, 133, 700, 64, 16, 17)]
    tokens, accepted = decode(target, prompts, rounds=16)
    total = sum(map(len, tokens))
    drafts = 16 * len(prompts) * 4
    print(f"{len(prompts)} requests, 16 rounds: {total} tokens, "
          f"{sum(map(sum, accepted)) / drafts:.2f} of the drafts accepted, "
          f"{total / (16 * len(prompts)):.2f} tokens a round")


if __name__ == "__main__":
    main()
