"""The paged-cache operators of a verification round, as measured work.

A round of draft-then-verify decoding runs the target once over the last kept
token and the drafts of every request. Around the verifier that takes three
operators on a paged key/value cache:

  step    after a verification: drop the rejected tokens of every request, give
          their pages back, take pages for the next round's tokens, and write
          the block table, the positions and the cache slots of those tokens;
  append  write the new tokens' keys and values to their slots;
  attend  attention of each request's new tokens over its pages: one token, a
          few drafts or a long chunk, with an optional sliding window beside
          which a few first tokens stay visible.

``run`` computes each in its plain form (elementary torch operations in 32
bits), or, where ``own`` is true, through this package's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # The smallest round: a few requests, three drafts each.
        dict(name="step_small", op="step", B=8, gamma_lo=3, gamma_hi=3, new_lo=4, new_hi=4,
             ctx_lo=100, ctx_hi=2000, page=16, width=160),
        # A full serving batch, one to seven drafts each (the ragged batch the verifier is
        # benchmarked on).
        dict(name="step_batch", op="step", B=1024, gamma_lo=1, gamma_hi=7, new_lo=2, new_hi=8,
             ctx_lo=50, ctx_hi=16000, page=16, width=1100),
        # Many short requests of which some bring a prompt chunk: long token lists.
        dict(name="step_chunks", op="step", B=6000, gamma_lo=0, gamma_hi=5, new_lo=1, new_hi=40,
             ctx_lo=1, ctx_hi=4000, page=32, width=200),
        # The new tokens of a small verification batch (latency).
        dict(name="append_round", op="append", T=320, kv_heads=8, dim=128, page=16, dtype="bf16",
             layout="token", idle=17),
        # A prompt chunk's keys and values, pages with the heads outside the tokens.
        dict(name="append_chunk", op="append", T=50001, kv_heads=8, dim=128, page=64,
             dtype="fp16", layout="head", idle=0),
        # One request, one token, a middling context: latency.
        dict(name="attend_one", op="attend", B=1, q_lo=1, q_hi=1, ctx_lo=4097, ctx_hi=4097,
             heads=32, kv_heads=8, dim=128, page=16, dtype="bf16", layout="token", window=0,
             sinks=0),
        # Plain decoding of a batch with ragged contexts.
        dict(name="attend_decode", op="attend", B=128, q_lo=1, q_hi=1, ctx_lo=150, ctx_hi=9000,
             heads=32, kv_heads=8, dim=128, page=16, dtype="bf16", layout="token", window=0,
             sinks=0),
        # A verification round: the last token and up to seven drafts per request.
        dict(name="attend_verify", op="attend", B=64, q_lo=2, q_hi=8, ctx_lo=1000, ctx_hi=30000,
             heads=32, kv_heads=8, dim=128, page=32, dtype="bf16", layout="token", window=0,
             sinks=0),
        # Few requests with long documents, smaller heads.
        dict(name="attend_long", op="attend", B=2, q_lo=5, q_hi=5, ctx_lo=190000, ctx_hi=200000,
             heads=28, kv_heads=4, dim=64, page=16, dtype="fp16", layout="head", window=0,
             sinks=0),
        # Prompt chunks over what is cached already.
        dict(name="attend_chunk", op="attend", B=2, q_lo=2048, q_hi=2048, ctx_lo=11000,
             ctx_hi=14000, heads=32, kv_heads=8, dim=128, page=64, dtype="bf16", layout="token",
             window=0, sinks=0),
        # A verification round of a model whose layers see a window and the first tokens.
        dict(name="attend_window", op="attend", B=64, q_lo=1, q_hi=6, ctx_lo=500, ctx_hi=25000,
             heads=32, kv_heads=8, dim=128, page=16, dtype="bf16", layout="token", window=1024,
             sinks=4),
        # A ragged chunked prefill with a window, odd head counts and a head size that is not
        # a power of two.
        dict(name="attend_window_chunk", op="attend", B=6, q_lo=77, q_hi=1500, ctx_lo=300,
             ctx_hi=8000, heads=14, kv_heads=2, dim=96, page=32, dtype="fp16", layout="head",
             window=2000, sinks=16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "append", "attend", "attend"])
    if op == "step":
        B = _log_int(rng, 1, 6000)
        g = rng.randint(0, 7)
        new_hi = _log_int(rng, 1, 40)
        page = rng.choice([8, 16, 32, 64])
        hi = _log_int(rng, 20, 16000 if B <= 1024 else 4000)
        return dict(op="step", B=B, gamma_lo=rng.randint(0, g), gamma_hi=g,
                    new_lo=rng.randint(0, new_hi), new_hi=new_hi, ctx_lo=rng.randint(1, 19),
                    ctx_hi=hi, page=page, width=-(-(hi + 60) // page) + rng.randint(0, 9))
    if op == "append":
        return dict(op="append", T=_log_int(rng, 1, 50000), kv_heads=rng.choice([1, 2, 4, 5, 8]),
                    dim=rng.choice([64, 80, 96, 128]), page=rng.choice([16, 32, 64]),
                    dtype=rng.choice(["bf16", "fp16"]), layout=rng.choice(["token", "head"]),
                    idle=rng.choice([0, 0, rng.randint(1, 50)]))
    top = [max(x) for x in zip(*(_cost(c) for c in listed() if c["op"] == "attend"))]
    while True:
        q_hi = _log_int(rng, 1, 2048)
        kv_heads = rng.choice([1, 2, 4, 5, 8])
        hi = _log_int(rng, 20, 200000)
        c = dict(op="attend", B=_log_int(rng, 1, 128), q_lo=rng.randint(1, q_hi), q_hi=q_hi,
                 ctx_lo=rng.randint(1, hi), ctx_hi=hi,
                 heads=kv_heads * rng.choice([1, 2, 3, 4, 7, 8]), kv_heads=kv_heads,
                 dim=rng.choice([64, 80, 96, 128]), page=rng.choice([16, 32, 64]),
                 dtype=rng.choice(["bf16", "fp16"]), layout=rng.choice(["token", "head"]),
                 window=rng.choice([0, 0, _log_int(rng, 16, 8192)]),
                 sinks=rng.choice([0, 4, rng.randint(1, 64)]))
        if not c["window"]:
            c["sinks"] = 0
        if all(x <= y for x, y in zip(_cost(c), top)):
            return c


def _cost(c):
    """What an attend case goes through in its padded plain form: elements of the keys,
    scores, and multiplications."""
    L = c["ctx_hi"] + c["q_hi"]
    scores = c["B"] * c["heads"] * c["q_hi"] * L
    return c["B"] * L * c["kv_heads"] * c["dim"], scores, scores * c["dim"]


def _spread(lo, hi, n, log):
    """n whole numbers from lo to hi at even steps (of the logarithm)."""
    at = [(i + 0.5) / n for i in range(n)]
    if log:
        return [int(lo * (hi / lo) ** x) for x in at]
    return [int(lo + x * (hi + 1 - lo)) for x in at]


def _live(c):
    """Tokens of an append case that have a slot."""
    return c["T"] - min(c["idle"], c["T"] - 1)


def _shuffled(values, g):
    """The values in an order that the generator gives, as an int64 tensor."""
    order = torch.randperm(len(values), generator=g, device="cuda")
    return torch.tensor(values, device="cuda", dtype=torch.int64)[order]


def _starts(lens):
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    return torch.cat([zero, torch.cumsum(lens, 0)]).to(torch.int32)


def _pool(pages, c, g):
    """Cache pages as [pages, page, kv_heads, dim], laid out with the tokens or the heads
    outside."""
    dims = (pages, c["page"], c["kv_heads"], c["dim"])
    if c["layout"] == "head":
        dims = (pages, c["kv_heads"], c["page"], c["dim"])
    x = torch.randn(dims, generator=g, device="cuda", dtype=DTYPES[c["dtype"]])
    return x.transpose(1, 2) if c["layout"] == "head" else x


def _tables(lens, page, width, pages, g):
    """A block table [B, width] of distinct pages in scattered order, -1 past each request's
    pages, and the pages that no request holds."""
    held = (lens + page - 1) // page
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    first = torch.cumsum(held, 0) - held
    col = torch.arange(width, device="cuda")
    at = (first[:, None] + col).clamp(max=pages - 1)
    table = torch.where(col < held[:, None], order[at], torch.full_like(at, -1, dtype=torch.int32))
    return table.contiguous(), order, int(held.sum())


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": c}
    if c["op"] == "step":
        B, page = c["B"], c["page"]
        draft = _shuffled(_spread(c["gamma_lo"], c["gamma_hi"], B, False), g)
        new = _shuffled(_spread(c["new_lo"], c["new_hi"], B, False), g)
        # what is held now: the context, the last token and the drafts just verified
        held = _shuffled(_spread(c["ctx_lo"], c["ctx_hi"], B, True), g) + draft + 1
        # a draft is accepted with probability 0.75, up to the first that is not
        hit = torch.rand((B, 8), generator=g, device="cuda") < 0.75
        run_len = torch.cumprod(hit.to(torch.int64), 1).sum(1)
        pages = int((held + new).sum()) // page + B + 64  # the same for every seed
        table, order, used = _tables(held, page, c["width"], pages, g)
        free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
        free[: pages - used] = order[used:]
        s.update(held=held.to(torch.int32), new=new.to(torch.int32), cu_draft=_starts(draft),
                 accepted=torch.minimum(run_len, draft).to(torch.int32), table=table, free=free,
                 free_count=torch.tensor([pages - used], dtype=torch.int32, device="cuda"),
                 tokens=B * c["new_hi"])
        return s
    if c["op"] == "append":
        T, page = c["T"], c["page"]
        pages = -(-T // page) * 5 // 4 + 2
        # the new tokens of a fused projection: q, k and v side by side
        qkv = torch.randn((T, 3 * c["kv_heads"], c["dim"]), generator=g, device="cuda",
                          dtype=DTYPES[c["dtype"]])
        s.update(k=qkv[:, c["kv_heads"]:2 * c["kv_heads"]], v=qkv[:, 2 * c["kv_heads"]:],
                 k_pages=_pool(pages, c, g), v_pages=_pool(pages, c, g))
        # runs of tokens on scattered pages; the tail of a padded batch has no slot
        order = torch.randperm(pages, generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        slots = order[t // page] * page + t % page
        s["slots"] = torch.where(t < _live(c), slots, -1)
        return s
    page = c["page"]
    q_lens = _shuffled(_spread(c["q_lo"], c["q_hi"], c["B"], False), g)
    kv_lens = _shuffled(_spread(c["ctx_lo"], c["ctx_hi"], c["B"], True), g) + q_lens
    pages = int(((kv_lens + page - 1) // page).sum()) + 8
    width = -(-(c["ctx_hi"] + c["q_hi"]) // page)
    table, _, _ = _tables(kv_lens, page, width, pages, g)
    T = int(q_lens.sum())
    qkv = torch.randn((T, c["heads"] + 2 * c["kv_heads"], c["dim"]), generator=g, device="cuda",
                      dtype=DTYPES[c["dtype"]])
    # scores of a deviation of 1.5: a few tokens carry most of a row, as in trained heads
    qkv[:, :c["heads"]] *= 1.5
    s.update(q=qkv[:, :c["heads"]], k_pages=_pool(pages, c, g), v_pages=_pool(pages, c, g),
             table=table, kv_lens=kv_lens.to(torch.int32), cu_q=_starts(q_lens))
    return s


def run(state):
    c = state["case"]
    if own:
        import speculative_decoding_rejection_02_gb300 as sv
        if c["op"] == "step":
            r = sv.cache_step(state["held"], state["new"], state["table"], state["free"],
                              state["free_count"], page_size=c["page"],
                              num_tokens=state["tokens"], cu_num_draft=state["cu_draft"],
                              num_accepted=state["accepted"])
            return dict(lens=r.lens, cu_new=r.cu_new, positions=r.positions, slots=r.slots,
                        table=state["table"], free=state["free"], free_count=r.free_count)
        if c["op"] == "append":
            sv.cache_append(state["k"], state["v"], state["slots"], state["k_pages"],
                            state["v_pages"])
            return dict(k_pages=state["k_pages"], v_pages=state["v_pages"])
        out, lse = sv.cache_attend(state["q"], state["k_pages"], state["v_pages"], state["table"],
                                   state["kv_lens"], state["cu_q"], max_q=c["q_hi"],
                                   window=c["window"], sinks=c["sinks"], return_lse=True)
        return dict(out=out, lse=lse)
    if c["op"] == "step":
        return _plain_step(state)
    if c["op"] == "append":
        return _plain_append(state)
    return _plain_attend(state)


def _plain_step(s):
    page, T = s["case"]["page"], s["tokens"]
    table, free, count = s["table"], s["free"], s["free_count"]
    B, width = table.shape
    draft = s["cu_draft"][1:] - s["cu_draft"][:-1]
    kept = s["held"] - (draft - s["accepted"])
    lens = kept + s["new"]
    have, need = (s["held"] + page - 1) // page, (lens + page - 1) // page
    gone, more = (have - need).clamp(min=0), (need - have).clamp(min=0)
    gone_at, more_at = torch.cumsum(gone, 0) - gone, torch.cumsum(more, 0) - more
    total = count + gone.sum()
    col = torch.arange(width, device=table.device)
    # freed pages go on top of the stack in order (requests, then pages) ...
    freed = (col >= need[:, None]) & (col < have[:, None])
    spot = torch.where(freed, count + gone_at[:, None] + col - need[:, None], free.numel())
    stack = torch.cat([free, free.new_zeros(1)])
    stack = stack.scatter(0, spot.reshape(-1).long(), table.reshape(-1))[:-1]
    # ... and new pages come off its top in the same order
    taken = (col >= have[:, None]) & (col < need[:, None])
    spot = total - 1 - (more_at[:, None] + col - have[:, None])
    table = torch.where(taken, stack[torch.where(taken, spot, 0).long()], table)
    cu_new = torch.cat([torch.zeros_like(count), torch.cumsum(s["new"], 0).to(torch.int32)])
    t = torch.arange(T, device=table.device, dtype=torch.int32)
    r = torch.searchsorted(cu_new[1:], t, right=True).clamp(max=B - 1)
    live = t < cu_new[-1]
    pos = torch.where(live, kept[r] + t - cu_new[r], -1)
    slots = table[r, (pos // page).clamp(min=0).long()].long() * page + pos % page
    return dict(lens=lens, cu_new=cu_new, positions=pos.to(torch.int32),
                slots=torch.where(live, slots, -1), table=table, free=stack,
                free_count=(total - more.sum()).to(torch.int32))


def _plain_append(s):
    page = s["case"]["page"]
    live = s["slots"] >= 0
    slots = s["slots"][live]
    s["k_pages"][slots // page, slots % page] = s["k"][live]
    s["v_pages"][slots // page, slots % page] = s["v"][live]
    return dict(k_pages=s["k_pages"], v_pages=s["v_pages"])


def _plain_attend(s):
    c = s["case"]
    page, Q = c["page"], c["q_hi"]
    H, K, D = c["heads"], c["kv_heads"], c["dim"]
    G = H // K
    q, cu = s["q"], s["cu_q"].long()
    T, B = q.shape[0], cu.numel() - 1
    L = s["table"].shape[1] * page
    q_lens, kv_lens = cu[1:] - cu[:-1], s["kv_lens"].long()
    j = torch.arange(L, device=q.device)
    there = j < kv_lens[:, None]
    pages = s["table"][:, j // page].clamp(min=0).long()
    k = s["k_pages"][pages, j % page].float()                       # [B, L, K, D]
    v = s["v_pages"][pages, j % page].float()
    v = torch.where(there[:, :, None, None], v, 0.0)
    i = torch.arange(Q, device=q.device)
    rows = q[(cu[:-1, None] + i).clamp(max=T - 1)].float()          # [B, Q, H, D]
    rows = rows.view(B, Q, K, G, D).permute(0, 2, 3, 1, 4).reshape(B, K, G * Q, D)
    pos = (kv_lens - q_lens)[:, None] + i                           # [B, Q]
    seen = there[:, None, :] & (j <= pos[:, :, None])
    if c["window"]:
        seen &= (j > pos[:, :, None] - c["window"]) | (j < c["sinks"])
    scores = torch.matmul(rows, k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(D))
    scores = scores.view(B, K, G, Q, L).masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, K, G * Q, L), v.permute(0, 2, 1, 3)).view(B, K, G, Q, D)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + torch.log(total))[..., 0]
    t = torch.arange(T, device=q.device)
    r = torch.searchsorted(cu[1:], t, right=True)
    at = t - cu[r]
    out = o.permute(0, 3, 1, 2, 4).reshape(B, Q, H, D)[r, at]
    lse = lse.permute(0, 3, 1, 2).reshape(B, Q, H)[r, at]
    return dict(out=out.to(q.dtype), lse=lse)


def work(case):
    c = case
    if c["op"] == "step":
        B, page = c["B"], c["page"]
        tokens = sum(_spread(c["new_lo"], c["new_hi"], B, False))
        # lengths, offsets and counts in and out; a page and a table entry for each page that
        # is crossed; a table entry, a position and a slot for each token's page and token
        return {"bytes": 4 * (6 * B + 2) + 16 * tokens / page + 12 * B * c["new_hi"] + 4 * B,
                "flops": 0}
    if c["op"] == "append":
        return {"bytes": 8 * c["T"] + 8 * _live(c) * c["kv_heads"] * c["dim"], "flops": 0}
    q_lens = _spread(c["q_lo"], c["q_hi"], c["B"], False)
    ctx = _spread(c["ctx_lo"], c["ctx_hi"], c["B"], True)
    seen = pairs = 0
    for n, L in ((n, x + n) for n, x in zip(q_lens, ctx)):
        if c["window"] and L > c["window"] + c["sinks"] + n:
            seen += c["window"] + c["sinks"] + n - 1
            pairs += n * (c["window"] + c["sinks"])
        else:
            seen += L
            pairs += n * (L - n) + n * (n + 1) // 2
    T = sum(q_lens)
    return {"bytes": 4 * seen * c["kv_heads"] * c["dim"] + T * c["heads"] * (4 * c["dim"] + 4),
            "flops": 4 * pairs * c["heads"] * c["dim"]}


def exact(case, seed):
    c = case
    if c["op"] == "append":
        return None  # copies: nothing is computed
    s = prepare(case, seed)
    if c["op"] == "step":
        return _exact_step(s)
    if 4.0 * c["B"] * c["heads"] * c["dim"] * c["q_hi"] * (c["ctx_hi"] + c["q_hi"]) > 5e12:
        return None
    # request by request and head by head, from the definition
    page, G = c["page"], c["heads"] // c["kv_heads"]
    q, cu, lens = s["q"], s["cu_q"].tolist(), s["kv_lens"].tolist()
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    for b, L in enumerate(lens):
        lo, hi = cu[b], cu[b + 1]
        held = s["table"][b, : -(-L // page)].long()
        ks = s["k_pages"][held].flatten(0, 1)[:L].double()
        vs = s["v_pages"][held].flatten(0, 1)[:L].double()
        at = torch.arange(L - (hi - lo), L, device=q.device)[:, None]
        back = at - torch.arange(L, device=q.device)
        hidden = back < 0
        if c["window"]:
            first = torch.arange(L, device=q.device) < c["sinks"]
            hidden = hidden | ((back >= c["window"]) & ~first)
        for h in range(c["heads"]):
            x = q[lo:hi, h].double() @ ks[:, h // G].T / math.sqrt(c["dim"])
            x = x.masked_fill(hidden, -math.inf)
            lse[lo:hi, h] = torch.logsumexp(x, 1)
            out[lo:hi, h] = torch.softmax(x, 1) @ vs[:, h // G]
    return dict(out=out, lse=lse)


def _exact_step(s):
    page, T = s["case"]["page"], s["tokens"]
    held, new, acc = s["held"].tolist(), s["new"].tolist(), s["accepted"].tolist()
    cu, table, stack = s["cu_draft"].tolist(), s["table"].tolist(), s["free"].tolist()
    n = int(s["free_count"])
    kept = [h - (cu[r + 1] - cu[r] - acc[r]) for r, h in enumerate(held)]
    have = [-(-h // page) for h in held]
    need = [-(-(k + m) // page) for k, m in zip(kept, new)]
    for r in range(len(held)):
        for x in range(need[r], have[r]):
            stack[n] = table[r][x]
            n += 1
    for r in range(len(held)):
        for x in range(have[r], need[r]):
            n -= 1
            table[r][x] = stack[n]
    pos, slots, starts = [], [], [0]
    for r, m in enumerate(new):
        for p in range(kept[r], kept[r] + m):
            pos.append(p)
            slots.append(table[r][p // page] * page + p % page)
        starts.append(len(pos))
    pad = [-1] * (T - len(pos))
    i32 = dict(dtype=torch.int32)
    return dict(lens=torch.tensor([k + m for k, m in zip(kept, new)], **i32),
                cu_new=torch.tensor(starts, **i32), positions=torch.tensor(pos + pad, **i32),
                slots=torch.tensor(slots + pad, dtype=torch.int64),
                table=torch.tensor(table, **i32), free=torch.tensor(stack, **i32),
                free_count=torch.tensor([n], **i32))
