"""Operators that keep a long paged cache affordable, as measured work.

Two ways of reading and holding less of a cache of many tokens:

Sparse attention over the pages that a cheap score selects for each query token:
  bounds    the least and the largest key of every channel, for each page and head;
  score     for each token, kv head and page an upper bound of its keys' scores, from
            the bounds alone;
  select    the pages of the highest scores, beside the first and the last ones;
  attend    attention over the selected pages.
Eviction by accumulated attention weight:
  weigh     add to every cached token the softmax weights that this round's queries
            gave it;
  evict     keep the tokens of the highest weights of every request and head, beside
            the first and the last ones, close the gaps and give pages back.

``run`` computes each in its plain form (elementary torch operations in 32 bits), or,
where ``own`` is true, through this package's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    wide = dict(heads=32, kv_heads=8, dim=128, dtype="bf16", layout="token")
    return [
        # After a verification round's append: the pages that its tokens were written to.
        dict(name="bounds_round", op="bounds", B=128, q_lo=2, q_hi=8, ctx_lo=150, ctx_hi=9000,
             page=16, fresh=True, **wide),
        # Whole prompts (or what an eviction left), heads outside the tokens.
        dict(name="bounds_prompt", op="bounds", B=4, q_lo=1, q_hi=1, ctx_lo=9001, ctx_hi=16000,
             page=64, fresh=False, **dict(wide, dtype="fp16", layout="head")),
        # One request, one token, a long context: latency.
        dict(name="score_one", op="score", B=1, q_lo=1, q_hi=1, ctx_lo=130001, ctx_hi=130001,
             page=32, **wide),
        # A verification round: the last token and up to seven drafts per request.
        dict(name="score_verify", op="score", B=64, q_lo=2, q_hi=8, ctx_lo=1000, ctx_hi=30000,
             page=16, **wide),
        # The lists of the same round.
        dict(name="select_verify", op="select", B=64, q_lo=2, q_hi=8, ctx_lo=1000, ctx_hi=30000,
             page=16, count=128, first=1, recent=2, **wide),
        # Few requests with long documents: long rows.
        dict(name="select_long", op="select", B=2, q_lo=5, q_hi=5, ctx_lo=190000, ctx_hi=200000,
             page=16, count=250, first=0, recent=1, **dict(wide, heads=28, kv_heads=4)),
        # One request, one token, some 2000 of 32000 tokens: latency.
        dict(name="attend_one", op="attend", B=1, q_lo=1, q_hi=1, ctx_lo=32001, ctx_hi=32001,
             page=32, count=64, **wide),
        # A verification round over 2048 selected tokens for each row.
        dict(name="attend_verify", op="attend", B=64, q_lo=2, q_hi=8, ctx_lo=1000, ctx_hi=30000,
             page=16, count=128, **wide),
        # The weights of a verification round over whole contexts.
        dict(name="weigh_verify", op="weigh", B=64, q_lo=2, q_hi=8, ctx_lo=1000, ctx_hi=30000,
             page=32, decay=1.0, **wide),
        # Prompt chunks over what is cached already.
        dict(name="weigh_chunk", op="weigh", B=2, q_lo=2048, q_hi=2048, ctx_lo=11000,
             ctx_hi=14000, page=64, decay=1.0, **wide),
        # A decoding batch that goes back to its budget of 2048 tokens.
        dict(name="evict_round", op="evict", B=64, q_lo=1, q_hi=1, ctx_lo=1990, ctx_hi=2500,
             page=16, keep=2048, first=4, recent=64, **wide),
        # Long prompts cut down to a few thousand tokens once, smaller heads.
        dict(name="evict_prompt", op="evict", B=3, q_lo=1, q_hi=1, ctx_lo=20001, ctx_hi=33000,
             page=32, keep=4096, first=16, recent=512,
             **dict(wide, heads=28, kv_heads=4, dim=64, dtype="fp16", layout="head")),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["bounds", "score", "select", "attend", "weigh", "evict"])
    tops = [_cost(c) for c in listed() if c["op"] == op]
    top = [max(x) for x in zip(*tops)]
    while True:
        kv_heads = rng.choice([1, 2, 4, 5, 8])
        hi = _log_int(rng, 20, 200000)
        q_hi = _log_int(rng, 1, {"weigh": 2048, "evict": 1, "bounds": 2048}.get(op, 64))
        c = dict(op=op, B=_log_int(rng, 1, 128), q_lo=rng.randint(1, q_hi), q_hi=q_hi,
                 ctx_lo=rng.randint(1, hi), ctx_hi=hi, page=rng.choice([8, 16, 32, 64]),
                 heads=kv_heads * rng.choice([1, 2, 3, 4, 7, 8]), kv_heads=kv_heads,
                 dim=rng.choice([64, 80, 96, 128]), dtype=rng.choice(["bf16", "fp16"]),
                 layout=rng.choice(["token", "head"]))
        if op == "bounds":
            c["fresh"] = rng.random() < 0.5
        if op in ("select", "attend"):
            c["count"] = _log_int(rng, 2, 300)
        if op == "select":
            c["first"] = rng.randint(0, min(4, c["count"] - 1))
            c["recent"] = rng.randint(0, min(8, c["count"] - c["first"]))
        if op == "weigh":
            c["decay"] = rng.choice([1.0, 1.0, 0.9, 0.0])
        if op == "evict":
            c["keep"] = _log_int(rng, 1, hi)
            c["first"] = rng.randint(0, min(64, c["keep"]))
            c["recent"] = rng.randint(0, min(512, c["keep"] - c["first"]))
        if all(x <= y for x, y in zip(_cost(c), top)):
            return c


def _cost(c):
    """What a case goes through in its padded plain form: elements of the keys, and of the
    scores or gathered rows."""
    L = c["ctx_hi"] + c["q_hi"]
    kv = c["B"] * L * c["kv_heads"] * c["dim"]
    rows = c["B"] * c["q_hi"] * c["heads"]
    if c["op"] == "attend":
        return kv, rows * c["count"] * c["page"] * c["dim"]
    if c["op"] in ("score", "select"):
        return kv, rows * (L // c["page"] + 1)
    return kv, rows * L if c["op"] == "weigh" else 0


def _spread(lo, hi, n, log):
    """n whole numbers from lo to hi at even steps (of the logarithm)."""
    at = [(i + 0.5) / n for i in range(n)]
    if log:
        return [int(lo * (hi / lo) ** x) for x in at]
    return [int(lo + x * (hi + 1 - lo)) for x in at]


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


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    B, page, K, D, dt = c["B"], c["page"], c["kv_heads"], c["dim"], DTYPES[c["dtype"]]
    q_lens = _shuffled(_spread(c["q_lo"], c["q_hi"], B, False), g)
    kv_lens = _shuffled(_spread(c["ctx_lo"], c["ctx_hi"], B, True), g) + q_lens
    held = (kv_lens + page - 1) // page
    used = int(held.sum())
    # the same number of pages for every seed
    most = sum(_spread(c["ctx_lo"], c["ctx_hi"], B, True))
    most += sum(_spread(c["q_lo"], c["q_hi"], B, False))
    pages = most // page + B + 8
    width = -(-(c["ctx_hi"] + c["q_hi"]) // page)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    at = (torch.cumsum(held, 0) - held)[:, None] + col
    table = torch.where(col < held[:, None], order[at.clamp(max=pages - 1)], -1).contiguous()
    T = int(q_lens.sum())
    s = dict(case=c, kv_lens=kv_lens.to(torch.int32), cu_q=_starts(q_lens), table=table, T=T)
    if c["op"] in ("score", "attend", "weigh"):
        # the new tokens of a fused projection: q, k and v side by side; scores of a
        # deviation of 1.5, so that a few tokens carry most of a row, as in trained heads
        qkv = torch.randn((T, c["heads"] + 2 * K, D), generator=g, device="cuda", dtype=dt)
        s["q"] = qkv[:, :c["heads"]]
        s["q"] *= 1.5
    if c["op"] in ("bounds", "attend", "weigh", "evict"):
        s["k_pages"] = _pool(pages, c, g)
    if c["op"] in ("attend", "evict"):
        s["v_pages"] = _pool(pages, c, g)
    if c["op"] == "bounds":
        s["bounds"] = torch.zeros((pages, K, 2, D), device="cuda", dtype=dt)
    if c["op"] == "score":
        # the extremes of a page's keys, about two deviations out, around the page's mean
        mid, off = _randn(g, pages, K, 1, D) * 0.5, _randn(g, pages, K, 2, D).abs() + 1.0
        off[:, :, 0] *= -1.0
        s["bounds"] = (mid + off).to(dt)
    if c["op"] == "select":
        s["scores"] = _likings(c, s, g) * 40.0
    if c["op"] == "attend":
        s["selected"] = _lists(c, s, g)
    if c["op"] == "weigh":
        # sums of earlier rounds; the slots of the new tokens hold those of earlier owners
        s["weights"] = torch.exp(2.0 * _randn(g, pages, K, page))
        s["lse"] = _lse(s)
    if c["op"] == "evict":
        w = torch.exp(2.0 * _randn(g, pages, K, page))
        # tokens that no query has looked at
        gone = torch.rand(w.shape, generator=g, device="cuda") < 0.1
        s["weights"] = torch.where(gone, 0.0, w)
        free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
        free[: pages - used] = order[used:]
        s.update(budget=torch.full((B,), c["keep"], dtype=torch.int32, device="cuda"), free=free,
                 free_count=torch.tensor([pages - used], dtype=torch.int32, device="cuda"))
    return s


def _rows(s):
    """The request and the position of every new token."""
    cu = s["cu_q"].long()
    t = torch.arange(s["T"], device=cu.device)
    r = torch.searchsorted(cu[1:], t, right=True)
    return r, s["kv_lens"].long()[r] - cu[r + 1] + t


def _likings(c, s, g):
    """[T, kv_heads, width]: how well each page suits each token; a request's tokens mostly
    agree."""
    r, _ = _rows(s)
    W = s["table"].shape[1]
    x = _randn(g, c["B"], c["kv_heads"], W)[r]
    return x + 0.5 * _randn(g, r.numel(), c["kv_heads"], W)


def _lists(c, s, g):
    """Ascending columns of the best pages of each token, the first and its own among them,
    -1 past the last."""
    x = _likings(c, s, g)
    _, pos = _rows(s)
    W = x.shape[2]
    own_page = (pos // c["page"])[:, None, None]
    col = torch.arange(W, device=x.device)
    x = torch.where((col == own_page) | (col == 0), math.inf, x)
    x = torch.where(col > own_page, -math.inf, x)
    n = min(c["count"], W)
    top, at = torch.topk(x, n, dim=2)
    at = torch.where(top > -math.inf, at, W).sort(2).values
    out = torch.full((*x.shape[:2], c["count"]), -1, dtype=torch.int32, device=x.device)
    out[:, :, :n] = torch.where(at < W, at, -1).to(torch.int32)
    return out


def _lse(s):
    """The logarithms [T, heads] of the attention's sums, as the attention over the whole
    cache gives them."""
    c = s["case"]
    G, D = c["heads"] // c["kv_heads"], c["dim"]
    cu, lens = s["cu_q"].tolist(), s["kv_lens"].tolist()
    lse = torch.empty(s["q"].shape[:2], device="cuda")
    for b, L in enumerate(lens):
        lo, hi = cu[b], cu[b + 1]
        k = s["k_pages"][s["table"][b, : -(-L // c["page"])].long()].flatten(0, 1)[:L].float()
        q = s["q"][lo:hi].float().view(hi - lo, c["kv_heads"], G, D).permute(1, 2, 0, 3)
        x = torch.matmul(q.reshape(c["kv_heads"], -1, D), k.permute(1, 2, 0)) / math.sqrt(D)
        x = x.view(c["kv_heads"], G, hi - lo, L)
        pos = torch.arange(L - hi + lo, L, device="cuda")[:, None]
        x.masked_fill_(torch.arange(L, device="cuda") > pos, -math.inf)
        lse[lo:hi] = torch.logsumexp(x, 3).permute(2, 0, 1).reshape(hi - lo, -1)
    return lse


def run(state):
    s, c = state, state["case"]
    if not own:
        return _PLAIN[c["op"]](s)
    import speculative_decoding_rejection_02_gb300 as sv
    if c["op"] == "bounds":
        sv.cache_bounds(s["k_pages"], s["table"], s["kv_lens"], s["bounds"],
                        cu_q=s["cu_q"] if c["fresh"] else None,
                        max_q=c["q_hi"] if c["fresh"] else None)
        return s["bounds"]
    if c["op"] == "score":
        return sv.cache_score(s["q"], s["bounds"], s["table"], s["kv_lens"], s["cu_q"],
                              page_size=c["page"], max_q=c["q_hi"])
    if c["op"] == "select":
        return sv.cache_select(s["scores"], s["kv_lens"], s["cu_q"], page_size=c["page"],
                               count=c["count"], first=c["first"], recent=c["recent"])
    if c["op"] == "attend":
        out, lse = sv.cache_attend_selected(s["q"], s["k_pages"], s["v_pages"], s["table"],
                                            s["kv_lens"], s["cu_q"], s["selected"],
                                            return_lse=True)
        return dict(out=out, lse=lse)
    if c["op"] == "weigh":
        sv.cache_weigh(s["q"], s["k_pages"], s["table"], s["kv_lens"], s["cu_q"], s["lse"],
                       s["weights"], max_q=c["q_hi"], decay=c["decay"])
        return s["weights"]
    r = sv.cache_evict(s["k_pages"], s["v_pages"], s["weights"], s["table"], s["kv_lens"],
                       s["budget"], s["free"], s["free_count"], first=c["first"],
                       recent=c["recent"])
    return dict(lens=r.lens, free_count=r.free_count, k_pages=s["k_pages"], v_pages=s["v_pages"],
                weights=s["weights"], free=s["free"])


def _plain_bounds(s):
    page, lens = s["case"]["page"], s["kv_lens"].long()
    cu = s["cu_q"].long()
    since = lens - (cu[1:] - cu[:-1]) if s["case"]["fresh"] else torch.zeros_like(lens)
    col = torch.arange(s["table"].shape[1], device=lens.device)
    b, x = torch.nonzero((col >= (since // page)[:, None]) & (col * page < lens[:, None]),
                         as_tuple=True)
    pages = s["table"][b, x].long()
    k = s["k_pages"][pages].float()                                  # [n, page, K, D]
    there = x[:, None] * page + torch.arange(page, device=x.device) < lens[b][:, None]
    there = there[:, :, None, None]
    low = torch.where(there, k, math.inf).amin(1)
    high = torch.where(there, k, -math.inf).amax(1)
    s["bounds"][pages] = torch.stack([low, high], 2).to(s["bounds"].dtype)
    return s["bounds"]


def _padded(s):
    """q as [B, kv_heads, G, most new tokens, dim] in 32 bits, and their positions."""
    c = s["case"]
    cu, lens = s["cu_q"].long(), s["kv_lens"].long()
    i = torch.arange(c["q_hi"], device=cu.device)
    rows = s["q"][(cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)].float()
    rows = rows.view(*rows.shape[:2], c["kv_heads"], -1, c["dim"]).permute(0, 2, 3, 1, 4)
    return rows, (lens - cu[1:] + cu[:-1])[:, None] + i


def _plain_score(s):
    c = s["case"]
    page, W = c["page"], s["table"].shape[1]
    col = torch.arange(W, device="cuda")
    held = col * page < s["kv_lens"][:, None]
    bounds = s["bounds"][torch.where(held, s["table"], 0).long()].float()  # [B, W, K, 2, D]
    rows, _ = _padded(s)
    up, down = rows.clamp(min=0).sum(2), rows.clamp(max=0).sum(2)          # [B, K, Q, D]
    x = torch.matmul(up, bounds[:, :, :, 1].permute(0, 2, 3, 1))
    x += torch.matmul(down, bounds[:, :, :, 0].permute(0, 2, 3, 1))        # [B, K, Q, W]
    r, pos = _rows(s)
    x = x[r, :, torch.arange(r.numel(), device="cuda") - s["cu_q"].long()[r]]
    return torch.where(col * page <= pos[:, None, None], x, -math.inf)


def _plain_select(s):
    c = s["case"]
    x, n = s["scores"], c["count"]
    _, pos = _rows(s)
    W = x.shape[2]
    col = torch.arange(W, device=x.device)
    own_page = (pos // c["page"])[:, None, None]
    # pages that the token does not see, then the others, then those that are always kept;
    # within each the highest score, within that the lowest column
    rank = (col <= own_page).int()
    always = (col < c["first"]) | (col > own_page - c["recent"])
    rank = torch.where(always & (rank > 0), 2, rank).expand(x.shape)
    by_score = torch.sort(torch.where(x.isnan(), math.inf, x), dim=2, descending=True,
                          stable=True).indices
    by_rank = torch.sort(rank.gather(2, by_score), dim=2, descending=True, stable=True)
    best = torch.where(by_rank.values > 0, by_score.gather(2, by_rank.indices), W)[:, :, :n]
    best = best.sort(2).values
    out = torch.full((*x.shape[:2], n), -1, dtype=torch.int32, device=x.device)
    out[:, :, : best.shape[2]] = torch.where(best < W, best, -1).to(torch.int32)
    return out


def _plain_attend(s):
    c = s["case"]
    page, K, D = c["page"], c["kv_heads"], c["dim"]
    G, n = c["heads"] // K, c["count"] * page
    r, pos = _rows(s)
    T = r.numel()
    out = torch.empty((T, K, G, D), dtype=s["q"].dtype, device="cuda")
    lse = torch.empty((T, K, G), device="cuda")
    head = torch.arange(K, device="cuda")[:, None]
    off = torch.arange(page, device="cuda")
    step = max(1, 2 ** 29 // (K * n * D))
    for t in range(0, T, step):
        at = slice(t, t + step)
        sel = s["selected"][at].long()                                     # [t, K, count]
        j = (sel[..., None] * page + off).flatten(2)                       # [t, K, n]
        seen = (sel >= 0)[..., None].expand(*sel.shape, page).flatten(2)
        seen = seen & (j <= pos[at][:, None, None])
        where = torch.where(seen, j, 0)
        pages = s["table"][r[at][:, None, None], where // page].long()
        k = s["k_pages"][pages, where % page, head].float()
        v = s["v_pages"][pages, where % page, head].float()
        q = s["q"][at].float().view(-1, K, G, D)
        x = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(D))
        x = x.masked_fill(~seen[:, :, None], -math.inf)
        top = x.amax(3, keepdim=True)
        top = torch.where(torch.isfinite(top), top, 0.0)
        p = torch.exp(x - top)
        total = p.sum(3, keepdim=True)
        o = torch.matmul(p, torch.where(seen[..., None], v, 0.0))
        out[at] = torch.where(total > 0, o / total, 0.0).to(out.dtype)
        lse[at] = (top + torch.log(total))[..., 0]
    return dict(out=out.view(T, -1, D), lse=lse.view(T, -1))


def _plain_weigh(s):
    c = s["case"]
    page, K, D, Q = c["page"], c["kv_heads"], c["dim"], c["q_hi"]
    G, B = c["heads"] // K, c["B"]
    lens, cu = s["kv_lens"].long(), s["cu_q"].long()
    new = cu[1:] - cu[:-1]
    L = s["table"].shape[1] * page
    j = torch.arange(L, device="cuda")
    there = j < lens[:, None]
    pages = s["table"][:, j // page].clamp(min=0).long()
    k = s["k_pages"][pages, j % page].float()                              # [B, L, K, D]
    rows, pos = _padded(s)
    x = torch.matmul(rows.reshape(B, K, G * Q, D), k.permute(0, 2, 3, 1))
    x = x.view(B, K, G, Q, L).mul_(1.0 / math.sqrt(D))
    i = torch.arange(Q, device="cuda")
    lse = s["lse"][(cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)]     # [B, Q, H]
    x -= lse.view(B, Q, K, G).permute(0, 2, 3, 1)[..., None]
    seen = (j <= pos[:, :, None]) & (i < new[:, None])[:, :, None]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    given = x.exp_().sum((2, 3))                                           # [B, K, L]
    b, j = torch.nonzero(there, as_tuple=True)
    at, off = pages[b, j], j % page
    before = s["weights"][at, :, off] * c["decay"]
    before = torch.where((j < (lens - new)[b])[:, None], before, 0.0)
    s["weights"][at, :, off] = before + given[b, :, j]
    return s["weights"]


def _plain_evict(s):
    c = s["case"]
    page, K = c["page"], c["kv_heads"]
    table, lens = s["table"], s["kv_lens"].long()
    B, width = table.shape
    L = width * page
    least = torch.minimum(lens, torch.full_like(lens, c["first"] + c["recent"]))
    kept = torch.minimum(lens, torch.maximum(s["budget"].long(), least))
    j = torch.arange(L, device="cuda")
    pages = table[:, j // page].clamp(min=0).long()
    w = s["weights"][pages, :, j % page].transpose(1, 2)                   # [B, K, L]
    n = lens[:, None, None]
    rank = torch.where((j < c["first"]) | (j >= n - c["recent"]), 2, 1)
    rank = torch.where(j < n, rank, 0).expand(w.shape)
    by_weight = torch.sort(torch.where(w.isnan(), math.inf, w), dim=2, descending=True,
                           stable=True).indices
    by_rank = torch.sort(rank.gather(2, by_weight), dim=2, descending=True, stable=True).indices
    best = by_weight.gather(2, by_rank)
    # the kept tokens in their old order
    src = torch.where(j < kept[:, None, None], best, L).sort(2).values
    b, h, i = torch.nonzero((j < kept[:, None, None]) & (src != j), as_tuple=True)
    src = src[b, h, i]
    old, new = pages[b, src], pages[b, i]
    for x in (s["k_pages"], s["v_pages"]):
        x[new, i % page, h] = x[old, src % page, h]
    s["weights"][new, h, i % page] = s["weights"][old, h, src % page]
    # pages past the kept tokens go on top of the stack, in order of requests and pages
    col = torch.arange(width, device="cuda")
    freed = (col * page < lens[:, None]) & (col * page >= kept[:, None])
    back = table[freed]
    spot = s["free_count"] + torch.arange(back.numel(), device="cuda")
    s["free"][spot] = back
    return dict(lens=kept.to(torch.int32),
                free_count=(s["free_count"] + back.numel()).to(torch.int32),
                k_pages=s["k_pages"], v_pages=s["v_pages"], weights=s["weights"],
                free=s["free"])


_PLAIN = dict(bounds=_plain_bounds, score=_plain_score, select=_plain_select,
              attend=_plain_attend, weigh=_plain_weigh, evict=_plain_evict)


def work(case):
    c = case
    page, K, D, H = c["page"], c["kv_heads"], c["dim"], c["heads"]
    q_lens = _spread(c["q_lo"], c["q_hi"], c["B"], False)
    lens = [x + n for x, n in zip(_spread(c["ctx_lo"], c["ctx_hi"], c["B"], True), q_lens)]
    T = sum(q_lens)
    row = 2 * K * D  # bytes of a token's keys
    pages = [-(-n // page) for n in lens]
    if c["op"] == "bounds":
        if c["fresh"]:
            seen = sum(n - (n - q) // page * page for n, q in zip(lens, q_lens))
            pages = [p - (n - q) // page for p, n, q in zip(pages, lens, q_lens)]
        else:
            seen = sum(lens)
        return {"bytes": row * seen + 2 * row * sum(pages), "flops": 2 * seen * K * D}
    if c["op"] == "score":
        pairs = sum(p * n for p, n in zip(pages, q_lens))
        return {"bytes": 2 * row * sum(pages) + 2 * T * H * D + 4 * pairs * K,
                "flops": 4 * pairs * K * D}
    if c["op"] == "select":
        pairs = sum(p * n for p, n in zip(pages, q_lens))
        return {"bytes": 4 * K * (pairs + T * c["count"]), "flops": pairs * K}
    if c["op"] == "attend":
        pairs = sum(n * min(c["count"] * page, L) for n, L in zip(q_lens, lens))
        # a request's tokens mostly agree: the pages of one of them, read once
        seen = sum(min(c["count"] * page, L) for L in lens)
        return {"bytes": 2 * row * seen + T * H * (4 * D + 4) + 4 * T * K * c["count"],
                "flops": 4 * pairs * H * D}
    if c["op"] == "weigh":
        pairs = sum(n * (L - n) + n * (n + 1) // 2 for n, L in zip(q_lens, lens))
        return {"bytes": (row + 8 * K) * sum(lens) + T * H * (2 * D + 4),
                "flops": 2 * pairs * H * D}
    kept = [min(n, max(c["keep"], c["first"] + c["recent"])) for n in lens]
    # tokens before the first one that goes stay where they are: those always kept, and on
    # average one of as many equal parts of the others as go, and one more
    stay = c["first"] + c["recent"]
    moved = sum(k - c["first"] - (n - stay) / (n - k + 1) for k, n in zip(kept, lens) if n > k)
    weights = sum(n for k, n in zip(kept, lens) if n > k)
    return {"bytes": 2 * (2 * row + 4 * K) * moved + 4 * K * weights, "flops": 0}


def exact(case, seed):
    c = case
    if c["op"] in ("bounds", "evict"):
        return None  # copies and comparisons: nothing is computed
    page, K, D = c["page"], c["kv_heads"], c["dim"]
    G = c["heads"] // K
    L = c["ctx_hi"] + c["q_hi"]
    cost = 2.0 * c["B"] * c["heads"] * D * c["q_hi"]
    if cost * dict(score=L / page, select=L / page, weigh=L).get(c["op"], 0) > 3e12 or (
            c["op"] == "attend" and c["B"] * c["q_hi"] * K > 12000):
        return None
    s = prepare(case, seed)
    cu, lens = s["cu_q"].tolist(), s["kv_lens"].tolist()
    T = cu[-1]
    own_pos = [n - cu[b + 1] + t for b, n in enumerate(lens) for t in range(cu[b], cu[b + 1])]
    if c["op"] == "select":
        rows = s["scores"].tolist()
        out = torch.full((T, K, c["count"]), -1, dtype=torch.int32)
        for t, p in enumerate(own_pos):
            n = p // page + 1
            for h in range(K):
                always = set(range(min(c["first"], n))) | set(range(max(0, n - c["recent"]), n))
                rest = [x for x in range(n) if x not in always]
                best = sorted(rest, key=lambda x, v=rows[t][h]: -v[x])
                got = sorted([*always, *best[: max(0, c["count"] - len(always))]])
                out[t, h, : len(got)] = torch.tensor(got, dtype=torch.int32)
        return out
    q = s["q"].double()
    if c["op"] == "score":
        out = torch.full((T, K, s["table"].shape[1]), -math.inf, dtype=torch.float64,
                         device="cuda")
        for b in range(c["B"]):
            n = -(-lens[b] // page)
            bounds = s["bounds"][s["table"][b, :n].long()].double()
            for t in range(cu[b], cu[b + 1]):
                n = own_pos[t] // page + 1
                for h in range(K):
                    x = q[t, h * G:(h + 1) * G, None] * bounds[None, :n, h, 0]
                    y = q[t, h * G:(h + 1) * G, None] * bounds[None, :n, h, 1]
                    out[t, h, :n] = torch.maximum(x, y).sum((0, 2))
        return out
    if c["op"] == "attend":
        out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
        lists = s["selected"].tolist()
        for b in range(c["B"]):
            held = s["table"][b, : -(-lens[b] // page)].long()
            ks = s["k_pages"][held].flatten(0, 1).transpose(0, 1)
            vs = s["v_pages"][held].flatten(0, 1).transpose(0, 1)
            for t in range(cu[b], cu[b + 1]):
                for h in range(K):
                    j = [x * page + y for x in lists[t][h] if x >= 0 for y in range(page)]
                    j = torch.tensor([x for x in j if x <= own_pos[t]], device="cuda")
                    x = ks[h, j].double() @ q[t, h * G:(h + 1) * G].T / math.sqrt(D)
                    lse[t, h * G:(h + 1) * G] = torch.logsumexp(x, 0)
                    out[t, h * G:(h + 1) * G] = torch.softmax(x, 0).T @ vs[h, j].double()
        return dict(out=out, lse=lse)
    weights = s["weights"].double()
    for b, L in enumerate(lens):
        lo, hi = cu[b], cu[b + 1]
        old = L - (hi - lo)
        held = s["table"][b, : -(-L // page)].long()
        at = torch.arange(L, device="cuda")
        hidden = at > torch.arange(old, L, device="cuda")[:, None]
        ks = s["k_pages"][held].flatten(0, 1)[:L]
        for h in range(K):
            kh = ks[:, h].double()
            given = torch.zeros(L, dtype=torch.float64, device="cuda")
            for x in range(h * G, (h + 1) * G):
                y = q[lo:hi, x] @ kh.T / math.sqrt(D) - s["lse"][lo:hi, x, None].double()
                given += torch.exp(y.masked_fill(hidden, -math.inf)).sum(0)
            before = weights[held[at // page], h, at % page] * c["decay"]
            weights[held[at // page], h, at % page] = torch.where(at < old, before, 0.0) + given
    return weights
