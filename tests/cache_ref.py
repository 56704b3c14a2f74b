"""Plain forms, in 64 bits or whole numbers, of the paged-cache operators, the
makers of their test inputs, and the error bounds of the attention."""
import math

import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a spacing at 1


def step(held, new, table, free, count, page, tokens, drafts=None, accepted=None):
    """spec_cache_step on lists; returns a dict, or None where it refuses."""
    table, free = [list(r) for r in table], list(free)
    B, width = len(held), len(table[0]) if table else 0
    gone = [0] * B if drafts is None else [d - a for d, a in zip(drafts, accepted)]
    kept = [h - x for h, x in zip(held, gone)]
    lens = [k + n for k, n in zip(kept, new)]
    have, need = [-(-h // page) for h in held], [-(-x // page) for x in lens]
    if any(x < 0 for x in held + new + kept) or any(x > width for x in have + need):
        return None
    if drafts is not None and any(not 0 <= a <= d for d, a in zip(drafts, accepted)):
        return None
    if sum(new) > tokens:
        return None
    for r in range(B):
        for c in range(need[r], have[r]):
            if count >= len(free):
                return None
            free[count] = table[r][c]
            count += 1
    if sum(max(0, n - h) for n, h in zip(need, have)) > count:
        return None
    for r in range(B):
        for c in range(have[r], need[r]):
            count -= 1
            table[r][c] = free[count]
    cu, pos, slots = [0], [], []
    for r in range(B):
        for p in range(kept[r], lens[r]):
            pos.append(p)
            slots.append(table[r][p // page] * page + p % page)
        cu.append(len(pos))
    pad = [-1] * (tokens - len(pos))
    return dict(lens=lens, cu_new=cu, positions=pos + pad, slots=slots + pad, table=table,
                free=free, free_count=count)


def cache(lens, page, kv_heads, dim, dtype, g, layout="token", spare=3, rubbish=float("nan")):
    """Pages holding random keys and values of requests of these lengths, in
    scattered order; every other slot, and every page that no request holds, is
    `rubbish`. Returns k_pages, v_pages, table, and the dense keys and values."""
    held = [-(-n // page) for n in lens]
    pages = sum(held) + spare
    width = max(held + [1]) + 2
    order = torch.randperm(pages, generator=g).tolist()
    table = torch.full((max(len(lens), 1), width), -1, dtype=torch.int32)[: len(lens)]
    kp = torch.full((pages, page, kv_heads, dim), rubbish, dtype=dtype)
    vp = torch.full((pages, page, kv_heads, dim), rubbish, dtype=dtype)
    ks, vs = [], []
    for r, n in enumerate(lens):
        k = torch.randn((n, kv_heads, dim), generator=g).to(dtype)
        v = torch.randn((n, kv_heads, dim), generator=g).to(dtype)
        ks.append(k)
        vs.append(v)
        for c in range(held[r]):
            x = order.pop()
            table[r, c] = x
            part = k[c * page: (c + 1) * page]
            kp[x, : len(part)] = part
            vp[x, : len(part)] = v[c * page: (c + 1) * page]
    if layout == "head":
        kp = kp.transpose(1, 2).contiguous().transpose(1, 2)
        vp = vp.transpose(1, 2).contiguous().transpose(1, 2)
    return kp, vp, table, ks, vs


def visible(n_q, n_kv, window, sinks):
    """[n_q, n_kv] truth values."""
    pos = torch.arange(n_kv - n_q, n_kv)[:, None]
    j = torch.arange(n_kv)[None, :]
    see = j <= pos
    if window:
        see = see & ((pos - j < window) | (j < sinks))
    return see


def attend(q, ks, vs, q_lens, scale=None, window=0, sinks=0):
    """Attention in 64 bits. Returns out, lse and the bounds of their errors.

    With u the rounding unit of the type (half a spacing at 1), e = 2^-24, D the
    head size, n the visible tokens and A = sum_j p_j |v_j|:
      a score is a D-term fp32 sum, off by at most ds = (D + 3) e scale sum |q||k|,
      plus two roundings of the scaled exponent (4 e |s|), and the exponential
      is good to 2^-22; so each weight is off by w = 2 ds + 8 e |s| + 2^-21 of
      itself, its rounding to the type adds u, and a weight below the type's
      least normal value is off by at most 2^-24 of the row's largest;
      the sums over n tokens add n e each; the final rounding adds u.
    """
    T, H, D = q.shape
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    u, e = UNIT[q.dtype], 2.0 ** -24
    out = torch.zeros((T, H, D), dtype=torch.float64)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    t0 = 0
    for n_q, k, v in zip(q_lens, ks, vs):
        n, K = k.shape[0], k.shape[1]
        G = H // K
        see = visible(n_q, n, window, sinks)
        for h in range(H):
            if n == 0 or n_q == 0:
                break
            kh, vh = k[:, h // G].double(), v[:, h // G].double()
            x = q[t0: t0 + n_q, h].double()
            s = (x @ kh.T * scale).masked_fill(~see, -math.inf)
            size = (x.abs() @ kh.abs().T * abs(scale)).masked_fill(~see, 0.0)
            some = see.any(1)
            lse[t0: t0 + n_q, h] = torch.logsumexp(s, 1)
            p = torch.where(some[:, None], torch.softmax(s, 1), torch.zeros(()).double())
            dead = ~see.any(0)
            vh = vh.masked_fill(dead[:, None], 0.0)  # what no row sees may be anything
            out[t0: t0 + n_q, h] = p @ vh
            A = p @ vh.abs()
            ds = ((D + 3) * e * size.amax(1) + 8 * e * s.masked_fill(~see, 0.0).abs().amax(1))
            w = 2 * ds + 2.0 ** -21 + 2 * n * e
            low = 2.0 ** -24 * n * p.amax(1, keepdim=True) * vh.abs().amax(0)
            out_tol[t0: t0 + n_q, h] = (2 * u + w[:, None]) * A + low + 1e-30
            lse_tol[t0: t0 + n_q, h] = ds + 2.0 ** -21 + n * e + torch.where(
                some, 4 * e * lse[t0: t0 + n_q, h].abs(), 0.0)
        t0 += n_q
    return out, lse, out_tol, lse_tol


def assert_attend(got, got_lse, want):
    out, lse, out_tol, lse_tol = want
    got, got_lse = got.double().cpu(), got_lse.double().cpu()
    none = torch.isinf(lse)
    assert torch.equal(none, torch.isinf(got_lse)), "rows that see nothing"
    assert torch.equal(got_lse[none], lse[none])
    assert not torch.isnan(got).any() and not torch.isnan(got_lse).any()
    assert (got[none] == 0).all()
    off = ((got_lse - lse).abs() - lse_tol)[~none]
    assert off.numel() == 0 or off.max() <= 0, ("lse", float(off.max()))
    off = (got - out).abs() - out_tol
    assert off.numel() == 0 or off.max() <= 0, ("out", float(off.max()), int(off.argmax()))
