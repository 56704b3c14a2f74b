"""Plain forms, in 64 bits or whole numbers, of the sparse-attention and eviction operators of
the paged cache, and the bounds of their errors. Caches and dense keys come from
cache_ref.cache; everything is on the CPU."""
import math

import torch

from cache_ref import UNIT

EPS = 2.0 ** -24  # fp32's rounding


def positions(q_lens, kv_lens):
    """The request and the position of every new token."""
    return [(r, n - m + i) for r, (m, n) in enumerate(zip(q_lens, kv_lens)) for i in range(m)]


def bounds(ks, page):
    """Per request the least and largest key of each page: [pages, kv_heads, 2, dim]."""
    out = []
    for k in ks:
        parts = [k[c: c + page] for c in range(0, k.shape[0], page)]
        out.append([torch.stack([p.amin(0), p.amax(0)], 1) for p in parts])
    return out


def score(q, page_bounds, q_lens, kv_lens, page, width):
    """Scores and the bounds of their errors. P and N are sums of G terms in fp32, their parts
    hold 24 bits, and the products are summed in fp32, by tensor cores that may cut off instead
    of rounding: (2 D + G + 8) roundings of twice EPS, relative to the sum of absolute values."""
    T, H, D = q.shape
    K = page_bounds[0].shape[1] if page_bounds else 1
    G = H // K
    out = torch.full((T, K, width), -math.inf, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for t, (r, pos) in enumerate(positions(q_lens, kv_lens)):
        n = 0 if pos < 0 else pos // page + 1
        if n == 0:
            continue
        b = torch.stack([page_bounds[r][c] for c in range(n)]).double()  # [n, K, 2, D]
        for h in range(K):
            x = q[t, h * G:(h + 1) * G].double()[:, None]
            best = torch.maximum(x * b[None, :, h, 0], x * b[None, :, h, 1])
            out[t, h, :n] = best.sum((0, 2))
            size = (x.clamp(min=0) * b[None, :, h, 1].abs() - x.clamp(max=0) * b[None, :, h, 0].abs())
            tol[t, h, :n] = (2 * D + G + 8) * 2 * EPS * size.sum((0, 2)) + 1e-37
    return out, tol


def select(scores, q_lens, kv_lens, page, count, first, recent):
    T, K, _ = scores.shape
    out = torch.full((T, K, count), -1, dtype=torch.int32)
    rows = scores.tolist()
    for t, (_, pos) in enumerate(positions(q_lens, kv_lens)):
        n = 0 if pos < 0 else pos // page + 1
        for h in range(K):
            always = [c for c in range(n) if c < first or c >= n - recent]
            if n <= count:
                always = list(range(n))
            free = [c for c in range(n) if c not in always]
            free.sort(key=lambda c: -(math.inf if math.isnan(rows[t][h][c]) else rows[t][h][c]))
            got = sorted(always + free[: max(0, count - len(always))])
            out[t, h, : len(got)] = torch.tensor(got, dtype=torch.int32)
    return out


def attend(q, ks, vs, q_lens, selected, page, scale=None):
    """Attention over the selected columns in 64 bits: out, lse and the bounds of their errors
    (see cache_ref.attend; the same operations in another order)."""
    T, H, D = q.shape
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    u = UNIT[q.dtype]
    out = torch.zeros((T, H, D), dtype=torch.float64)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    for t, (r, pos) in enumerate(positions(q_lens, [k.shape[0] for k in ks])):
        K = ks[r].shape[1]
        G = H // K
        for h in range(K):
            j = [c * page + x for c in selected[t, h].tolist() if c >= 0 for x in range(page)]
            j = torch.tensor([x for x in j if x <= pos], dtype=torch.long)
            if j.numel() == 0:
                continue
            k, v = ks[r][j, h].double(), vs[r][j, h].double()
            x = q[t, h * G:(h + 1) * G].double()
            s = x @ k.T * scale
            size = x.abs() @ k.abs().T * abs(scale)
            n = j.numel()
            p = torch.softmax(s, 1)
            at = slice(h * G, (h + 1) * G)
            out[t, at], lse[t, at] = p @ v, torch.logsumexp(s, 1)
            ds = (2 * D + 6) * EPS * size.amax(1) + 8 * EPS * s.abs().amax(1)
            w = 2 * ds + 2.0 ** -21 + 4 * n * EPS
            low = 2.0 ** -24 * n * p.amax(1, keepdim=True) * v.abs().amax(0)
            out_tol[t, at] = (2 * u + w[:, None]) * (p @ v.abs()) + low + 1e-30
            lse_tol[t, at] = ds + 2.0 ** -21 + 2 * n * EPS + 4 * EPS * lse[t, at].abs()
    return out, lse, out_tol, lse_tol


def weigh(q, ks, q_lens, lse, before, scale=None, decay=1.0):
    """Per request the weights [kv_heads, tokens] after the call, and the bounds of their errors.
    ``before`` likewise. A weight e^(s - lse) is off by a score's error (ds), the exponent's
    roundings (4 EPS of |s| + |lse|) and the exponential's (2^-21), a sum of n by n roundings."""
    D = q.shape[2]
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out, tol, t0 = [], [], 0
    for n, k, w in zip(q_lens, ks, before):
        L, K = k.shape[0], k.shape[1]
        G = q.shape[1] // K
        got, off = w.double().clone(), torch.zeros_like(w, dtype=torch.float64)
        for h in range(K if n else 0):
            kh = k[:, h].double()
            total, size = torch.zeros(L, dtype=torch.float64), torch.zeros(L, dtype=torch.float64)
            for g in range(h * G, (h + 1) * G):
                x, z = q[t0: t0 + n, g].double(), lse[t0: t0 + n, g].double()[:, None]
                s = x @ kh.T * scale
                seen = torch.arange(L) <= torch.arange(L - n, L)[:, None]
                seen = seen & (z > -math.inf)
                e = torch.where(seen, torch.exp(s - z), 0.0)
                ds = (2 * D + 6) * EPS * (x.abs() @ kh.abs().T) * abs(scale)
                ds = ds + 4 * EPS * (s.abs() + z.abs()) + 2.0 ** -21
                total += e.sum(0)
                size += torch.where(seen, e * ds, 0.0).sum(0)
            old = torch.arange(L) < L - n
            kept = torch.where(old, got[h] * decay, 0.0) if decay else torch.zeros(L).double()
            got[h] = kept + total
            off[h] = size + 2 * n * G * EPS * total + 4 * EPS * kept.abs() + n * G * 2.0 ** -126
        out.append(got)
        tol.append(off)
        t0 += n
    return out, tol


def evict(kp, vp, weights, table, lens, budget, free, count, first, recent):
    """The pools, the lengths and the stack after the call, or None where it refuses."""
    page, K = kp.shape[1], kp.shape[2]
    width = table.shape[1]
    if any(n < 0 or n > width * page for n in lens) or min(budget + [0]) < 0:
        return None
    kept = [min(n, max(b, first + recent)) for n, b in zip(lens, budget)]
    gone = sum(-(-n // page) - -(-m // page) for n, m in zip(lens, kept))
    if count < 0 or count + gone > len(free):
        return None
    out_k, out_v, out_w, free = kp.clone(), vp.clone(), weights.clone(), list(free)
    for r, (n, m) in enumerate(zip(lens, kept)):
        row = table[r].tolist()
        for c in range(-(-m // page), -(-n // page)):
            free[count] = row[c]
            count += 1
        if n == m:
            continue
        j = torch.arange(n)
        where, off = torch.tensor(row)[j // page].long(), j % page
        for h in range(K):
            w = weights[where, h, off].double()
            w = torch.where(w.isnan(), math.inf, w)
            always = (j < first) | (j >= n - recent)
            rest = torch.sort(w[first: n - recent], descending=True, stable=True).indices + first
            stay = torch.cat([j[always], rest[: m - int(always.sum())]]).sort().values
            out_k[where[:m], off[:m], h] = kp[where[stay], off[stay], h]
            out_v[where[:m], off[:m], h] = vp[where[stay], off[stay], h]
            out_w[where[:m], h, off[:m]] = weights[where[stay], h, off[stay]]
    return out_k, out_v, out_w, kept, free, count
