"""Sparse-attention and eviction calls where one form of a kernel ends and the next begins, and
where the work of cache_weigh is cut between blocks."""
import pytest
import torch

import cache_ref
import sparse_ref as ref
import speculative_decoding_rejection_02_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float16


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return ints(out)


def same(a, b):
    return torch.equal(torch.nan_to_num(a.float().cpu(), nan=7777.0),
                       torch.nan_to_num(b.float().cpu(), nan=7777.0))


@pytest.mark.parametrize("columns", [511, 512, 513, 1024, 1025, 2048, 2049, 4096, 4097, 8193,
                                     16384, 16385])
@pytest.mark.parametrize("values", ["random", "few", "equal"])
def test_select_at_the_limits_of_its_forms(columns, values):
    g = torch.Generator().manual_seed(21)
    x = torch.randn((9, 1, columns), generator=g)
    if values == "few":
        x = (x * 2).round()
    if values == "equal":
        x[:] = -0.5
    count, first, recent = 41, 3, 2
    lens = [8 * (columns - 7 * r) for r in range(9)]
    got = sv.cache_select(x.to(DEV), ints(lens), starts([1] * 9), page_size=8, count=count,
                          first=first, recent=recent).cpu().long()
    for r, n in enumerate(lens):
        n //= 8
        best = torch.sort(x[r, 0, first:n - recent], descending=True, stable=True).indices
        best = best[: count - first - recent] + first
        want = torch.cat([torch.arange(first), best, torch.arange(n - recent, n)]).sort().values
        assert torch.equal(got[r, 0], want), r


@pytest.mark.parametrize("most", [8, 120, 2040, 2048, 2056, 4096, 4104, 16384, 16392])
@pytest.mark.parametrize("values", ["random", "few", "equal"])
@pytest.mark.parametrize("always", [(0, 0), (3, 60)])
def test_evict_at_the_limits_of_its_forms(most, values, always):
    g = torch.Generator().manual_seed(22)
    first, recent = always
    lens = [most, max(most - 5, 1), most // 2, 1, most]
    budget = [most // 3, most - 6 if most > 8 else 1, 0, 0, most - 1]
    kp, vp, table, _, _ = cache_ref.cache(lens, 8, 2, 8, BF, g)
    weights = torch.randn((kp.shape[0], 2, 8), generator=g)
    if values == "few":
        weights = (weights * 2).round()
    if values == "equal":
        weights[:] = 0.25
    free = [-9] * kp.shape[0]
    want = ref.evict(kp, vp, weights, table, lens, budget, free, 0, first, recent)
    k, v, w, f = kp.to(DEV), vp.to(DEV), weights.to(DEV), ints(free)
    status = ints([0])
    r = sv.cache_evict(k, v, w, table.to(DEV), ints(lens), ints(budget), f, ints([0]), first=first,
                       recent=recent, status=status)
    assert int(status) == 0
    assert r.lens.tolist() == want[3] and f.tolist() == want[4]
    assert same(w, want[2]) and same(k, want[0]) and same(v, want[1])


@pytest.mark.parametrize("q_lens,kv_lens,page,heads,kv_heads,dim,dtype", [
    ([1200, 0, 3, 700], [1200, 40, 3, 1900], 16, 8, 2, 64, BF),   # prompts, columns in tiles of 32
    ([900, 1], [2500, 2500], 128, 7, 1, 128, FP),                 # tiles of 18 tokens, ragged
    ([300, 299], [301, 2000], 8, 33, 1, 80, BF),                  # three tokens a tile
    ([700, 40], [690, 30], 32, 4, 4, 64, BF)])                    # more tokens than are held
def test_weigh_of_prompts_and_chunks(q_lens, kv_lens, page, heads, kv_heads, dim, dtype):
    g = torch.Generator().manual_seed(23)
    kp, vp, table, ks, vs = cache_ref.cache(kv_lens, page, kv_heads, dim, dtype, g)
    q = torch.randn((sum(q_lens), heads, dim), generator=g).to(dtype)
    _, lse, _, _ = cache_ref.attend(q, ks, vs, q_lens)
    lse = lse.float()
    before = [torch.rand((kv_heads, n), generator=g) for n in kv_lens]
    weights = torch.full((kp.shape[0], kv_heads, page), -3.0)
    for w, t in zip(before, table):
        for c in range(-(-w.shape[1] // page)):
            part = w[:, c * page:(c + 1) * page]
            weights[t[c], :, : part.shape[1]] = part
    want, tol = ref.weigh(q, ks, q_lens, lse, before, decay=0.5)
    got, status = weights.to(DEV), ints([0])
    sv.cache_weigh(q.to(DEV), kp.to(DEV), table.to(DEV), ints(kv_lens), starts(q_lens),
                   lse.to(DEV), got, decay=0.5, status=status)
    assert int(status) == 0
    for r, (w, off) in enumerate(zip(want, tol)):
        n = w.shape[1]
        rows = [got[table[r, c]] for c in range(-(-n // page))]
        mine = torch.cat(rows, 1)[:, :n].double().cpu()
        over = (mine - w).abs() - off
        assert over.max() <= 0, float(over.max())
