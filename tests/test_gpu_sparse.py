"""Sparse attention and eviction on the GPU against their plain forms in 64 bits."""
import math

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


def starts(lens, first=0):
    out = [first]
    for n in lens:
        out.append(out[-1] + n)
    return ints(out)


def status_word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def on_gpu(pool):
    """With the same order of its axes in memory."""
    order = sorted(range(pool.dim()), key=lambda i: -pool.stride(i))
    back = [order.index(i) for i in range(pool.dim())]
    return pool.permute(order).contiguous().to(DEV).permute(back)


def same(a, b):
    """Equal to the bit but for NaN's."""
    a, b = a.cpu(), b.cpu()
    return torch.equal(torch.nan_to_num(a.float(), nan=7777.0), torch.nan_to_num(b.float(), nan=7777.0))


# (new tokens of each request, their lengths, page, heads, kv heads, dim)
SHAPES = [
    ([1], [1], 16, 4, 1, 64),
    ([1], [700], 16, 32, 8, 128),
    ([3, 0, 1, 8, 2], [50, 33, 1, 200, 2], 16, 8, 2, 128),
    ([8, 1, 5], [9, 140, 77], 8, 7, 1, 96),
    ([2, 9, 1], [129, 64, 65], 32, 6, 2, 72),
    ([17, 40], [300, 40], 64, 3, 3, 80),
    ([1, 1, 1, 1], [15, 16, 17, 0], 16, 16, 1, 64),
    ([70], [333], 8, 40, 1, 8),
    ([4, 6], [2, 3], 8, 2, 1, 64),       # more new tokens than tokens: the first see nothing
]


def inputs(shape, dtype, layout, seed, rubbish=float("nan")):
    q_lens, kv_lens, page, heads, kv_heads, dim = shape
    g = torch.Generator().manual_seed(seed)
    kp, vp, table, ks, vs = cache_ref.cache(kv_lens, page, kv_heads, dim, dtype, g, layout=layout,
                                            rubbish=rubbish)
    q = (torch.randn((sum(q_lens), heads + 2, dim), generator=g) * 1.5).to(dtype)[:, 1:-1]
    return g, q, kp, vp, table, ks, vs


def kinds(f):
    f = pytest.mark.parametrize("dtype,layout", [(BF, "token"), (FP, "head")])(f)
    return pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"p{s[2]}h{s[3]}k{s[4]}d{s[5]}")(f)


# ---------------------------------------------------------------- bounds

@kinds
@pytest.mark.parametrize("fresh", [False, True])
def test_bounds(shape, dtype, layout, fresh):
    q_lens, kv_lens, page, _, kv_heads, dim = shape
    q_lens = [min(m, n) for m, n in zip(q_lens, kv_lens)]
    _, _, kp, _, table, ks, _ = inputs(shape, dtype, layout, 3)
    held = torch.full((kp.shape[0], kv_heads, 2, dim), 5.0, dtype=dtype)
    want = held.clone()
    for r, pages in enumerate(ref.bounds(ks, page)):
        for c, b in enumerate(pages):
            if not fresh or (q_lens[r] and c >= (kv_lens[r] - q_lens[r]) // page):
                want[table[r, c]] = b
    for max_q in (None, 1):
        got, status = held.to(DEV), status_word()
        sv.cache_bounds(on_gpu(kp), table.to(DEV), ints(kv_lens), got,
                        cu_q=starts(q_lens) if fresh else None, max_q=max_q, status=status)
        assert int(status) == 0
        assert torch.equal(got.cpu(), want)


def test_bounds_keep_nan_and_drop_what_a_step_dropped():
    _, _, kp, _, table, ks, _ = inputs(([1], [40], 16, 4, 2, 64), BF, "token", 4)
    kp[table[0, 1], 3, 1, 5] = math.nan
    got = torch.zeros((kp.shape[0], 2, 2, 64), dtype=BF, device=DEV)
    sv.cache_bounds(kp.to(DEV), table.to(DEV), ints([33]), got)
    x = got[table[0].tolist()[:3]].float().cpu()
    assert torch.isnan(x[1, 1, :, 5]).all()
    assert int(torch.isnan(x).sum()) == 2
    assert torch.equal(x[2, :, 0], ks[0][32].float()) and torch.equal(x[2, :, 1], x[2, :, 0])


# ---------------------------------------------------------------- scores

@kinds
def test_score(shape, dtype, layout):
    q_lens, kv_lens, page, heads, kv_heads, dim = shape
    g, q, kp, _, table, ks, _ = inputs(shape, dtype, layout, 5)
    pages = ref.bounds(ks, page)
    pool = torch.full((kp.shape[0], kv_heads, 2, dim), math.nan, dtype=dtype)
    for r, row in enumerate(pages):
        for c, b in enumerate(row):
            pool[table[r, c]] = b
    dense = [torch.stack(row) if row else torch.zeros((0, kv_heads, 2, dim)) for row in pages]
    want, tol = ref.score(q, dense, q_lens, kv_lens, page, table.shape[1])
    pad = 3
    q = torch.cat([q, q[:1].expand(pad, -1, -1)]).to(DEV)
    for max_q in (None, max(q_lens), 1):
        status = status_word()
        got = sv.cache_score(q, pool.to(DEV), table.to(DEV), ints(kv_lens), starts(q_lens),
                             page_size=page, max_q=max_q, status=status).double().cpu()
        assert int(status) == 0
        assert (got[-pad:] == -math.inf).all()
        got = got[:-pad]
        none = torch.isinf(want)
        assert torch.equal(none, torch.isinf(got)) and (got[none] < 0).all()
        off = ((got - want).abs() - tol)[~none]
        assert off.numel() == 0 or off.max() <= 0, float(off.max())


@pytest.mark.parametrize("dtype,size", [(BF, 1e30), (BF, 1e-30), (FP, 6e4), (FP, 1e-6)])
def test_score_of_large_and_small_queries(dtype, size):
    g = torch.Generator().manual_seed(2)
    q = (torch.randn((2, 8, 64), generator=g).clamp(-1, 1) * size).to(dtype)
    b = torch.randn((3, 2, 2, 64), generator=g).sort(2).values.to(dtype)
    want, tol = ref.score(q, [b], [2], [40], 16, 3)
    got = sv.cache_score(q.to(DEV), b.to(DEV), ints([[0, 1, 2]]), ints([40]), ints([0, 2]),
                         page_size=16)
    none = torch.isinf(want)
    assert not torch.isnan(got).any()
    assert ((got.double().cpu() - want).abs() <= tol)[~none].all()


def test_score_into_a_strided_output():
    _, q, kp, _, table, ks, _ = inputs(SHAPES[2], BF, "token", 6)
    pool = torch.zeros((kp.shape[0], 2, 2, 128), dtype=BF)
    q, pool, table = q.to(DEV), pool.to(DEV), table.to(DEV)
    lens, cu = ints(SHAPES[2][1]), starts(SHAPES[2][0])
    sv.cache_bounds(kp.to(DEV), table, lens, pool)
    want = sv.cache_score(q, pool, table, lens, cu, page_size=16)
    room = torch.full((q.shape[0], 3, table.shape[1] + 5), 9.0, device=DEV)
    out = room[:, 1:, 2:-3]
    assert sv.cache_score(q, pool, table, lens, cu, page_size=16, out=out) is out
    assert torch.equal(out, want)
    assert (room[:, 0] == 9).all() and (room[:, :, :2] == 9).all() and (room[:, :, -3:] == 9).all()


# ---------------------------------------------------------------- selection

@pytest.mark.parametrize("q_lens,kv_lens,page,kv_heads,count,first,recent", [
    ([1], [1], 16, 1, 1, 0, 0), ([3, 0, 1, 8], [50, 33, 1, 200], 8, 2, 5, 1, 2),
    ([2, 5], [3000, 800], 8, 3, 64, 0, 1), ([1], [20000], 8, 1, 300, 2, 3),
    ([1], [200000], 16, 2, 250, 0, 0), ([2], [100000], 8, 1, 12499, 0, 0),
    ([4], [640], 8, 2, 7, 3, 4), ([6], [3], 8, 1, 2, 0, 1), ([1, 1], [16, 17], 16, 1, 1, 1, 0)])
@pytest.mark.parametrize("values", ["random", "few", "special"])
def test_select(q_lens, kv_lens, page, kv_heads, count, first, recent, values):
    g = torch.Generator().manual_seed(7)
    width = max(-(-n // page) for n in kv_lens) + 3
    x = torch.randn((sum(q_lens), kv_heads, width), generator=g)
    if values == "few":  # many equal ones
        x = (x * 2).round()
    if values == "special":
        odd = torch.tensor([math.inf, -math.inf, math.nan, 0.0, -0.0, 1e-40, -1e-40, 3e38])
        x = odd[torch.randint(0, 8, x.shape, generator=g)]
    want = ref.select(x, q_lens, kv_lens, page, count, first, recent)
    x = torch.cat([x, x[:1]]).to(DEV)  # and a row of no request
    status = status_word()
    got = sv.cache_select(x, ints(kv_lens), starts(q_lens), page_size=page, count=count,
                          first=first, recent=recent, status=status)
    assert int(status) == 0
    assert (got[-1] == -1).all()
    assert torch.equal(got[:-1].cpu(), want)


# ---------------------------------------------------------------- attention

def lists(g, q_lens, kv_lens, page, kv_heads, count):
    """Ascending lists of any visible columns, some empty, some longer than what is seen."""
    out = torch.full((sum(q_lens), kv_heads, count), -1, dtype=torch.int32)
    for t, (r, pos) in enumerate(ref.positions(q_lens, kv_lens)):
        held = -(-kv_lens[r] // page)
        for h in range(kv_heads):
            n = int(torch.randint(0, min(count, held) + 1, (1,), generator=g))
            cols = torch.randperm(held, generator=g)[:n].sort().values
            out[t, h, :n] = cols.to(torch.int32)
    return out


@kinds
@pytest.mark.parametrize("count", [1, 9, 800])
def test_attend_selected(shape, dtype, layout, count):
    q_lens, kv_lens, page, heads, kv_heads, dim = shape
    g, q, kp, vp, table, ks, vs = inputs(shape, dtype, layout, 8)
    sel = lists(g, q_lens, kv_lens, page, kv_heads, count)
    want = ref.attend(q, ks, vs, q_lens, sel, page)
    pad = 2
    q = torch.cat([q, q[:1].expand(pad, -1, -1)]).to(DEV)
    sel = torch.cat([sel, sel[:1].expand(pad, -1, -1)]).to(DEV)
    status = status_word()
    out, lse = sv.cache_attend_selected(q, on_gpu(kp), on_gpu(vp), table.to(DEV), ints(kv_lens),
                                        starts(q_lens), sel, return_lse=True, status=status)
    assert int(status) == 0
    assert (out[-pad:] == 0).all() and (lse[-pad:] == -math.inf).all()
    cache_ref.assert_attend(out[:-pad], lse[:-pad], want)


@pytest.mark.parametrize("heads,kv_heads", [(4, 1), (8, 1), (12, 1), (20, 1), (33, 1), (128, 1), (8, 8)])
@pytest.mark.parametrize("dim", [64, 128])
def test_attend_selected_heads(heads, kv_heads, dim):
    shape = ([7, 1, 12], [400, 90, 700], 16, heads, kv_heads, dim)
    g, q, kp, vp, table, ks, vs = inputs(shape, BF, "token", 9)
    sel = lists(g, shape[0], shape[1], 16, kv_heads, 20)
    want = ref.attend(q, ks, vs, shape[0], sel, 16, scale=0.2)
    out, lse = sv.cache_attend_selected(q.to(DEV), kp.to(DEV), vp.to(DEV), table.to(DEV),
                                        ints(shape[1]), starts(shape[0]), sel.to(DEV), scale=0.2,
                                        return_lse=True)
    cache_ref.assert_attend(out, lse, want)


def test_attend_selected_one_token_over_more_pages_than_a_list():
    """Parts of the list, clusters of blocks, a negative and a zero scale."""
    shape = ([1], [20000], 8, 8, 2, 64)
    g, q, kp, vp, table, ks, vs = inputs(shape, FP, "token", 10)
    sel = torch.arange(2500, dtype=torch.int32).expand(1, 2, 2500).contiguous()
    for scale in (0.125, -0.125, 0.0):
        want = ref.attend(q, ks, vs, [1], sel, 8, scale=scale)
        out, lse = sv.cache_attend_selected(q.to(DEV), kp.to(DEV), vp.to(DEV), table.to(DEV),
                                            ints([20000]), ints([0, 1]), sel.to(DEV), scale=scale,
                                            return_lse=True)
        cache_ref.assert_attend(out, lse, want)


def test_attend_selected_is_attend_where_all_is_selected():
    shape = ([5, 1, 3], [500, 77, 3], 16, 8, 2, 128)
    g, q, kp, vp, table, ks, vs = inputs(shape, BF, "token", 11)
    sel = torch.full((9, 2, 32), -1, dtype=torch.int32)
    for t, (r, pos) in enumerate(ref.positions(shape[0], shape[1])):
        sel[t, :, : pos // 16 + 1] = torch.arange(pos // 16 + 1, dtype=torch.int32)
    args = (q.to(DEV), kp.to(DEV), vp.to(DEV), table.to(DEV), ints(shape[1]), starts(shape[0]))
    want = ref.attend(q, ks, vs, shape[0], sel, 16)
    for out, lse in (sv.cache_attend(*args, return_lse=True),
                     sv.cache_attend_selected(*args, sel.to(DEV), return_lse=True)):
        cache_ref.assert_attend(out, lse, want)


# ---------------------------------------------------------------- weights

def spread_weights(weights, per_request, table, page):
    """[kv_heads, tokens] of each request into the pool's slots."""
    for r, w in enumerate(per_request):
        for c in range(-(-w.shape[1] // page)):
            part = w[:, c * page: (c + 1) * page]
            weights[table[r, c], :, : part.shape[1]] = part.to(weights.dtype)


@kinds
@pytest.mark.parametrize("decay", [1.0, 0.5, 0.0])
def test_weigh(shape, dtype, layout, decay):
    q_lens, kv_lens, page, heads, kv_heads, dim = shape
    g, q, kp, vp, table, ks, vs = inputs(shape, dtype, layout, 12)
    _, lse, _, _ = cache_ref.attend(q, ks, vs, q_lens)
    lse = lse.float()
    before = [torch.rand((kv_heads, n), generator=g) for n in kv_lens]
    for w, m, n in zip(before, q_lens, kv_lens):
        w[:, max(n - m, 0):] = math.nan if m else 0.25
        if decay == 0 and m:
            w[:] = math.nan
    weights = torch.full((kp.shape[0], kv_heads, page), -3.0)
    spread_weights(weights, before, table, page)
    want, tol = ref.weigh(q, ks, q_lens, lse, before, decay=decay)
    q = torch.cat([q, q[:1]]).to(DEV)
    lse = torch.cat([lse, lse[:1]]).to(DEV)
    for max_q in (None, max(q_lens), 1):
        got, status = weights.to(DEV), status_word()
        sv.cache_weigh(q, on_gpu(kp), table.to(DEV), ints(kv_lens), starts(q_lens), lse, got,
                       max_q=max_q, decay=decay, status=status)
        assert int(status) == 0
        got = got.double().cpu()
        for r, (w, off) in enumerate(zip(want, tol)):
            n = w.shape[1]
            rows = [got[table[r, c]] for c in range(-(-n // page))]
            mine = torch.cat(rows, 1)[:, :n] if rows else w
            assert not torch.isnan(mine).any()
            over = (mine - w).abs() - off
            assert over.numel() == 0 or over.max() <= 0, float(over.max())
        # slots of no token stay as they are
        used = torch.zeros(weights.shape, dtype=torch.bool)
        spread_weights(used, [torch.ones((kv_heads, n)) for n in kv_lens], table, page)
        assert (got[~used] == -3.0).all()


# ---------------------------------------------------------------- eviction

@pytest.mark.parametrize("dtype,layout", [(BF, "token"), (FP, "head")])
@pytest.mark.parametrize("lens,budget,first,recent,page,kv_heads,dim", [
    ([40], [20], 0, 0, 16, 1, 64), ([40], [20], 3, 5, 16, 2, 128),
    ([100, 3, 0, 64, 65], [50, 50, 0, 64, 64], 2, 4, 16, 2, 64),
    ([333, 200], [1, 0], 4, 7, 8, 3, 80), ([70, 70], [0, 69], 0, 0, 8, 1, 72),
    ([900, 1200], [300, 1100], 10, 40, 32, 2, 96), ([65], [0], 40, 40, 64, 2, 8)])
@pytest.mark.parametrize("values", ["random", "few"])
def test_evict(dtype, layout, lens, budget, first, recent, page, kv_heads, dim, values):
    g = torch.Generator().manual_seed(13)
    kp, vp, table, _, _ = cache_ref.cache(lens, page, kv_heads, dim, dtype, g, layout=layout)
    weights = torch.rand((kp.shape[0], kv_heads, page), generator=g)
    if values == "few":
        odd = torch.tensor([0.0, -0.0, 1.0, math.inf, math.nan, 1e-41, -1.0, 2.0])
        weights = odd[torch.randint(0, 8, weights.shape, generator=g)]
    held = {x for r, n in enumerate(lens) for x in table[r, : -(-n // page)].tolist()}
    spare = [x for x in range(kp.shape[0]) if x not in held]
    free = spare + [-9] * len(held)
    want = ref.evict(kp, vp, weights, table, lens, budget, free, len(spare), first, recent)
    k, v, w, f = on_gpu(kp), on_gpu(vp), weights.to(DEV), ints(free)
    t, status = table.to(DEV), status_word()
    r = sv.cache_evict(k, v, w, t, ints(lens), ints(budget), f, ints([len(spare)]), first=first,
                       recent=recent, status=status)
    assert int(status) == 0
    assert r.lens.tolist() == want[3]
    assert f.tolist() == want[4] and int(r.free_count) == want[5]
    assert torch.equal(t.cpu(), table)
    assert same(w, want[2]) and same(k, want[0]) and same(v, want[1])


@pytest.mark.parametrize("lens,budget,first,recent,page,kv_heads", [
    ([20000, 9000], [3000, 8999], 5, 100, 16, 2),      # clusters of blocks
    ([70000], [100], 0, 0, 64, 1), ([140000], [139000], 3, 9, 32, 1),  # longer than registers
    ([5000] * 20, [4097] * 20, 0, 1, 16, 8)])           # a block for each of many
@pytest.mark.parametrize("values", ["random", "few"])
def test_evict_long(lens, budget, first, recent, page, kv_heads, values):
    g = torch.Generator().manual_seed(14)
    kp, vp, table, _, _ = cache_ref.cache(lens, page, kv_heads, 8, BF, g)
    weights = torch.rand((kp.shape[0], kv_heads, page), generator=g)
    if values == "few":
        weights = (weights * 5).floor()
    free = [-9] * kp.shape[0]
    want = ref.evict(kp, vp, weights, table, lens, budget, free, 0, first, recent)
    k, v, w, f = kp.to(DEV), vp.to(DEV), weights.to(DEV), ints(free)
    status = status_word()
    r = sv.cache_evict(k, v, w, table.to(DEV), ints(lens), ints(budget), f, ints([0]), first=first,
                       recent=recent, status=status)
    assert int(status) == 0
    assert r.lens.tolist() == want[3] and f.tolist() == want[4]
    assert same(w, want[2]) and same(k, want[0]) and same(v, want[1])


@pytest.mark.parametrize("rows,columns,count", [
    (1, 5000, 77), (30, 9000, 500), (200, 3000, 64), (200, 6000, 5999), (160, 12000, 250),
    (3, 60000, 1000), (100, 20000, 19000), (1, 140000, 3)])
@pytest.mark.parametrize("values", ["random", "few", "spikes"])
def test_select_long(rows, columns, count, values):
    g = torch.Generator().manual_seed(15)
    x = torch.randn((rows, 1, columns), generator=g)
    if values == "few":
        x = (x * 2).round()
    if values == "spikes":  # nearly all in one place, a few orders of magnitude away
        x = torch.where(torch.rand(x.shape, generator=g) < 0.01, x * 1e30, x * 1e-30)
    lens = [columns * 8 - 8 * (r % 7) for r in range(rows)]
    got = sv.cache_select(x.to(DEV), ints(lens), starts([1] * rows), page_size=8, count=count,
                          first=2, recent=1)
    for r in range(rows):
        n = lens[r] // 8
        score = x[r, 0, 2:n - 1].double()
        best = torch.sort(score, descending=True, stable=True).indices[: count - 3] + 2
        want = torch.full((count,), -1)  # past the last where fewer are visible
        chosen = torch.cat([torch.tensor([0, 1, n - 1]), best]).sort().values
        want[: len(chosen)] = chosen
        assert torch.equal(got[r, 0].cpu().long(), want), r
