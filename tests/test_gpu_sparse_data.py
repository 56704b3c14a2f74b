"""Sparse attention and eviction: errors in device data, odd layouts, large addresses, ragged
batches over many blocks."""
import math

import pytest
import torch

import cache_ref
import sparse_ref as ref
import speculative_decoding_rejection_02_gb300 as sv
from test_gpu_sparse import BF, DEV, FP, inputs, ints, lists, on_gpu, same, starts, status_word

pytestmark = pytest.mark.gpu

SHAPE = ([3, 1, 6], [70, 33, 200], 16, 8, 2, 64)


def everything(shape=SHAPE, dtype=BF, seed=20):
    """Arguments of all calls, as a dict of tensors on the GPU."""
    g, q, kp, vp, table, ks, vs = inputs(shape, dtype, "token", seed, rubbish=0.0)
    q_lens, lens, page, heads, kv_heads, dim = shape
    x = dict(q=q, k=kp, v=vp, table=table, lens=torch.tensor(lens, dtype=torch.int32),
             cu=starts(q_lens).cpu(), bounds=torch.zeros((kp.shape[0], kv_heads, 2, dim), dtype=dtype),
             sel=lists(g, q_lens, lens, page, kv_heads, 5), lse=torch.zeros(q.shape[:2]),
             weights=torch.rand((kp.shape[0], kv_heads, page), generator=g),
             budget=torch.full((len(lens),), 40, dtype=torch.int32),
             free=torch.full((kp.shape[0],), -1, dtype=torch.int32),
             count=torch.zeros(1, dtype=torch.int32))
    return {k: v.to(DEV) for k, v in x.items()}


def run_all(x, status):
    """All calls on the same state; their outputs."""
    out = {}
    page = x["k"].shape[1]
    sv.cache_bounds(x["k"], x["table"], x["lens"], x["bounds"], cu_q=x["cu"], status=status)
    out["score"] = sv.cache_score(x["q"], x["bounds"], x["table"], x["lens"], x["cu"],
                                  page_size=page, status=status)
    out["select"] = sv.cache_select(out["score"], x["lens"], x["cu"], page_size=page, count=3,
                                    status=status)
    out["out"], out["lse"] = sv.cache_attend_selected(
        x["q"], x["k"], x["v"], x["table"], x["lens"], x["cu"], x["sel"], return_lse=True,
        status=status)
    sv.cache_weigh(x["q"], x["k"], x["table"], x["lens"], x["cu"], x["lse"], x["weights"],
                   status=status)
    r = sv.cache_evict(x["k"], x["v"], x["weights"], x["table"], x["lens"], x["budget"], x["free"],
                       x["count"], first=2, recent=3, status=status)
    out.update(lens=r.lens, count=r.free_count)
    torch.cuda.synchronize()
    return out


CALLS = ["bounds", "score", "select", "attend_selected", "weigh", "evict"]


def run_one(name, x, status):
    page = x["k"].shape[1]
    if name == "bounds":
        sv.cache_bounds(x["k"], x["table"], x["lens"], x["bounds"], status=status)
    if name == "score":
        return sv.cache_score(x["q"], x["bounds"], x["table"], x["lens"], x["cu"], page_size=page,
                              status=status)
    if name == "select":
        scores = torch.rand((x["q"].shape[0], x["k"].shape[2], x["table"].shape[1]), device=DEV)
        return sv.cache_select(scores, x["lens"], x["cu"], page_size=page, count=3, status=status)
    if name == "attend_selected":
        return sv.cache_attend_selected(x["q"], x["k"], x["v"], x["table"], x["lens"], x["cu"],
                                        x["sel"], return_lse=True, status=status)
    if name == "weigh":
        sv.cache_weigh(x["q"], x["k"], x["table"], x["lens"], x["cu"], x["lse"], x["weights"],
                       status=status)
    if name == "evict":
        return sv.cache_evict(x["k"], x["v"], x["weights"], x["table"], x["lens"], x["budget"],
                              x["free"], x["count"], status=status)


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("length", [-1, 10 ** 6, 2 ** 31 - 1])
def test_lengths_that_cannot_be(name, length):
    x, good = everything(), everything()
    x["lens"][1] = length
    status = status_word()
    got, want = run_one(name, x, status), run_one(name, good, status_word())
    assert int(status) == sv.CACHE_BAD_LENGTHS
    if name == "score":
        assert (got[3] == -math.inf).all()
        assert torch.equal(got[:3], want[:3]) and torch.equal(got[4:], want[4:])
    if name == "select":
        assert (got[3] == -1).all()
    if name == "attend_selected":
        assert (got[0][3] == 0).all() and (got[1][3] == -math.inf).all()
        assert torch.equal(got[0][4:], want[0][4:]) and torch.equal(got[1][:3], want[1][:3])
    if name == "weigh":
        other = [0, 2]
        for r in other:
            pages = x["table"][r, : -(-SHAPE[1][r] // 16)].long()
            assert torch.equal(x["weights"][pages], good["weights"][pages])
        assert torch.equal(x["weights"][x["table"][1, :3].long()],
                           everything()["weights"][x["table"][1, :3].long()])
    if name == "evict":  # nothing at all
        for k in ("k", "v", "weights", "free"):
            assert torch.equal(x[k], everything()[k]), k
        assert torch.equal(got.lens, x["lens"]) and int(got.free_count) == 0


@pytest.mark.parametrize("change", [dict(budget=-1), dict(count=-1), dict(count=10 ** 6),
                                    dict(count="full")])
def test_evict_refuses_as_a_whole(change):
    x = everything()
    before = {k: v.clone() for k, v in x.items()}
    if "budget" in change:
        x["budget"][2] = -1
    elif change["count"] == "full":
        x["count"][0] = x["free"].numel() - 3
    else:
        x["count"][0] = change["count"]
    status = status_word()
    r = run_one("evict", x, status)
    assert int(status) == sv.CACHE_BAD_LENGTHS
    for k in ("k", "v", "weights", "free", "table"):
        assert torch.equal(x[k], before[k]), k
    assert torch.equal(r.lens, x["lens"]) and torch.equal(r.free_count, x["count"])


@pytest.mark.parametrize("name", ["bounds", "score", "attend_selected", "weigh", "evict"])
@pytest.mark.parametrize("page", [-1, 10 ** 9, 2 ** 31 - 1])
def test_page_numbers_outside_the_pool(name, page):
    x, good = everything(), everything()
    for y in (x, good):
        y["sel"][0, :, 0] = 1
        y["sel"][0, :, 1:] = -1
    x["table"][0, 1] = page
    status = status_word()
    got, want = run_one(name, x, status), run_one(name, good, status_word())
    assert int(status) == sv.CACHE_BAD_PAGE
    if name == "score":
        assert (got[:3, :, 1] == -math.inf).all() and torch.equal(got[3:], want[3:])
    if name == "attend_selected":
        assert torch.equal(got[0][3:], want[0][3:])
    if name in ("weigh", "evict"):
        for r in (1, 2):
            pages = x["table"][r, : -(-SHAPE[1][r] // 16)].long()
            assert torch.equal(x["weights"][pages], good["weights"][pages])


@pytest.mark.parametrize("offsets", [[0, 3, 2, 10], [-1, 3, 4, 10], [0, 3, 4, 11], [5, 0, 0, 10]])
@pytest.mark.parametrize("name", ["bounds", "score", "select", "attend_selected", "weigh"])
def test_offsets_that_cannot_be(name, offsets):
    x = everything()
    x["cu"].copy_(torch.tensor(offsets))
    if name == "bounds":  # which has no rows to count
        if offsets[-1] == 11:
            return
    status = status_word()
    if name == "bounds":
        sv.cache_bounds(x["k"], x["table"], x["lens"], x["bounds"], cu_q=x["cu"], status=status)
    else:
        run_one(name, x, status)
    assert int(status) == sv.CACHE_BAD_LENGTHS


@pytest.mark.parametrize("entries", [[2, 1], [1, 1], [-1, 1], [0, 5], [4, 10 ** 9]])
@pytest.mark.parametrize("tokens", [1, 5])
def test_selections_that_cannot_be(entries, tokens):
    shape = ([tokens], [75], 16, 4, 1, 64)  # five columns
    x = everything(shape)
    x["sel"] = torch.full((tokens, 1, 4), -1, dtype=torch.int32, device=DEV)
    x["sel"][tokens // 2, 0, :2] = ints(entries)
    status = status_word()
    run_one("attend_selected", x, status)
    assert int(status) == sv.CACHE_BAD_SELECTION


def test_status_bits_without_a_word():
    sv.cache_status(DEV)
    x = everything()
    x["lens"][0] = -4
    run_one("score", x, None)
    assert sv.cache_status(DEV) == sv.CACHE_BAD_LENGTHS
    assert sv.cache_status(DEV) == 0


# ---------------------------------------------------------------- layouts

def test_offsets_that_do_not_start_at_zero():
    """Rows before the first request's belong to none."""
    x, y = everything(), everything()
    x["cu"] += 2
    x["q"] = torch.cat([x["q"][:2], x["q"], x["q"][:3]])
    for k in ("sel", "lse"):
        x[k] = torch.cat([x[k][:2], x[k], x[k][:3]])
    status = status_word()
    got, want = run_all(x, status), run_all(y, status)
    assert int(status) == 0
    T = y["q"].shape[0]
    for k, fill in (("score", -math.inf), ("select", -1), ("out", 0), ("lse", -math.inf)):
        assert torch.equal(got[k][2:2 + T], want[k]), k
        assert (got[k][:2] == fill).all() and (got[k][2 + T:] == fill).all(), k
    assert torch.equal(x["weights"], y["weights"]) and torch.equal(x["bounds"], y["bounds"])


def test_nothing():
    """No requests, and requests without tokens."""
    x = everything()
    none = dict(x, table=x["table"][:0], lens=x["lens"][:0], cu=x["cu"][:1].clone(),
                budget=x["budget"][:0])
    status = status_word()
    got = run_all(none, status)
    assert int(status) == 0
    assert (got["score"] == -math.inf).all() and (got["select"] == -1).all()
    assert (got["out"] == 0).all() and (got["lse"] == -math.inf).all()
    assert got["lens"].numel() == 0 and int(got["count"]) == 0
    for k in ("weights", "bounds", "k", "free"):
        assert torch.equal(none[k], everything()[k]), k
    empty = everything(([0, 0], [0, 20], 16, 8, 2, 64))
    empty["sel"] = empty["sel"][:0]
    got = run_all(empty, status)
    assert int(status) == 0 and got["lens"].tolist() == [0, 20]
    assert got["score"].shape[0] == 0


def interleaved(x):
    """Keys and values as views of one pool, weights and bounds as slices of wider ones."""
    pool = torch.stack([x["k"], x["v"]], 1)
    wide = torch.zeros((*x["weights"].shape[:2], x["weights"].shape[2] + 3), device=DEV)
    wide[:, :, :-3] = x["weights"]
    side = torch.zeros((x["bounds"].shape[0], x["bounds"].shape[1] + 1, 2, x["bounds"].shape[3] + 8),
                       dtype=x["bounds"].dtype, device=DEV)
    return dict(x, k=pool[:, 0], v=pool[:, 1], weights=wide[:, :, :-3], bounds=side[:, 1:, :, :-8],
                table=torch.cat([x["table"], x["table"]], 1)[:, : x["table"].shape[1]])


@pytest.mark.parametrize("dtype", [BF, FP])
def test_other_strides(dtype):
    x, y = everything(dtype=dtype), interleaved(everything(dtype=dtype))
    status = status_word()
    got, want = run_all(y, status), run_all(x, status)
    assert int(status) == 0
    for k in want:
        assert torch.equal(got[k], want[k]), k
    for k in ("k", "v", "weights", "bounds", "free"):
        assert same(y[k], x[k]), k


def test_pages_beyond_32_bits():
    """Pages 2^31 elements apart."""
    small = everything(([2, 1], [30, 20], 16, 4, 1, 64))
    n = small["k"].shape[0]
    far = dict(small)
    for k in ("k", "v", "bounds", "weights"):
        t = small[k]
        pool = torch.empty(2 ** 31 * (n - 1) + t[0].numel(), dtype=t.dtype, device=DEV)
        far[k] = pool.as_strided(t.shape, (2 ** 31, *t.stride()[1:]))
        far[k].copy_(t)
    status = status_word()
    got, want = run_all(far, status), run_all(small, status)
    assert int(status) == 0
    for k in want:
        assert torch.equal(got[k], want[k]), k
    for k in ("k", "v", "weights", "bounds"):
        assert same(far[k], small[k]), k


def test_the_same_to_the_bit():
    shape = ([40, 1, 7, 1], [3000, 5000, 900, 1], 16, 8, 2, 128)
    first = None
    for _ in range(5):
        x = everything(shape, seed=21)
        got = run_all(x, status_word())
        got.update({k: x[k] for k in ("k", "v", "weights", "bounds", "free")})
        first = first or got
        for k in got:
            assert torch.equal(got[k], first[k]), k


# ---------------------------------------------------------------- many blocks

@pytest.mark.parametrize("dtype,heads,kv_heads,dim", [(BF, 8, 2, 128), (FP, 14, 2, 96), (BF, 4, 4, 64)])
def test_weigh_chunks_beside_single_tokens(dtype, heads, kv_heads, dim):
    """Several column tiles in some requests and one in others, parts of the list that begin and
    end within requests."""
    q_lens = [300, 1, 5, 0, 77, 1, 130, 2, 1, 64] * 3
    g = torch.Generator().manual_seed(22)
    lens = [n + int(c) for n, c in zip(q_lens, torch.randint(0, 2000, (30,), generator=g))]
    shape = (q_lens, lens, 16, heads, kv_heads, dim)
    _, q, kp, _, table, ks, vs = inputs(shape, dtype, "token", 23)
    _, lse, _, _ = cache_ref.attend(q, ks, vs, q_lens)
    lse = lse.float()
    before = [torch.rand((kv_heads, n), generator=g) for n in lens]
    weights = torch.zeros((kp.shape[0], kv_heads, 16))
    for r, w in enumerate(before):
        for c in range(-(-lens[r] // 16)):
            part = w[:, 16 * c: 16 * c + 16]
            weights[table[r, c], :, : part.shape[1]] = part
    want, tol = ref.weigh(q, ks, q_lens, lse, before)
    for max_q in (300, 1):
        got, status = weights.to(DEV), status_word()
        sv.cache_weigh(q.to(DEV), kp.to(DEV), table.to(DEV), ints(lens), starts(q_lens),
                       lse.to(DEV), got, max_q=max_q, status=status)
        assert int(status) == 0
        got = got.double().cpu()
        for r, (w, off) in enumerate(zip(want, tol)):
            rows = [got[table[r, c]] for c in range(-(-lens[r] // 16))]
            mine = torch.cat(rows, 1)[:, : lens[r]]
            assert ((mine - w).abs() <= off).all(), r


@pytest.mark.parametrize("dtype,heads,kv_heads,dim", [(BF, 8, 2, 128), (FP, 6, 3, 72)])
def test_score_of_chunks_beside_single_tokens(dtype, heads, kv_heads, dim):
    q_lens = [90, 1, 5, 0, 33, 1, 64, 2] * 2
    g = torch.Generator().manual_seed(24)
    lens = [n + int(c) for n, c in zip(q_lens, torch.randint(0, 1500, (16,), generator=g))]
    shape = (q_lens, lens, 8, heads, kv_heads, dim)
    _, q, kp, _, table, ks, _ = inputs(shape, dtype, "token", 25)
    pages = [torch.stack(r) if r else torch.zeros((0, kv_heads, 2, dim)) for r in ref.bounds(ks, 8)]
    want, tol = ref.score(q, pages, q_lens, lens, 8, table.shape[1])
    bounds = torch.full((kp.shape[0], kv_heads, 2, dim), math.nan, dtype=dtype, device=DEV)
    sv.cache_bounds(on_gpu(kp), table.to(DEV), ints(lens), bounds)
    for max_q in (None, 90, 5):
        got = sv.cache_score(q.to(DEV), bounds, table.to(DEV), ints(lens), starts(q_lens),
                             page_size=8, max_q=max_q).double().cpu()
        none = torch.isinf(want)
        assert torch.equal(none, torch.isinf(got))
        assert ((got - want).abs() <= tol)[~none].all()
