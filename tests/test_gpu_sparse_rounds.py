"""The sparse-attention and eviction calls as they are used: rounds of step, append, bounds,
score, select, attend, weigh and evict one behind the other, eagerly and captured."""
import math

import pytest
import torch

import cache_ref
import sparse_ref as ref
import speculative_decoding_rejection_02_gb300 as sv
from test_gpu_sparse import BF, DEV, ints, status_word

pytestmark = pytest.mark.gpu

B, HEADS, KV, DIM, PAGE, WIDTH, PAGES, COUNT = 5, 8, 2, 64, 16, 14, 80, 4


class Plain:
    """The cache as dense tensors on the CPU, one list of tokens for each request and kv head."""

    def __init__(self):
        self.k = [torch.zeros((0, KV, DIM), dtype=BF) for _ in range(B)]
        self.v = [torch.zeros((0, KV, DIM), dtype=BF) for _ in range(B)]
        self.w = [torch.zeros((KV, 0), dtype=torch.float64) for _ in range(B)]


def buffers():
    nan = torch.full((PAGES, PAGE, KV, DIM), math.nan, dtype=BF, device=DEV)
    return dict(k=nan.clone(), v=nan.clone(),
                weights=torch.full((PAGES, KV, PAGE), math.nan, device=DEV),
                bounds=torch.full((PAGES, KV, 2, DIM), math.nan, dtype=BF, device=DEV),
                table=torch.full((B, WIDTH), -1, dtype=torch.int32, device=DEV),
                free=torch.arange(PAGES, dtype=torch.int32, device=DEV))


def one_round(x, held, new, count, qkv, budget, tokens, status, cu_draft=None, accepted=None):
    """Every call of a round, without a look at its results."""
    step = sv.cache_step(held, new, x["table"], x["free"], count, page_size=PAGE,
                         num_tokens=tokens, cu_num_draft=cu_draft, num_accepted=accepted,
                         status=status)
    q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], qkv[:, HEADS + KV:]
    sv.cache_append(k, v, step.slots, x["k"], x["v"], status=status)
    sv.cache_bounds(x["k"], x["table"], step.lens, x["bounds"], cu_q=step.cu_new, max_q=40,
                    status=status)
    scores = sv.cache_score(q, x["bounds"], x["table"], step.lens, step.cu_new, page_size=PAGE,
                            max_q=40, status=status)
    selected = sv.cache_select(scores, step.lens, step.cu_new, page_size=PAGE, count=COUNT,
                               first=1, recent=1, status=status)
    sparse, sparse_lse = sv.cache_attend_selected(q, x["k"], x["v"], x["table"], step.lens,
                                                  step.cu_new, selected, return_lse=True,
                                                  status=status)
    full, lse = sv.cache_attend(q, x["k"], x["v"], x["table"], step.lens, step.cu_new, max_q=40,
                                return_lse=True, status=status)
    sv.cache_weigh(q, x["k"], x["table"], step.lens, step.cu_new, lse, x["weights"], max_q=40,
                   decay=0.75, status=status)
    kept = sv.cache_evict(x["k"], x["v"], x["weights"], x["table"], step.lens, budget, x["free"],
                          step.free_count, first=2, recent=12, status=status)
    sv.cache_bounds(x["k"], x["table"], kept.lens, x["bounds"], status=status)
    return dict(lens=step.lens, scores=scores, selected=selected, sparse=sparse,
                sparse_lse=sparse_lse, full=full, lse=lse, kept=kept.lens, count=kept.free_count,
                weights=x["weights"])


def check_round(plain, x, got, qkv, q_lens, gone, budget):
    """Against the plain forms, each on the inputs that the GPU's calls had; the plain cache then
    goes on with what the GPU selected."""
    cu, t0 = 0, 0
    q = qkv[: sum(q_lens), :HEADS].cpu()
    table = x["table"].cpu()
    for r in range(B):
        new = qkv[t0: t0 + q_lens[r]].cpu()
        n = plain.k[r].shape[0] - gone[r]
        plain.k[r] = torch.cat([plain.k[r][:n], new[:, HEADS:HEADS + KV]])
        plain.v[r] = torch.cat([plain.v[r][:n], new[:, HEADS + KV:]])
        plain.w[r] = torch.cat([plain.w[r][:, :n], torch.zeros((KV, q_lens[r])).double()], 1)
        t0 += q_lens[r]
    lens = [k.shape[0] for k in plain.k]
    assert got["lens"].tolist() == lens
    T = sum(q_lens)
    pages = [torch.stack(p) if p else torch.zeros((0, KV, 2, DIM))
             for p in ref.bounds(plain.k, PAGE)]
    want, tol = ref.score(q, pages, q_lens, lens, PAGE, WIDTH)
    scores = got["scores"][:T].cpu()
    none = torch.isinf(want)
    assert torch.equal(none, torch.isinf(scores))
    assert ((scores.double() - want).abs() <= tol)[~none].all()
    selected = got["selected"][:T].cpu()
    assert torch.equal(selected, ref.select(scores, q_lens, lens, PAGE, COUNT, 1, 1))
    cache_ref.assert_attend(got["sparse"][:T], got["sparse_lse"][:T],
                            ref.attend(q, plain.k, plain.v, q_lens, selected, PAGE))
    cache_ref.assert_attend(got["full"][:T], got["lse"][:T],
                            cache_ref.attend(q, plain.k, plain.v, q_lens))
    want, tol = ref.weigh(q, plain.k, q_lens, got["lse"][:T].cpu(), plain.w, decay=0.75)
    weights, kept = got["weights"].cpu(), []
    for r in range(B):
        m = min(lens[r], max(budget[r], 14))
        kept.append(m)
        stay = []
        for h in range(KV):
            w = want[r][h]
            order = sorted(range(2, lens[r] - 12), key=lambda j: (-w[j].item(), j))
            best = sorted(set(range(min(2, lens[r]))) | set(range(max(0, lens[r] - 12), lens[r]))
                          | set(order[: max(0, m - 14)]))
            stay.append(best if m < lens[r] else list(range(lens[r])))
            # the weight at the border is far from its neighbour beside its error, or another
            # token might rightly have been kept
            if m < lens[r] and 14 < m:
                gap = w[order[m - 15]] - w[order[m - 14]]
                assert gap > 2 * tol[r][h].max(), "the test's own data: choose another seed"
        at = torch.tensor(stay, dtype=torch.long).T  # [kept, KV]
        heads = torch.arange(KV)
        plain.k[r], plain.v[r] = plain.k[r][at, heads], plain.v[r][at, heads]
        off = tol[r].T[at, heads].T
        plain.w[r] = want[r].T[at, heads].T.contiguous()
        mine = [weights[table[r, c]] for c in range(-(-m // PAGE))]
        mine = torch.cat(mine, 1)[:, :m].double() if mine else plain.w[r]
        assert ((mine - plain.w[r]).abs() <= off).all()
        plain.w[r] = mine  # (the next round starts from what the GPU has)
        if m:
            slots = torch.arange(m)
            where = table[r, slots // PAGE].long()
            assert torch.equal(x["k"].cpu()[where, slots % PAGE], plain.k[r])
            assert torch.equal(x["v"].cpu()[where, slots % PAGE], plain.v[r])
    assert got["kept"].tolist() == kept
    held = sum(-(-m // PAGE) for m in kept)
    assert int(got["count"]) == PAGES - held
    rest = x["free"][: PAGES - held].tolist()
    used = [int(table[r, c]) for r in range(B) for c in range(-(-kept[r] // PAGE))]
    assert sorted(rest + used) == list(range(PAGES))


ROUNDS = [  # new tokens, accepted drafts of the round before
    ([40, 3, 17, 0, 30], None), ([5, 5, 5, 5, 5], None), ([1, 4, 5, 2, 3], [4, 0, 2, 1, 3]),
    ([5, 5, 5, 5, 5], [0, 3, 1, 1, 0]), ([1, 1, 1, 1, 1], [4, 4, 4, 4, 4])]


def data(r, T):
    g = torch.Generator().manual_seed(100 + r)
    return torch.randn((T, HEADS + 2 * KV, DIM), generator=g).to(BF).to(DEV)


def rounds():
    """(new tokens, dropped of the round before, offsets of drafts, accepted), new before first."""
    before = None
    for new, accepted in ROUNDS:
        drafts = None if accepted is None else [max(n - 1, 0) for n in before]
        gone = [0] * B if drafts is None else [d - min(a, d) for d, a in zip(drafts, accepted)]
        yield new, gone, drafts, accepted
        before = new


def test_rounds():
    plain, x, status = Plain(), buffers(), status_word()
    lens, count = ints([0] * B), ints([PAGES])
    budget = [24, 30, 20, 64, 16]
    for r, (new, gone, drafts, accepted) in enumerate(rounds()):
        qkv = data(r, sum(new) + 3)
        cu = acc = None
        if drafts:
            cu = ints([sum(drafts[:i]) for i in range(B + 1)])
            acc = ints([min(a, d) for d, a in zip(drafts, accepted)])
        got = one_round(x, lens, ints(new), count, qkv, ints(budget), qkv.shape[0], status, cu, acc)
        assert int(status) == 0
        check_round(plain, x, got, qkv, new, gone, budget)
        lens, count = got["kept"], got["count"]


def test_rounds_in_a_graph():
    """One round captured, replayed with other lengths, tokens and pages each time; a second graph
    of the same calls is replayed between, on a cache of its own."""
    tokens = 100

    def capture():
        x = buffers()
        io = dict(held=ints([0] * B), new=ints([1] * B), count=ints([PAGES]),
                  qkv=torch.zeros((tokens, HEADS + 2 * KV, DIM), dtype=BF, device=DEV),
                  budget=ints([16] * B), status=status_word(), cu=ints([0] * (B + 1)),
                  acc=ints([0] * B))
        start = {k: v.clone() for k, v in x.items()}

        def run():
            return one_round(x, io["held"], io["new"], io["count"], io["qkv"], io["budget"], tokens,
                             io["status"], io["cu"], io["acc"])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run()
        for k, v in start.items():
            x[k].copy_(v)
        return graph, x, io, got

    graphs = [capture(), capture()]
    plains = [Plain(), Plain()]
    state = [([0] * B, PAGES)] * 2
    budgets = [[24, 30, 20, 64, 16], [100, 18, 15, 14, 40]]
    for r, (new, gone, drafts, accepted) in enumerate(rounds()):
        for i, (graph, x, io, got) in enumerate(graphs):
            qkv = data(r + 50 * i, sum(new))
            io["held"].copy_(torch.tensor(state[i][0]))
            io["new"].copy_(torch.tensor(new))
            io["count"].fill_(state[i][1])
            io["qkv"].zero_()
            io["qkv"][: sum(new)] = qkv
            io["budget"].copy_(torch.tensor(budgets[i]))
            d = drafts or [0] * B
            a = [min(z, y) for y, z in zip(d, accepted or [0] * B)]
            io["cu"].copy_(torch.tensor([sum(d[:j]) for j in range(B + 1)]))
            io["acc"].copy_(torch.tensor(a))
            graph.replay()
        for i, (graph, x, io, got) in enumerate(graphs):
            assert int(io["status"]) == 0
            check_round(plains[i], x, got, io["qkv"], new, gone, budgets[i])
            state[i] = (got["kept"].tolist(), int(got["count"]))


def test_rounds_on_another_stream():
    """Two caches on two streams at once, the calls' ``stream`` argument and the current stream."""
    results = []
    for _ in range(2):
        streams = [torch.cuda.Stream() for _ in range(2)]
        caches, outs = [buffers(), buffers()], [None, None]
        status = [status_word(), status_word()]
        lens = [(ints([0] * B), ints([PAGES])) for _ in range(2)]
        qkvs = [data(r, sum(new)) for r, (new, _) in enumerate(ROUNDS[:2])]
        budget, news = ints([24] * B), [ints(new) for new, _ in ROUNDS[:2]]
        torch.cuda.synchronize()
        for r, (new, _) in enumerate(ROUNDS[:2]):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    outs[i] = one_round(caches[i], lens[i][0], news[r], lens[i][1], qkvs[r], budget,
                                        sum(new), status[i])
                lens[i] = (outs[i]["kept"], outs[i]["count"])
        torch.cuda.synchronize()
        assert [int(s) for s in status] == [0, 0]
        for k in outs[0]:
            if k != "weights":
                assert torch.equal(outs[0][k], outs[1][k]), k
        results.append(outs[0])
    for k in ("sparse", "scores", "kept"):
        assert torch.equal(results[0][k], results[1][k])


def test_stream_argument():
    x, y = buffers(), buffers()
    new, qkv, status = ROUNDS[0][0], data(0, sum(ROUNDS[0][0])), status_word()
    want = one_round(x, ints([0] * B), ints(new), ints([PAGES]), qkv, ints([24] * B), sum(new), status)
    step = sv.cache_step(ints([0] * B), ints(new), y["table"], y["free"], ints([PAGES]),
                         page_size=PAGE, num_tokens=sum(new), status=status)
    q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], qkv[:, HEADS + KV:]
    sv.cache_append(k, v, step.slots, y["k"], y["v"], status=status)
    full, lse = sv.cache_attend(q, y["k"], y["v"], y["table"], step.lens, step.cu_new,
                                return_lse=True, status=status)
    budget = ints([24] * B)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    kw = dict(status=status, stream=s)
    sv.cache_bounds(y["k"], y["table"], step.lens, y["bounds"], cu_q=step.cu_new, **kw)
    scores = sv.cache_score(q, y["bounds"], y["table"], step.lens, step.cu_new, page_size=PAGE, **kw)
    selected = sv.cache_select(scores, step.lens, step.cu_new, page_size=PAGE, count=COUNT, first=1,
                               **kw)
    sparse = sv.cache_attend_selected(q, y["k"], y["v"], y["table"], step.lens, step.cu_new,
                                      selected, **kw)
    sv.cache_weigh(q, y["k"], y["table"], step.lens, step.cu_new, lse, y["weights"], decay=0.75, **kw)
    kept = sv.cache_evict(y["k"], y["v"], y["weights"], y["table"], step.lens, budget, y["free"],
                          step.free_count, first=2, recent=12, **kw)
    s.synchronize()
    assert int(status) == 0
    assert torch.equal(scores, want["scores"]) and torch.equal(selected, want["selected"])
    assert torch.equal(sparse, want["sparse"]) and torch.equal(kept.lens, want["kept"])
