"""The paged-cache calls one right behind the other, where each reads what the one
before it wrote."""
import math

import pytest
import torch

import cache_ref as ref
import speculative_decoding_rejection_02_gb300 as sv
from test_gpu_cache import BF, DEV, ints, run_step, status_word, step_case

pytestmark = pytest.mark.gpu


def test_attend_reads_the_table_of_the_step_before_it():
    """Every round gives all pages back and takes them in another order, and the attention
    launched right behind it has to see the new order: page x holds the value x."""
    B, page, rounds = 61, 8, 200
    pages = B + 2
    k_pages = torch.zeros((pages, page, 1, 64), dtype=BF, device=DEV)
    v_pages = torch.arange(pages, device=DEV).view(-1, 1, 1, 1).expand(-1, page, 1, 64)
    v_pages = v_pages.to(BF).contiguous()
    table = torch.full((B, 2), -1, dtype=torch.int32, device=DEV)
    free, count = torch.arange(pages, dtype=torch.int32, device=DEV), ints([pages])
    lens, none, full = ints([0] * B), ints([0] * B), ints([page] * B)
    drafts = ints([page * r for r in range(B + 1)])
    q = torch.zeros((B, 1, 64), dtype=BF, device=DEV)
    cu_q, status = ints(list(range(B + 1))), status_word()
    kw = dict(page_size=page, num_tokens=page * B, status=status)
    tables, outs = [], []
    for k in range(rounds):
        # take a page each, look at it, drop its tokens and with them the page
        step = sv.cache_step(lens, full, table, free, count, **kw)
        outs.append(sv.cache_attend(q, k_pages, v_pages, table, step.lens, cu_q, max_q=1,
                                    status=status))
        tables.append(table[:, 0].clone())
        step = sv.cache_step(step.lens, none, table, free, step.free_count,
                             cu_num_draft=drafts, num_accepted=none, **kw)
        if k % 3 == 2:  # another order (all pages are free now)
            free = free.roll(k)
        lens, count = step.lens, step.free_count
    assert int(status) == 0
    for pages_held, out in zip(tables, outs):
        assert torch.equal(out[:, 0, 0].float(), pages_held.float())
    assert len({tuple(t.tolist()) for t in tables}) > 2


def plain_step(state, new, drafts, accepted, page, tokens):
    """The step in whole numbers on the host state (lens, table, free stack, count)."""
    want = ref.step(held=state["lens"], new=new, table=state["table"], free=state["free"],
                    count=state["count"], page=page, tokens=tokens, drafts=drafts,
                    accepted=accepted)
    assert want is not None
    state.update(lens=want["lens"], table=want["table"], free=want["free"],
                 count=want["free_count"])
    return want


@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3)])
def test_round_in_a_graph(window, sinks):
    """Step, append and attend captured as one round, replayed with other lengths, drafts,
    tokens and pages each time, against the plain forms on a cache kept beside it."""
    g = torch.Generator().manual_seed(5)
    B, heads, kv, dim, page, width, gamma = 7, 8, 2, 64, 8, 12, 4
    pages, T = 60, B * (gamma + 1) + 3
    k_pages = torch.full((pages, page, kv, dim), math.nan, dtype=BF, device=DEV)
    v_pages = torch.full_like(k_pages, math.nan)
    state = dict(lens=[0] * B, table=[[-1] * width for _ in range(B)], free=list(range(pages)),
                 count=pages)
    table, free = ints(state["table"]), ints(state["free"])
    held, new, cu_draft, accepted, count = (ints([0] * n) for n in (B, B, B + 1, B, 1))
    x = torch.zeros((T, heads + 2 * kv, dim), dtype=BF, device=DEV)
    out, status = torch.empty((T, heads, dim), dtype=BF, device=DEV), status_word()

    def round_():
        step = sv.cache_step(held, new, table, free, count, page_size=page, num_tokens=T,
                             cu_num_draft=cu_draft, num_accepted=accepted, status=status)
        sv.cache_append(x[:, heads:heads + kv], x[:, heads + kv:], step.slots, k_pages, v_pages,
                        status=status)
        _, lse = sv.cache_attend(x[:, :heads], k_pages, v_pages, table, step.lens, step.cu_new,
                                 max_q=gamma + 1, window=window, sinks=sinks, out=out,
                                 return_lse=True, status=status)
        return step, lse
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        round_()  # nothing held, nothing new
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step, lse = round_()
    dense = [torch.zeros((0, 2 * kv, dim), dtype=BF) for _ in range(B)]

    def pick(lo, hi):
        return torch.randint(lo, hi + 1, (B,), generator=g).tolist()
    drafts = [0] * B
    for k in range(9):
        acc = [min(a, d) for a, d in zip(pick(0, gamma), drafts)]
        fresh = [0] * B if k == 4 else pick(0, gamma + 1)
        if k == 6:  # some requests end: all their tokens are dropped
            drafts = [state["lens"][r] if r % 3 == 0 else drafts[r] for r in range(B)]
            acc = [0 if r % 3 == 0 else acc[r] for r in range(B)]
        for r in range(B):
            dense[r] = dense[r][: state["lens"][r] - drafts[r] + acc[r]]
        qkv = torch.randn((T, heads + 2 * kv, dim), generator=g).to(BF)
        # what the round reads, in place; what it writes, poisoned
        held.copy_(ints(state["lens"]))
        new.copy_(ints(fresh))
        cu_draft.copy_(ints([sum(drafts[:r]) for r in range(B + 1)]))
        accepted.copy_(ints(acc))
        count.copy_(ints([state["count"]]))
        x.copy_(qkv)
        for t in (out, lse):
            t.fill_(math.nan)
        for t in (*step,):
            t.fill_(-77)
        graph.replay()
        want = plain_step(state, fresh, drafts, acc, page, T)
        for name in ("lens", "cu_new", "positions", "slots"):
            assert getattr(step, name).tolist() == want[name], (k, name)
        assert int(step.free_count) == want["free_count"] and table.tolist() == want["table"]
        assert free.tolist()[: state["count"]] == want["free"][: state["count"]]
        at = 0
        for r, n in enumerate(fresh):
            dense[r] = torch.cat([dense[r], qkv[at: at + n, heads:]])
            at += n
            assert len(dense[r]) == state["lens"][r]
        ref.assert_attend(out[:at], lse[:at], ref.attend(
            qkv[:at, :heads], [d[:, :kv] for d in dense], [d[:, kv:] for d in dense], fresh,
            window=window, sinks=sinks))
        assert (out[at:] == 0).all() and (lse[at:] == -math.inf).all()
        drafts = [max(0, n - 1) for n in fresh]
    assert int(status) == 0


@pytest.mark.parametrize("B,new_hi,page", [(300, 1400, 16), (1500, 260, 5), (2000, 200, 16)])
def test_step_past_one_pass_of_its_grid(B, new_hi, page):
    """More token slots than the grid's threads (up to 152 x 1024), with pages taken and given
    back in numbers past them too."""
    c = step_case(B, page, B, new_hi=new_hi, ctx_hi=900)
    c["drafts"] = [h // 2 if r % 2 else d for r, (h, d) in enumerate(zip(c["held"], c["drafts"]))]
    c["accepted"] = [0 if r % 2 else a for r, a in enumerate(c["accepted"])]
    want = ref.step(**c)
    assert want is not None and c["tokens"] > 170000
    got, status = run_step(c)
    assert status == 0 and got == want
