"""The paged-cache calls one right behind the other, where each reads what the one
before it wrote."""
import pytest
import torch

import speculative_decoding_rejection_02_gb300 as sv
from test_gpu_cache import BF, DEV, ints, status_word

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
