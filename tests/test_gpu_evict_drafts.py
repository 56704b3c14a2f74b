"""Eviction between the append of a round's drafts and their verdict, and after it: the drop of
rejected drafts takes drafts alone."""
import pytest
import torch

import speculative_decoding_rejection_02_gb300 as sv
from test_gpu_sparse import BF, DEV, ints, status_word

pytestmark = pytest.mark.gpu

KV, PAGE, PAGES, WIDTH = 2, 8, 96, 20
HELD, NEW, ACCEPTED, BUDGET = [60, 33, 90, 7], [5, 3, 5, 1], [0, 2, 4, 0], [24, 20, 30, 40]
OLD = [n - m for n, m in zip(HELD, NEW)]


class Cache:
    """Pages whose keys say which token they hold: request * 256 + position. Old tokens have
    random weights, new ones less than any of those."""

    def __init__(self):
        g = torch.Generator().manual_seed(71)
        self.table = torch.full((4, WIDTH), -1, dtype=torch.int32, device=DEV)
        self.free = torch.arange(PAGES, dtype=torch.int32, device=DEV)
        self.status = status_word()
        step = sv.cache_step(ints([0] * 4), ints(HELD), self.table, self.free, ints([PAGES]),
                             page_size=PAGE, num_tokens=sum(HELD), status=self.status)
        self.k = torch.zeros((PAGES, PAGE, KV, 8), dtype=BF, device=DEV)
        self.v = torch.zeros_like(self.k)
        self.w = torch.zeros((PAGES, KV, PAGE), device=DEV)
        label = torch.tensor([256 * r + j for r, n in enumerate(HELD) for j in range(n)])
        x = torch.stack([label // 256, label % 256], 1).to(DEV, BF)  # both exact
        rows = torch.zeros((label.numel(), KV, 8), dtype=BF, device=DEV)
        rows[:, :, :2] = x[:, None]
        sv.cache_append(rows, rows, step.slots, self.k, self.v, status=self.status)
        for r, n in enumerate(HELD):
            for j in range(n):
                w = torch.rand((KV,), generator=g) + 1.0 if j < OLD[r] else torch.full((KV,), 0.01)
                self.w[int(self.table[r, j // PAGE]), :, j % PAGE] = w.to(DEV)
        self.count = step.free_count

    def evict(self, lens, recent):
        r = sv.cache_evict(self.k, self.v, self.w, self.table, lens, ints(BUDGET), self.free,
                           self.count, recent=recent, status=self.status)
        self.count = r.free_count
        return r.lens

    def drop(self, lens, new):
        """The step after the verdict."""
        drafts = [m - 1 for m in NEW]
        cu = ints([sum(drafts[:i]) for i in range(5)])
        step = sv.cache_step(lens, ints(new), self.table, self.free, self.count, page_size=PAGE,
                             num_tokens=sum(new), cu_num_draft=cu, num_accepted=ints(ACCEPTED),
                             status=self.status)
        self.count = step.free_count
        return step.lens

    def held(self, lens):
        """The positions that each request and kv head holds, of its own tokens alone."""
        out = []
        for r, n in enumerate(lens):
            j = torch.arange(n, device=DEV)
            rows = self.k[self.table[r].long()[j // PAGE], j % PAGE].float()
            assert (rows[:, :, 0] == r).all()
            out.append(rows[:, :, 1].long().T.tolist())
        assert int(self.status) == 0
        return out


KEPT = [n - (m - 1 - a) for n, m, a in zip(HELD, NEW, ACCEPTED)]  # without rejected drafts


@pytest.mark.parametrize("new", [[0] * 4, [5, 5, 1, 2]])
def test_before_the_drop_with_all_new_tokens_recent(new):
    c = Cache()
    lens = c.evict(ints(HELD), max(NEW))
    assert lens.tolist() == [min(n, b) for n, b in zip(HELD, BUDGET)]
    lens = c.drop(lens, new).tolist()
    held = c.held([n - m for n, m in zip(lens, new)])
    for r, heads in enumerate(held):
        fresh = list(range(OLD[r], KEPT[r]))
        for x in heads:
            assert x == sorted(x) and x[-1] < KEPT[r]          # no rejected draft
            assert x[len(x) - len(fresh):] == fresh            # every accepted one


def test_after_a_drop_without_new_tokens():
    c = Cache()
    lens = c.drop(ints(HELD), [0] * 4)
    assert lens.tolist() == KEPT
    lens = c.evict(lens, 0).tolist()
    assert lens == [min(n, b) for n, b in zip(KEPT, BUDGET)]
    for r, heads in enumerate(c.held(lens)):
        for x in heads:
            assert x == sorted(x) and x[-1] < KEPT[r]


def test_positions_alone_tell_what_a_step_drops():
    """What the header warns of: drafts go first where `recent` does not hold them, and the step
    then takes old tokens."""
    c = Cache()
    lens = c.drop(c.evict(ints(HELD), 0), [0] * 4).tolist()
    first = c.held(lens)[0][0]
    assert len(first) == BUDGET[0] - 4 and max(first) < OLD[0] and len(set(first)) == len(first)
