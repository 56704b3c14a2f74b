"""cache_evict with table entries that are no pages: what goes back on the stack is pages alone."""
import pytest
import torch

import cache_ref
import sparse_ref as ref
import speculative_decoding_rejection_02_gb300 as sv
from test_gpu_sparse import BF, DEV, ints, same, status_word

pytestmark = pytest.mark.gpu

FORMS = [  # lengths, budgets, first, recent, page, kv heads, broken columns (request, column)
    ([70, 33, 200, 90], [40, 8, 5, 90], 2, 3, 16, 2, [(0, 4), (2, 1), (2, 12)]),  # short rows
    ([70, 33, 200], [0, 0, 0], 0, 0, 16, 1, [(0, 0), (1, 1), (1, 2), (2, 6)]),
    ([3000, 2500], [100, 2400], 0, 5, 8, 2, [(0, 100), (1, 311)]),
    ([9000, 100], [300, 100], 5, 5, 8, 2, [(0, 40), (0, 1124)]),                 # one block a row
    ([20000, 18000], [3000, 17000], 5, 100, 16, 2, [(0, 200), (1, 1124)]),       # clusters
    ([70000], [100], 0, 0, 64, 1, [(0, 2), (0, 1093)]),
    ([140000, 60], [0, 20], 0, 0, 32, 1, [(0, 4000), (0, 4374)])]                # any length


@pytest.mark.parametrize("lens,budget,first,recent,page,kv_heads,broken", FORMS)
@pytest.mark.parametrize("number", [-1, 2 ** 31 - 1, "pages"])
def test_numbers_that_are_no_pages_stay_off_the_stack(lens, budget, first, recent, page, kv_heads,
                                                      broken, number):
    g = torch.Generator().manual_seed(41)
    kp, vp, table, _, _ = cache_ref.cache(lens, page, kv_heads, 8, BF, g)
    pages = kp.shape[0]
    weights = torch.rand((pages, kv_heads, page), generator=g)
    held = {x for r, n in enumerate(lens) for x in table[r, : -(-n // page)].tolist()}
    spare = [x for x in range(pages) if x not in held]
    free = spare + [-9] * len(held)
    want_k, want_v, want_w, kept, want_free, want_count = ref.evict(
        kp, vp, weights, table, lens, budget, free, len(spare), first, recent)
    gone = {int(table[r, c]) for r, c in broken}
    for r, c in broken:
        assert c >= -(-kept[r] // page)  # (a column that is given back)
        table[r, c] = pages if number == "pages" else number
    want_free = [x for x in want_free[:want_count] if x not in gone]
    k, v, w, f = kp.to(DEV), vp.to(DEV), weights.to(DEV), ints(free)
    status = status_word()
    r = sv.cache_evict(k, v, w, table.to(DEV), ints(lens), ints(budget), f, ints([len(spare)]),
                       first=first, recent=recent, status=status)
    assert int(status) == sv.CACHE_BAD_PAGE
    assert r.lens.tolist() == kept
    assert int(r.free_count) == len(want_free)
    assert f.tolist()[: len(want_free)] == want_free
    for x in range(len(lens)):  # requests whose tables are whole
        if all(b != x for b, _ in broken):
            at = table[x, : -(-kept[x] // page)].long()
            assert same(k[at], want_k[at]) and same(v[at], want_v[at]) and same(w[at], want_w[at])
    # the next round hands out pages alone
    new = ints([1] + [0] * (len(lens) - 1))
    wide = torch.full((len(lens), table.shape[1] + 2), -1, dtype=torch.int32, device=DEV)
    wide[:, :-2] = table.to(DEV)
    step = sv.cache_step(r.lens, new, wide, f, r.free_count, page_size=page, num_tokens=1)
    assert 0 <= int(step.slots[0]) < pages * page


def test_a_broken_column_that_a_later_call_finds_whole():
    """One graph, replayed with a broken table and with a whole one: no call looks at what the one
    before found."""
    lens, page = [40, 64], 8
    g = torch.Generator().manual_seed(42)
    kp, vp, table, _, _ = cache_ref.cache(lens, page, 1, 8, BF, g)
    weights = torch.rand((kp.shape[0], 1, page), generator=g)
    k, v, w, t = kp.to(DEV), vp.to(DEV), weights.to(DEV), table.to(DEV)
    free, status = ints([-9] * kp.shape[0]), status_word()
    args = (k, v, w, t, ints(lens), ints([8, 8]), free, ints([0]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sv.cache_evict(*args, status=status)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = sv.cache_evict(*args, status=status)
    good = table[0, 1:5].tolist() + table[1, 1:8].tolist()
    for column in (2, None, 4, None):
        status.zero_()
        t.copy_(table)
        if column is not None:
            t[0, column] = -1
        graph.replay()
        want = [x for x in good if column is None or x != int(table[0, column])]
        assert int(status) == (0 if column is None else sv.CACHE_BAD_PAGE)
        assert int(got.free_count) == len(want) and free.tolist()[: len(want)] == want
