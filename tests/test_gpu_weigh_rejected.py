"""cache_weigh after a verification: rows whose lse is -inf give nothing."""
import math

import pytest
import torch

import cache_ref
import sparse_ref as ref
import speculative_decoding_rejection_02_gb300 as sv
from test_gpu_sparse import BF, DEV, FP, inputs, ints, spread_weights, starts, status_word

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_lens,accepted,kv_lens,page,heads,kv_heads,dim,dtype", [
    ([5, 1, 3, 5], [2, 0, 0, 4], [300, 41, 3, 777], 16, 8, 2, 128, BF),
    ([8, 2], [0, 0], [64, 2], 8, 7, 1, 96, FP),
    ([140, 60, 1], [37, 0, 0], [900, 60, 500], 32, 4, 2, 64, BF)])   # several column tiles
def test_rejected_drafts_leave_nothing(q_lens, accepted, kv_lens, page, heads, kv_heads, dim, dtype):
    _, q, kp, vp, table, ks, vs = inputs((q_lens, kv_lens, page, heads, kv_heads, dim), dtype,
                                         "token", 81)
    g = torch.Generator().manual_seed(82)
    _, lse, _, _ = cache_ref.attend(q, ks, vs, q_lens)
    lse = lse.float()
    before = [torch.rand((kv_heads, n), generator=g) for n in kv_lens]
    weights = torch.full((kp.shape[0], kv_heads, page), -3.0)
    spread_weights(weights, before, table, page)
    # as if the rejected tokens had never been there
    stay = [torch.arange(n) <= a for n, a in zip(q_lens, accepted)]
    kept = [n - m + min(a + 1, m) for n, m, a in zip(kv_lens, q_lens, accepted)]
    rows = torch.cat(stay)
    want, tol = ref.weigh(q[rows], [k[:n] for k, n in zip(ks, kept)], [int(s.sum()) for s in stay],
                          lse[rows], [w[:, :n] for w, n in zip(before, kept)], decay=0.5)
    # the mask as sparse.py gives it
    lens, cu, acc = ints(kv_lens), starts(q_lens), ints(accepted)
    row = torch.arange(len(rows), device=DEV)
    request = torch.searchsorted(cu[1:], row, right=True)
    rejected = row - cu[request] > acc[request]
    assert torch.equal(rejected.cpu(), ~rows)
    got, status = weights.to(DEV), status_word()
    sv.cache_weigh(q.to(DEV), kp.to(DEV), table.to(DEV), lens, cu,
                   lse.to(DEV).masked_fill(rejected[:, None], -math.inf), got, decay=0.5,
                   status=status)
    assert int(status) == 0
    got = got.double().cpu()
    for r, (w, off) in enumerate(zip(want, tol)):
        mine = torch.cat([got[table[r, c]] for c in range(-(-kv_lens[r] // page))], 1)
        assert ((mine[:, : kept[r]] - w).abs() <= off).all(), r
        assert (mine[:, kept[r]: kv_lens[r]] == 0).all(), r  # slots of rejected tokens
