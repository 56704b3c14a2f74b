"""Rows of q that no request owns, and requests whose offsets cannot be."""
import math

import pytest
import torch

import cache_ref as ref
import speculative_decoding_rejection_02_gb300 as sv
from test_gpu_cache import BF, DEV, attend_case, ints, status_word

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("offsets", [
    [2, 5, 5, 9], [9, 9, 9, 9], [0, 99, 2, 5], [0, -1, 3, 6], [7, 3, 6, 9], [0, 4, 4, 10],
    [3, 2, 1, 0], [1, 4, 3, 5], [-5, -2, 4, 4]])
@pytest.mark.parametrize("spread", [1, 200])
def test_rows_of_no_request(offsets, spread):
    """`spread` - 1 empty requests stand between the given ones."""
    T, kv = 9, [40, 700, 130]
    gpu, (q, ks, vs, _) = attend_case([3, 3, 3], kv, 8, 2, 128, 16, BF)
    cu, lens, table = [offsets[0]], [], []
    for r in range(3):
        cu += [offsets[r + 1]] * spread
        lens += [kv[r]] + [0] * (spread - 1)
        table += [gpu["block_table"][r: r + 1]] + [gpu["block_table"][:1]] * (spread - 1)
    gpu.update(cu_q=ints(cu), kv_lens=ints(lens), block_table=torch.cat(table))
    out, status = torch.full_like(gpu["q"], math.nan), status_word()
    got, lse = sv.cache_attend(**gpu, max_q=T, out=out, return_lse=True, status=status)
    assert got is out or got.data_ptr() == out.data_ptr()
    real = [lo >= 0 and lo <= hi <= T for lo, hi in zip(offsets, offsets[1:])]
    ends = [x for x in offsets if not 0 <= x <= T]
    assert int(status) == (0 if all(real) and not ends else sv.CACHE_BAD_LENGTHS)
    owned = set()
    for r in range(3):
        lo, hi = offsets[r], offsets[r + 1]
        rows = [t for t in range(max(lo, 0), hi) if real[r] and all(
            not (real[x] and offsets[x] <= t < offsets[x + 1]) for x in range(3) if x != r)]
        if real[r] and hi > lo:
            want = ref.attend(q[lo:hi], [ks[r]], [vs[r]], [hi - lo])
            at = [t - lo for t in rows]
            ref.assert_attend(got[rows], lse[rows], tuple(x[at] for x in want))
            owned |= set(range(lo, hi))
    nobody = [t for t in range(T) if t not in owned]
    assert (got[nobody] == 0).all() and (lse[nobody] == -math.inf).all()


def test_more_work_than_one_call_takes():
    """2^22 tokens in units of two over 2^31 are 2^45 steps: no row sees anything, and the status
    says so. (The pages are one page of 2^24 tokens over and over; none is read.)"""
    T, page = 2 ** 22, 2 ** 24
    pages = torch.zeros((1, page, 1, 8), dtype=BF, device=DEV)
    q = torch.ones((T, 1, 8), dtype=BF, device=DEV)
    out, status = torch.full_like(q, math.nan), status_word()
    table = torch.zeros((1, 128), dtype=torch.int32, device=DEV)
    got, lse = sv.cache_attend(q, pages, pages, table, ints([2 ** 31 - 2 ** 16]), ints([0, T]),
                               max_q=1, out=out, return_lse=True, status=status)
    assert int(status) == sv.CACHE_BAD_LENGTHS
    assert (got == 0).all() and (lse == -math.inf).all()
