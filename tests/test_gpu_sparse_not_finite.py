"""cache_attend_selected with keys and values that are not finite: which rows they reach."""
import math

import pytest
import torch

import cache_ref
import sparse_ref as ref
import speculative_decoding_rejection_02_gb300 as sv
from test_gpu_sparse import BF, DEV, FP, inputs, ints, starts

pytestmark = pytest.mark.gpu

SHAPE = ([6, 1, 9], [120, 40, 90], 8, 8, 2, 64)
TOKEN, HEAD, COLUMN, CHANNEL = 3, 1, 4, 10  # the row and page that meet in request 0


def given(dtype):
    """Random inputs, where of request 0 and kv head 1 only token 3 selects column 4."""
    q_lens, kv_lens, page, heads, kv_heads, dim = SHAPE
    _, q, kp, vp, table, ks, vs = inputs(SHAPE, dtype, "token", 61)
    sel = torch.full((sum(q_lens), kv_heads, 6), -1, dtype=torch.int32)
    for t, (r, pos) in enumerate(ref.positions(q_lens, kv_lens)):
        columns = [c for c in (0, 2, 3, 5, 7) if c <= pos // page]
        sel[t, :, : len(columns)] = torch.tensor(columns, dtype=torch.int32)
    sel[TOKEN, HEAD] = torch.tensor([0, 2, COLUMN, 5, 7, -1], dtype=torch.int32)
    want = ref.attend(q, ks, vs, q_lens, sel, page)
    return q, kp, vp, table, sel, want


def attend(q, kp, vp, table, sel):
    return sv.cache_attend_selected(q.to(DEV), kp.to(DEV), vp.to(DEV), table.to(DEV),
                                    ints(SHAPE[1]), starts(SHAPE[0]), sel.to(DEV), return_lse=True)


def group(x):
    """The rows of request 0 and kv head 1 of an output."""
    G = SHAPE[3] // SHAPE[4]
    return x[: SHAPE[0][0], HEAD * G:(HEAD + 1) * G]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_a_value_stays_in_its_request_head_and_channel(dtype, value):
    q, kp, vp, table, sel, want = given(dtype)
    vp[table[0, COLUMN], 3, HEAD, CHANNEL] = value
    out, lse = attend(q, kp, vp, table, sel)
    assert not torch.isfinite(group(out)[TOKEN, :, CHANNEL]).any()
    # the other rows of the group may have it in its channel; there is nothing anywhere else
    rest = out.double().cpu().clone()
    mine = group(rest)[:, :, CHANNEL]
    other = ~torch.isfinite(mine)
    assert other[TOKEN].all()
    mine[other] = group(want[0])[:, :, CHANNEL][other]
    cache_ref.assert_attend(rest, lse, want)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_a_key_stays_with_the_rows_that_see_it(dtype, value):
    q, kp, vp, table, sel, want = given(dtype)
    kp[table[0, COLUMN], 3, HEAD, CHANNEL] = value
    out, lse = attend(q, kp, vp, table, sel)
    for x, y in ((out, want[0]), (lse, want[1])):  # the row that sees it may be anything
        group(x)[TOKEN] = group(y)[TOKEN].to(x)
    cache_ref.assert_attend(out, lse, want)


def test_one_token_alone_sees_its_own_list():
    """Requests of one token each: no row shares a product with another's."""
    q, kp, vp, table, sel, want = given(BF)
    vp[table[0, COLUMN], 3, HEAD] = math.nan
    for t in range(SHAPE[0][0]):
        n = SHAPE[1][0] - SHAPE[0][0] + t + 1
        out = sv.cache_attend_selected(q[t:t + 1].to(DEV), kp.to(DEV), vp.to(DEV),
                                       table[:1].to(DEV), ints([n]), ints([0, 1]),
                                       sel[t:t + 1].to(DEV))
        bad = torch.isnan(out).flatten(1).any(1)
        assert bool(bad) == (t == TOKEN)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("tokens", [1, 4])
def test_an_infinite_value_that_a_row_sees_stays_infinite(dtype, tokens):
    """Keys of one direction, so that many weights are the same power of two, which the type holds
    without a rest, and others that it does not hold."""
    g = torch.Generator().manual_seed(62)
    n, page, dim = 64, 16, 64
    k = torch.ones((4, page, 1, dim), dtype=dtype)
    k[1::2] *= torch.rand((2, page, 1, 1), generator=g).to(dtype)
    v = torch.randn((4, page, 1, dim), generator=g).to(dtype)
    v[0, 5, 0, 3], v[1, 6, 0, 7] = math.inf, -math.inf
    q = torch.full((tokens, 2, dim), 0.25, dtype=dtype)
    q[:, 1] = 0
    sel = torch.arange(4, dtype=torch.int32).expand(tokens, 1, 4).contiguous()
    out = sv.cache_attend_selected(q.to(DEV), k.to(DEV), v.to(DEV), ints([[0, 1, 2, 3]]), ints([n]),
                                   ints([0, tokens]), sel.to(DEV))
    assert (out[:, :, 3] == math.inf).all() and (out[:, :, 7] == -math.inf).all()
    assert int(torch.isfinite(out).sum()) == tokens * 2 * (dim - 2)
