"""The arithmetic of the sparse-attention calls against 64 bits, held to what they state."""
import math

import pytest
import torch

import cache_ref
import sparse_ref as ref
import speculative_decoding_rejection_02_gb300 as sv
from test_gpu_sparse import BF, DEV, FP, inputs, ints, starts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("shape", [
    ([6], [6], 8, 8, 2, 128),                    # few tokens, whose weights' roundings stand out
    ([1], [3], 16, 4, 1, 64), ([1] * 40, [2 + i % 7 for i in range(40)], 8, 4, 2, 64),
    ([5, 3, 8, 1], [40, 9, 30, 100], 8, 4, 1, 72),
    ([9, 12], [20, 90], 16, 16, 1, 128)])        # 32 columns a block
def test_attend_selected_rounds_its_outputs_alone(shape, dtype):
    """Beside fp32's own errors (ref.attend's, without the rounding of the weights to the type) a
    weight is off by 2 u^2, since the first part, cut off, leaves less than 2 u of it, of which the
    second is off by u, and by 2^-23, which is added; and the output by its one rounding, u of it and
    of what it was off by already."""
    q_lens, kv_lens, page, heads, kv_heads, dim = shape
    g, q, kp, vp, table, ks, vs = inputs(shape, dtype, "token", 31)
    held = max(-(-n // page) for n in kv_lens)
    sel = torch.full((sum(q_lens), kv_heads, held), -1, dtype=torch.int32)
    for t, (_, pos) in enumerate(ref.positions(q_lens, kv_lens)):
        sel[t, :, : pos // page + 1] = torch.arange(pos // page + 1, dtype=torch.int32)
    want, lse, loose, _ = ref.attend(q, ks, vs, q_lens, sel, page)
    # what |out| would be with all values positive: the weights' errors meet these
    size = ref.attend(q, ks, [v.abs() for v in vs], q_lens, sel, page)[0]
    u = cache_ref.UNIT[dtype]
    tol = loose - 2 * u * size                   # fp32's errors
    tol = tol + (2 * u * u + 2.0 ** -23) * size
    tol = tol + u * (want.abs() + tol) + 2.0 ** -25   # (and an output below fp16's least normal)
    out = sv.cache_attend_selected(q.to(DEV), kp.to(DEV), vp.to(DEV), table.to(DEV), ints(kv_lens),
                                   starts(q_lens), sel.to(DEV)).double().cpu()
    over = ((out - want).abs() - tol).max()
    assert over <= 0, float(over)
    assert not math.isnan(float(out.sum()))


@pytest.mark.parametrize("q_size,b_size", [(1e-3, 1e35), (1e-30, 3e38), (1e-38, 3e38), (1.0, 1e35),
                                           (1e28, 1e7), (1e30, 1e-30), (3e38, 1e-5), (1e-20, 1e-10)])
@pytest.mark.parametrize("signs", ["mixed", "below", "above"])
def test_score_of_bounds_of_any_size(q_size, b_size, signs):
    """Scores that fp32 holds, of queries and finite bounds up to the type's largest (ref.score's
    error bounds, which count roundings relative to the sums of absolute values)."""
    g = torch.Generator().manual_seed(32)
    q = (torch.randn((3, 8, 64), generator=g).clamp(-1, 1) * q_size).to(BF)
    b = torch.randn((4, 2, 2, 64), generator=g).clamp(-1, 1)
    if signs != "mixed":  # P . hi and N . lo of opposite signs or one
        b = b.abs() * (1 if signs == "above" else -1)
    b = (b.sort(2).values * b_size).to(BF)
    assert torch.isfinite(b).all() and torch.isfinite(q).all()
    want, tol = ref.score(q, [b], [3], [60], 16, 4)
    got = sv.cache_score(q.to(DEV), b.to(DEV), ints([[0, 1, 2, 3]]), ints([60]), ints([0, 3]),
                         page_size=16).double().cpu()
    assert torch.isfinite(want).all() and want.abs().max() < 3e38
    over = ((got - want).abs() - tol).max()
    assert over <= 0, float(over)


def test_score_of_channels_of_different_sizes():
    """A channel of large queries and small bounds beside others the other way round."""
    g = torch.Generator().manual_seed(33)
    q, b = torch.randn((2, 4, 64), generator=g), torch.randn((3, 1, 2, 64), generator=g)
    q[..., 1:] *= 1e-25
    b[..., 0] *= 1e-30
    b[..., 1:] *= 1e20
    q, b = q.to(BF), b.sort(2).values.to(BF)
    want, tol = ref.score(q, [b], [2], [48], 16, 3)
    got = sv.cache_score(q.to(DEV), b.to(DEV), ints([[0, 1, 2]]), ints([48]), ints([0, 2]),
                         page_size=16).double().cpu()
    assert ((got - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("kv_heads,G,dim", [(2, 1, 128), (2, 1, 64), (4, 3, 96), (1, 8, 128)])
def test_score_sums_do_not_drift(dtype, kv_heads, G, dim):
    """Scores whose terms are all positive, in the mean over many. Two instructions' sums are cut off
    under 2^-23 of what they sum, half of that on average and the first one's half the pair: 0.75
    2^-23 at most; the additions after it and those of P and N round, 2^-24 / sqrt(3) each in the
    mean, of partial sums, in no direction: together under 2^-23."""
    g = torch.Generator().manual_seed(34)
    q = (torch.randn((40, kv_heads * G, dim), generator=g) * 1.5).to(dtype)
    b = torch.randn((64, kv_heads, 2, dim), generator=g).abs() + 1.0
    b[:, :, 0] *= -1.0
    b = b.to(dtype)
    want, _ = ref.score(q, [b], [40], [16 * 64], 16, 64)
    got = sv.cache_score(q.to(DEV), b.to(DEV), ints([list(range(64))]), ints([16 * 64]),
                         ints([0, 40]), page_size=16).double().cpu()
    there = torch.isfinite(want)
    off = (got[there] - want[there]) / want[there]
    assert float(off.pow(2).mean().sqrt()) < 2.0 ** -23
