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
    weight is off by u^2, since its second part is off by u of what the first left over, at most u
    of it; and the output by its one rounding, u of it and of what it was off by already."""
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
    tol = tol + u * u * size
    tol = tol + u * (want.abs() + tol) + 2.0 ** -25   # (and an output below fp16's least normal)
    out = sv.cache_attend_selected(q.to(DEV), kp.to(DEV), vp.to(DEV), table.to(DEV), ints(kv_lens),
                                   starts(q_lens), sel.to(DEV)).double().cpu()
    over = ((out - want).abs() - tol).max()
    assert over <= 0, float(over)
    assert not math.isnan(float(out.sum()))
