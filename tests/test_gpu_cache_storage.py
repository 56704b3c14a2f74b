"""What a round keeps of a step does not keep the step's token lists."""
import pytest
import torch

import speculative_decoding_rejection_02_gb300 as sv
from test_gpu_cache import DEV, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,tokens", [(3, 100000), (1, 0), (700, 5)])
def test_kept_lengths_do_not_hold_the_tokens(B, tokens):
    table = torch.full((B, 4), -1, dtype=torch.int32, device=DEV)
    free = torch.arange(B, dtype=torch.int32, device=DEV)
    r = sv.cache_step(ints([0] * B), ints([0] * B), table, free, ints([B]), page_size=16,
                      num_tokens=tokens)
    for kept in (r.lens, r.cu_new, r.free_count):
        assert kept.untyped_storage().nbytes() <= 4 * (2 * B + 2)
    for x in (r.positions, r.slots):
        assert x.untyped_storage().nbytes() <= 12 * tokens
    assert r.lens.shape == (B,) and r.cu_new.shape == (B + 1,) and r.free_count.shape == (1,)
    assert r.positions.shape == r.slots.shape == (tokens,)
    assert (r.positions == -1).all() and (r.slots == -1).all() and int(r.free_count) == B
