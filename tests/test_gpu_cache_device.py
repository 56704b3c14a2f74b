"""Tensors on another GPU than the current one (needs two)."""
import pytest
import torch

import cache_ref as ref
import speculative_decoding_rejection_02_gb300 as sv
from test_gpu_cache import BF, attend_case, status_word

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(torch.cuda.device_count() < 2,
                                                  reason="needs two GPUs")]


@pytest.mark.parametrize("current", [0, 1])
def test_attend_on_the_tensors_device(current):
    gpu, host = attend_case([3, 9], [333, 50], 8, 2, 128, 16, BF)
    there = {n: t.to("cuda:1") for n, t in gpu.items()}
    status = status_word().to("cuda:1")
    with torch.cuda.device(current):
        got, lse = sv.cache_attend(**there, return_lse=True, status=status)
        assert torch.cuda.current_device() == current
    assert got.device == lse.device == torch.device("cuda:1") and int(status) == 0
    ref.assert_attend(got, lse, ref.attend(*host))
