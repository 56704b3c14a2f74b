"""Arguments of the cache's calls that are of the wrong kind."""
import pytest
import torch

import speculative_decoding_rejection_02_gb300 as sv
from test_gpu_cache import BF, DEV, attend_case

pytestmark = pytest.mark.gpu


class NoTruth:
    def __bool__(self):
        raise ArithmeticError("neither")


def test_flag_without_a_truth_value():
    gpu, _ = attend_case([2], [50], 8, 2, 128, 16, BF)
    with pytest.raises(ArithmeticError):
        sv.cache_attend(**gpu, return_lse=NoTruth())
    assert len(sv.cache_attend(**gpu, return_lse=1)) == 2


def test_status_is_an_integer():
    gpu, _ = attend_case([2], [50], 8, 2, 128, 16, BF)
    for bad in (torch.zeros(1, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV),
                torch.zeros(1, dtype=torch.int64, device=DEV)):
        with pytest.raises(ValueError):
            sv.cache_attend(**gpu, status=bad)
    for good in (torch.int32, torch.uint32):
        sv.cache_attend(**gpu, status=torch.zeros(1, dtype=good, device=DEV))
