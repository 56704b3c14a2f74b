"""Arguments of the cache's calls that are of the wrong kind."""
import pytest

import speculative_decoding_rejection_02_gb300 as sv
from test_gpu_cache import BF, attend_case

pytestmark = pytest.mark.gpu


class NoTruth:
    def __bool__(self):
        raise ArithmeticError("neither")


def test_flag_without_a_truth_value():
    gpu, _ = attend_case([2], [50], 8, 2, 128, 16, BF)
    with pytest.raises(ArithmeticError):
        sv.cache_attend(**gpu, return_lse=NoTruth())
    assert len(sv.cache_attend(**gpu, return_lse=1)) == 2

