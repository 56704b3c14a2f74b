"""spec_cache_status without a device."""
import ctypes as C

import pytest
import torch

import speculative_decoding_rejection_02_gb300 as sv
from speculative_decoding_rejection_02_gb300 import _build


def test_refusals():
    _build.build()
    L = sv.lib()
    assert "spec_cache_status" in sv.CACHE_ENTRY_POINTS
    assert L.spec_cache_status(None) == -1
    if not torch.cuda.is_available():
        assert L.spec_cache_status(C.byref(C.c_uint())) == -2
        with pytest.raises((sv.SpecVerifyError, RuntimeError, AssertionError)):
            sv.cache_status()
