"""Scores are taken times scale * log2(e) in fp32: a scale that overflows there is refused."""
import ctypes as C

import pytest

import speculative_decoding_rejection_02_gb300 as sv
from speculative_decoding_rejection_02_gb300 import _build
from test_cache_host import attend_args


@pytest.mark.parametrize("scale,fits", [
    (3.0e38, False), (-3.0e38, False), (2.36e38, False), (float("-inf"), False),
    (2.35e38, True), (-2.35e38, True), (0.0, True), (1e-45, True)])
def test_scale(scale, fits):
    _build.build()
    rc = sv.lib().spec_cache_attend(C.byref(attend_args(scale=scale)), None, None)
    # past that check: no workspace here, or no sm_103
    assert rc == -1 if not fits else rc in (-2, -5)
