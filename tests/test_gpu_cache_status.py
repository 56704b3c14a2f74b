"""Errors in device data of calls without a status word of their own."""
import os
import subprocess
import sys

import pytest
import torch

import speculative_decoding_rejection_02_gb300 as sv
from test_gpu_cache import BF, DEV, attend_case, ints, status_word

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean():
    sv.cache_status()


def bad_step(**kw):
    sv.cache_step(ints([0]), ints([40]), ints([[-1] * 9]), ints([3, 1]), ints([1]),
                  page_size=16, num_tokens=40, **kw)  # three pages wanted, one free


def bad_append(**kw):
    pages = torch.zeros((2, 16, 1, 64), dtype=BF, device=DEV)
    x = torch.ones((1, 1, 64), dtype=BF, device=DEV)
    sv.cache_append(x, x, torch.tensor([32], device=DEV), pages, pages.clone(), **kw)


def bad_attend(**kw):
    gpu, _ = attend_case([2, 3], [50, 60], 8, 2, 128, 16, BF)
    gpu["block_table"][1, 1] = 10 ** 6
    sv.cache_attend(**gpu, **kw)


CALLS = [(bad_step, sv.CACHE_NO_PAGES), (bad_append, sv.CACHE_BAD_SLOT),
         (bad_attend, sv.CACHE_BAD_PAGE)]


@pytest.mark.parametrize("call,bit", CALLS)
def test_bits_are_kept_until_read(call, bit):
    call()
    assert sv.cache_status() == bit
    assert sv.cache_status() == 0
    own = status_word()
    call(status=own)
    assert int(own) == bit and sv.cache_status() == 0


def test_bits_of_several_calls_and_streams():
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for k, (call, _) in enumerate(CALLS):
        call(stream=side if k == 1 else None)
    assert sv.cache_status(DEV) == sv.CACHE_NO_PAGES | sv.CACHE_BAD_SLOT | sv.CACHE_BAD_PAGE
    assert sv.cache_status(torch.device(DEV)) == 0


def test_good_calls_leave_none():
    gpu, _ = attend_case([2, 3], [50, 60], 8, 2, 128, 16, BF)
    sv.cache_attend(**gpu)
    assert sv.cache_status() == 0


def test_first_call_of_a_process_captured():
    """The word's address is found without breaking a capture."""
    code = """
import torch, speculative_decoding_rejection_02_gb300 as sv
pages = torch.zeros((2, 16, 1, 64), dtype=torch.bfloat16, device="cuda")
x, v = torch.ones((1, 1, 64), dtype=torch.bfloat16, device="cuda"), pages.clone()
slots = torch.tensor([32], device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    sv.cache_append(x, x, slots, pages, v)
assert sv.cache_status() == 0
graph.replay()
assert sv.cache_status() == sv.CACHE_BAD_SLOT
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], cwd=root, check=True, timeout=300)
