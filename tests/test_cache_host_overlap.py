"""spec_cache_step refuses arguments that overlap: every block reads all lengths while
others write already. The addresses are made up, so only where no kernel can start."""
import ctypes as C

import pytest
import torch

import speculative_decoding_rejection_02_gb300 as sv
from speculative_decoding_rejection_02_gb300 import _build

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")
B, T, WIDTH, STRIDE, PAGES = 5, 33, 7, 9, 40
INPUTS = dict(held_lens=4 * B, new_lens=4 * B, cu_num_draft=4 * (B + 1), num_accepted=4 * B,
              free_count=4)
UPDATED = dict(block_table=4 * ((B - 1) * STRIDE + WIDTH), free_pages=4 * PAGES)
OUTPUTS = dict(lens=4 * B, cu_new=4 * (B + 1), positions=4 * T, slots=8 * T, free_count_out=4)
SIZES = {**INPUTS, **UPDATED, **OUTPUTS}
WRITTEN = [*UPDATED, *OUTPUTS]


@pytest.fixture(scope="module")
def L():
    _build.build()
    return sv.lib()


def call(L, **kw):
    """All arguments apart from each other, but for those given."""
    at, places = 0x10000, {}
    for name, size in SIZES.items():
        places[name] = at
        at += (size + 15) // 8 * 8  # at least 8 bytes between
    places.update(kw)
    a = sv.StepArgs(B=B, width=WIDTH, table_stride=STRIDE, page_size=16, num_pages=PAGES,
                    num_tokens=T, **places)
    return L.spec_cache_step(C.byref(a), None, None), places


def test_apart_is_accepted(L):
    rc, places = call(L)
    assert rc == -2  # past the argument checks: no sm_103 here
    assert call(L, positions=None)[0] == -2
    assert call(L, new_lens=places["held_lens"], num_accepted=places["held_lens"])[0] == -2
    # one ends where the other begins
    assert call(L, lens=places["held_lens"] - 4 * B)[0] == -2
    assert call(L, cu_new=0x8000, lens=0x8000 + 4 * (B + 1))[0] == -2


@pytest.mark.parametrize("one", WRITTEN)
@pytest.mark.parametrize("other", list(SIZES))
def test_overlap_is_refused(L, one, other):
    if one == other:
        return
    places = call(L)[1]
    assert call(L, **{one: places[other]})[0] == -1                     # the same
    step = 8 if "slots" in (one, other) else 4
    assert call(L, **{one: places[other] - SIZES[one] // step * step + step})[0] == -1  # by its end
    if SIZES[other] > step:
        assert call(L, **{one: places[other] + SIZES[other] - step})[0] == -1
