"""Argument checks of the paged-cache calls, which need no device: the C ABI's
(before anything is enqueued) and the binding's."""
import ctypes as C

import pytest
import torch

import speculative_decoding_rejection_02_gb300 as sv
from speculative_decoding_rejection_02_gb300 import _build

OK_HERE = 0 if torch.cuda.is_available() else -2  # no sm_103 here: refused after the checks
FAKE = 0x1000  # host-side checks never dereference


@pytest.fixture(scope="module")
def L():
    _build.build()
    return sv.lib()


def fields(kind, base, kw):
    base.update(kw)
    return kind(**base)


def step_args(**kw):
    return fields(sv.StepArgs, dict(
        B=4, width=8, table_stride=8, page_size=16, num_pages=64, num_tokens=0, held_lens=FAKE,
        new_lens=FAKE, cu_num_draft=FAKE, num_accepted=FAKE, block_table=FAKE, free_pages=FAKE,
        free_count=FAKE, lens=FAKE + 64, cu_new=FAKE, positions=FAKE, slots=FAKE,
        free_count_out=FAKE + 64), kw)


def append_args(**kw):
    return fields(sv.AppendArgs, dict(
        num_tokens=4, kv_heads=2, dim=64, page_size=16, num_pages=8, dtype=1, k=FAKE,
        k_token=128, k_head=64, v=FAKE, v_token=128, v_head=64, slots=FAKE, k_pages=FAKE,
        kp_page=2048, kp_token=128, kp_head=64, v_pages=FAKE, vp_page=2048, vp_token=128,
        vp_head=64), kw)


def attend_args(**kw):
    return fields(sv.AttendArgs, dict(
        B=2, num_tokens=4, max_q=2, heads=8, kv_heads=2, dim=64, page_size=16, width=8,
        num_pages=8, dtype=1, q=FAKE, q_token=512, q_head=64, k_pages=FAKE, kp_page=2048,
        kp_token=128, kp_head=64, v_pages=FAKE, vp_page=2048, vp_token=128, vp_head=64,
        block_table=FAKE, table_stride=8, kv_lens=FAKE, cu_q=FAKE, out=FAKE, out_token=512,
        out_head=64, lse=None, scale=0.125, window=0, sinks=0, workspace=None,
        workspace_bytes=0), kw)


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), -1), (dict(width=0), -1), (dict(table_stride=7), -1), (dict(page_size=0), -1),
    (dict(num_pages=0), -1), (dict(num_tokens=-1), -1), (dict(held_lens=None), -1),
    (dict(new_lens=None), -1), (dict(block_table=None), -1), (dict(free_pages=None), -1),
    (dict(free_count=None), -1), (dict(lens=None), -1), (dict(cu_new=None), -1),
    (dict(free_count_out=None), -1), (dict(num_tokens=3, slots=None), -1),
    (dict(num_accepted=None), -1), (dict(cu_num_draft=None), -1),
    (dict(lens=FAKE), -1), (dict(free_count_out=FAKE), -1)])
def test_step_refuses(L, kw, rc):
    assert L.spec_cache_step(C.byref(step_args(**kw)), None, None) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(num_tokens=-1), -1), (dict(kv_heads=0), -1), (dict(dim=0), -1),
    (dict(page_size=0), -1), (dict(num_pages=0), -1), (dict(dtype=0), -1), (dict(dtype=3), -1),
    (dict(k=None), -1), (dict(v=None), -1), (dict(slots=None), -1), (dict(k_pages=None), -1),
    (dict(v_pages=None), -1), (dict(k_token=-1), -1), (dict(k=FAKE + 1), -1),
    (dict(kv_heads=1 << 15, dim=1 << 10), -2)])
def test_append_refuses(L, kw, rc):
    assert L.spec_cache_append(C.byref(append_args(**kw)), None, None) == rc


ATTEND_SIZES = [
    (dict(B=-1), -1), (dict(num_tokens=-1), -1), (dict(max_q=0), -1), (dict(heads=0), -1),
    (dict(kv_heads=0), -1), (dict(kv_heads=3), -1), (dict(dim=0), -1), (dict(page_size=0), -1),
    (dict(width=0), -1), (dict(num_pages=0), -1), (dict(dtype=0), -1), (dict(window=-1), -1),
    (dict(sinks=-1), -1), (dict(dim=60), -2), (dict(dim=136), -2), (dict(page_size=4), -2),
    (dict(page_size=48), -2), (dict(heads=129, kv_heads=1), -2), (dict(num_pages=1 << 31), -2)]
ATTEND_POINTERS = [
    (dict(q=None), -1), (dict(out=None), -1), (dict(cu_q=None), -1), (dict(k_pages=None), -1),
    (dict(v_pages=None), -1), (dict(block_table=None), -1), (dict(kv_lens=None), -1),
    (dict(table_stride=7), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(q=FAKE + 8), -1), (dict(k_pages=FAKE + 2), -1), (dict(q_token=513), -1),
    (dict(kp_head=68), -1), (dict(out_head=4), -1), (dict(vp_page=-2048), -1)]


@pytest.mark.parametrize("kw,rc", ATTEND_SIZES + ATTEND_POINTERS)
def test_attend_refuses(L, kw, rc):
    assert L.spec_cache_attend(C.byref(attend_args(**kw)), None, None) == rc


@pytest.mark.parametrize("kw,rc", ATTEND_SIZES)
def test_workspace_refuses(L, kw, rc):
    assert L.spec_cache_attend_workspace(C.byref(attend_args(**kw))) == rc


def test_null_args(L):
    assert L.spec_cache_step(None, None, None) == -1
    assert L.spec_cache_append(None, None, None) == -1
    assert L.spec_cache_attend(None, None, None) == -1
    assert L.spec_cache_attend_workspace(None) == -1


def test_no_tokens_is_no_launch(L):
    assert L.spec_cache_append(C.byref(append_args(num_tokens=0, k=None)), None,
                               None) == OK_HERE
    assert L.spec_cache_attend(C.byref(attend_args(num_tokens=0, q=None)), None,
                               None) == OK_HERE


def test_declared_cache_calls_are_exported(L):
    for name in sv.CACHE_ENTRY_POINTS:
        assert hasattr(L, name), name


def test_binding_refuses_host_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        sv.cache_step(i, i, torch.zeros((2, 3), dtype=torch.int32), i, i[:1], page_size=16,
                      num_tokens=4)
    pages = torch.zeros((2, 16, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        sv.cache_append(pages[0], pages[0], torch.zeros(16, dtype=torch.int64), pages, pages)
    with pytest.raises(ValueError, match="CUDA device"):
        sv.cache_attend(pages[0], pages, pages, torch.zeros((1, 1), dtype=torch.int32), i[:1], i)
