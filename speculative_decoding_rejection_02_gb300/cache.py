"""The paged key/value cache of a verification round: binding of
``include/spec_cache.h``.

``cache_step`` keeps block tables, free pages and slots between two rounds,
``cache_append`` writes new keys and values, ``cache_attend`` reads them. Each
is one call of the C ABI on torch tensors: argument checks here and in the
library raise before anything is enqueued, and outputs and workspace come from
torch's allocator on the stream that the call runs on (``stream``, or the
current one; with ``stream`` the caller orders it after the inputs' stream and
keeps the inputs until it is done, as for any work on another stream). Errors
in device data set bits of ``status`` (an int32 tensor of one element, OR-ed),
or without one are kept for ``cache_status``. There is no backward pass: a
tensor that requires a gradient is refused while gradients are enabled.

The calls on tensors are ``csrc/cache_binding.cpp``; the structures of the C
ABI are here for callers that come with addresses of their own.
"""
from __future__ import annotations

import ctypes as C
import importlib.machinery
import importlib.util
import os
from typing import NamedTuple

import torch

import speculative_decoding_rejection_02_gb300 as _sv

CACHE_NO_PAGES = 0x100
CACHE_BAD_LENGTHS = 0x200
CACHE_BAD_SLOT = 0x400
CACHE_BAD_PAGE = 0x800

_I, _L, _P = C.c_int, C.c_longlong, C.c_void_p


class StepArgs(C.Structure):
    _fields_ = [("B", _I), ("width", _I), ("table_stride", _L), ("page_size", _I),
                ("num_pages", _I), ("num_tokens", _I), ("held_lens", _P), ("new_lens", _P),
                ("cu_num_draft", _P), ("num_accepted", _P), ("block_table", _P),
                ("free_pages", _P), ("free_count", _P), ("lens", _P), ("cu_new", _P),
                ("positions", _P), ("slots", _P), ("free_count_out", _P)]


class AppendArgs(C.Structure):
    _fields_ = [("num_tokens", _L), ("kv_heads", _I), ("dim", _I), ("page_size", _I),
                ("num_pages", _L), ("dtype", _I), ("k", _P), ("k_token", _L), ("k_head", _L),
                ("v", _P), ("v_token", _L), ("v_head", _L), ("slots", _P), ("k_pages", _P),
                ("kp_page", _L), ("kp_token", _L), ("kp_head", _L), ("v_pages", _P),
                ("vp_page", _L), ("vp_token", _L), ("vp_head", _L)]


class AttendArgs(C.Structure):
    _fields_ = [("B", _I), ("num_tokens", _I), ("max_q", _I), ("heads", _I), ("kv_heads", _I),
                ("dim", _I), ("page_size", _I), ("width", _I), ("num_pages", _L), ("dtype", _I),
                ("q", _P), ("q_token", _L), ("q_head", _L), ("k_pages", _P), ("kp_page", _L),
                ("kp_token", _L), ("kp_head", _L), ("v_pages", _P), ("vp_page", _L),
                ("vp_token", _L), ("vp_head", _L), ("block_table", _P), ("table_stride", _L),
                ("kv_lens", _P), ("cu_q", _P), ("out", _P), ("out_token", _L), ("out_head", _L),
                ("lse", _P), ("scale", C.c_float), ("window", _I), ("sinks", _I),
                ("workspace", _P), ("workspace_bytes", C.c_size_t)]


class CacheStep(NamedTuple):
    """What ``cache_step`` computes, besides the block table and the stack. ``positions`` and
    ``slots`` share one storage, the other three another: clone what is to be saved alone."""
    lens: torch.Tensor        # int32 [B] tokens of each request
    cu_new: torch.Tensor      # int32 [B + 1] offsets of the new tokens
    positions: torch.Tensor   # int32 [num_tokens], -1 past the last new token
    slots: torch.Tensor       # int64 [num_tokens], -1 past the last new token
    free_count: torch.Tensor  # int32 [1]


class _Native:
    """cache_binding.cpp, built and bound to the library at the first call (the package imports
    without it)."""

    def __getattr__(self, name):
        lib = _sv.lib()
        path = _sv._build.BINDING_PATH
        if not os.path.exists(path):
            raise ImportError(f"the cache binding is not built ({path}); "
                              "run __graft_entry__.build()")
        if _sv._build.binding_torch() != torch.__version__:  # its C++ interface differs
            raise ImportError(f"the cache binding was built for torch "
                              f"{_sv._build.binding_torch()}, not {torch.__version__}; "
                              "run __graft_entry__.build()")
        loader = importlib.machinery.ExtensionFileLoader("_cache_binding", path)
        spec = importlib.util.spec_from_loader("_cache_binding", loader)
        module = importlib.util.module_from_spec(spec)
        loader.exec_module(module)
        module.bind(*(C.cast(getattr(lib, "spec_cache_" + n), C.c_void_p).value
                      for n in ("step", "append", "attend", "attend_workspace", "bounds", "score",
                                "select", "attend_selected", "weigh", "evict",
                                "evict_workspace")))
        for n in ("step", "append", "attend", "bounds", "score", "select", "attend_selected",
                  "weigh", "evict"):
            setattr(self, n, getattr(module, n))
        return object.__getattribute__(self, name)


_native = _Native()


def _on(stream, call, *args, **kw):
    """The whole call, its allocations too, on another stream."""
    with torch.cuda.stream(stream):
        return call(*args, **kw)


def cache_step(held_lens, new_lens, block_table, free_pages, free_count, *, page_size,
               num_tokens, cu_num_draft=None, num_accepted=None, status=None,
               stream=None) -> CacheStep:
    """Drop the rejected drafts of every request, return their pages, take
    pages for ``new_lens`` more tokens, and write the tokens' slots.

    ``held_lens`` [B] counts the tokens whose pages are held, the drafts just
    verified among them; ``cu_num_draft`` and ``num_accepted`` are the
    verifier's (without them nothing is dropped). ``block_table`` [B, width]
    and the stack ``free_pages`` are updated in place, ``free_count`` [1] is
    read. ``num_tokens`` is the most new tokens that there can be (a number of
    the host: the call never waits for the device). If the pages run short or a
    length cannot be, nothing changes and ``status`` gets CACHE_NO_PAGES or
    CACHE_BAD_LENGTHS. All integers are int32, slots int64.
    """
    if stream is not None:
        return _on(stream, cache_step, held_lens, new_lens, block_table, free_pages, free_count,
                   page_size=page_size, num_tokens=num_tokens, cu_num_draft=cu_num_draft,
                   num_accepted=num_accepted, status=status)
    r = _native.step(held_lens, new_lens, block_table, free_pages, free_count, page_size,
                     num_tokens, cu_num_draft, num_accepted, status)
    if type(r) is int:
        raise _sv.SpecVerifyError(r, "spec_cache_step")
    return tuple.__new__(CacheStep, r)  # (as CacheStep(*r), without its Python)


def cache_append(k, v, slots, k_pages, v_pages, *, status=None, stream=None) -> None:
    """Write the keys and values [T, kv_heads, dim] of T tokens to their
    ``slots`` (int64 [T], negative: none) of the pages
    [pages, page_size, kv_heads, dim]. Any strides whose last one is 1."""
    if stream is not None:
        return _on(stream, cache_append, k, v, slots, k_pages, v_pages, status=status)
    r = _native.append(k, v, slots, k_pages, v_pages, status)
    if r is not None:
        raise _sv.SpecVerifyError(r, "spec_cache_append")


def cache_attend(q, k_pages, v_pages, block_table, kv_lens, cu_q, *, max_q=None, scale=None,
                 window=0, sinks=0, out=None, return_lse=False, status=None, stream=None):
    """Attention of the new tokens ``q`` [T, heads, dim] over their requests'
    pages; returns ``out`` like q, and with ``return_lse`` also the fp32
    logarithm [T, heads] of each row's sum of exponentials.

    Rows cu_q[r] .. cu_q[r + 1] - 1 (int32 [B + 1]) are the last tokens of
    request r, which has kv_lens[r] tokens in all (int32 [B]); each sees the
    tokens up to itself, with ``window`` only the last ``window`` of them and
    the first ``sinks``. ``max_q`` is the most new tokens of one request that
    are expected (speed only; without it, as many as q has, which costs calls of a few tokens
    a request 1 to 3 %). Heads are shared by groups of heads / kv_heads.
    The page size is a power of two from 8, dim a multiple of 8 up to 128;
    addresses and strides are multiples of 16 bytes.
    """
    if stream is not None:
        return _on(stream, cache_attend, q, k_pages, v_pages, block_table, kv_lens, cu_q,
                   max_q=max_q, scale=scale, window=window, sinks=sinks, out=out,
                   return_lse=return_lse, status=status)
    r = _native.attend(q, k_pages, v_pages, block_table, kv_lens, cu_q, max_q, scale, window,
                       sinks, out, return_lse, status)
    if type(r) is int:
        raise _sv.SpecVerifyError(r, "spec_cache_attend")
    return r


def cache_status(device=None) -> int:
    """Wait for the device's work (the current device's) and return the status bits of the
    cache's calls that came without ``status``, which are cleared."""
    bits = C.c_uint(0)
    with torch.cuda.device(device):
        rc = _sv.lib().spec_cache_status(C.byref(bits))
    if rc not in (_sv.SPEC_OK, -6):
        raise _sv.SpecVerifyError(rc, "spec_cache_status")
    return int(bits.value)
