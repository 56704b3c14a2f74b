"""The paged key/value cache of a verification round: binding of
``include/spec_cache.h``.

``cache_step`` keeps block tables, free pages and slots between two rounds,
``cache_append`` writes new keys and values, ``cache_attend`` reads them. Each
is one call of the C ABI on torch tensors: argument checks here and in the
library raise before anything is enqueued, outputs and workspace come from
torch's allocator on the stream that the call runs on (``stream``, or the
current one), and errors in device data set bits of ``status`` (an int32
tensor of one element, OR-ed).
"""
from __future__ import annotations

import ctypes as C
import functools
import math
from typing import NamedTuple

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
    """What ``cache_step`` computes, besides the block table and the stack."""
    lens: "torch.Tensor"        # int32 [B] tokens of each request  # noqa: F821
    cu_new: "torch.Tensor"      # int32 [B + 1] offsets of the new tokens  # noqa: F821
    positions: "torch.Tensor"   # int32 [num_tokens], -1 past the last new token  # noqa: F821
    slots: "torch.Tensor"       # int64 [num_tokens], -1 past the last new token  # noqa: F821
    free_count: "torch.Tensor"  # int32 [1]  # noqa: F821


def _on_stream(call):
    """``stream=``: run the whole call, its allocations too, on that stream."""
    @functools.wraps(call)
    def run(*args, stream=None, **kw):
        if stream is None:
            return call(*args, **kw)
        import torch
        with torch.cuda.stream(stream):
            return call(*args, **kw)
    return run


def _on_device(first, tensors):
    """Tensors of one call are on one CUDA device, which is made the current one."""
    import torch
    dev = first.device
    if dev.type != "cuda":
        raise ValueError(f"the tensors must be on a CUDA device, not {dev}")
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors on {dev} and {t.device}")
    return dev, torch.cuda.current_stream(dev).cuda_stream


def _int32(t, what, shape):
    import torch
    if t.dtype != torch.int32 or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor of shape {shape}, not "
                         f"{t.dtype} {tuple(t.shape)}")


def _status(t):
    if t is None:
        return None
    if t.numel() != 1 or t.element_size() != 4:
        raise ValueError("status must be one 32-bit integer")
    return t.data_ptr()


def _table(t, B):
    import torch
    if t.dtype != torch.int32 or t.dim() != 2 or t.shape[0] != B or t.shape[1] < 1 or (
            t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError(f"block_table must be int32 [{B}, width] with adjacent columns, not "
                         f"{t.dtype} {tuple(t.shape)}")
    return t.stride(0) if B > 1 else max(t.stride(0), t.shape[1])


def _dtype(t):
    import torch
    if t.dtype == torch.bfloat16:
        return 1
    if t.dtype == torch.float16:
        return 2
    raise TypeError(f"the cache holds bfloat16 or float16, not {t.dtype}")


def _rows(t, what, heads, dim, dtype):
    """Strides of [tokens, heads, dim] with adjacent elements."""
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim or t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype} [tokens, {heads}, {dim}], not {t.dtype} "
                         f"{tuple(t.shape)}")
    s = t.stride()
    if s[2] != 1 and dim > 1:
        raise ValueError(f"the elements of a head of {what} must be adjacent")
    return s[0], s[1]


def _pages(t, what, like=None):
    """Strides of [pages, page_size, kv_heads, dim] with adjacent elements."""
    if t.dim() != 4 or (like is not None and (t.shape != like.shape or t.dtype != like.dtype)):
        raise ValueError(f"{what} must be [pages, page_size, kv_heads, dim], alike for keys and "
                         f"values, not {t.dtype} {tuple(t.shape)}")
    s = t.stride()
    if s[3] != 1 and t.shape[3] > 1:
        raise ValueError(f"the elements of a head of {what} must be adjacent")
    return s[0], s[1], s[2]


def _call(name, args, stream, status, device):
    import torch
    fn = getattr(_sv.lib(), name)
    if torch.cuda.current_device() == device.index:
        rc = fn(C.byref(args), stream, status)
    else:
        with torch.cuda.device(device):
            rc = fn(C.byref(args), stream, status)
    if rc != 0:
        raise _sv.SpecVerifyError(rc, name)


@_on_stream
def cache_step(held_lens, new_lens, block_table, free_pages, free_count, *, page_size,
               num_tokens, cu_num_draft=None, num_accepted=None, status=None) -> CacheStep:
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
    import torch
    B = held_lens.numel()
    dev, stream = _on_device(held_lens, (new_lens, block_table, free_pages, free_count,
                                         cu_num_draft, num_accepted, status))
    _int32(held_lens, "held_lens", (B,))
    _int32(new_lens, "new_lens", (B,))
    _int32(free_pages, "free_pages", (free_pages.numel(),))
    _int32(free_count, "free_count", (1,))
    if cu_num_draft is not None:
        _int32(cu_num_draft, "cu_num_draft", (B + 1,))
    if num_accepted is not None:
        _int32(num_accepted, "num_accepted", (B,))
    stride = _table(block_table, B)
    num_tokens = int(num_tokens)
    # one allocation for the 32-bit outputs
    ints = torch.empty(2 * B + 2 + num_tokens, dtype=torch.int32, device=dev)
    lens, cu_new, count, positions = ints.split((B, B + 1, 1, num_tokens))
    slots = torch.empty(num_tokens, dtype=torch.int64, device=dev)
    args = StepArgs(B, block_table.shape[1], stride, page_size, free_pages.numel(), num_tokens,
                    held_lens.data_ptr(), new_lens.data_ptr(), _sv._ptr(cu_num_draft),
                    _sv._ptr(num_accepted), block_table.data_ptr(), free_pages.data_ptr(),
                    free_count.data_ptr(), lens.data_ptr(), cu_new.data_ptr(),
                    positions.data_ptr(), slots.data_ptr(), count.data_ptr())
    _call("spec_cache_step", args, stream, _status(status), dev)
    return CacheStep(lens, cu_new, positions, slots, count)


@_on_stream
def cache_append(k, v, slots, k_pages, v_pages, *, status=None) -> None:
    """Write the keys and values [T, kv_heads, dim] of T tokens to their
    ``slots`` (int64 [T], negative: none) of the pages
    [pages, page_size, kv_heads, dim]. Any strides whose last one is 1."""
    import torch
    dev, stream = _on_device(k_pages, (k, v, slots, v_pages, status))
    n_pages, page_size, heads, dim = k_pages.shape
    T = k.shape[0]
    if slots.dtype != torch.int64 or tuple(slots.shape) != (T,) or not slots.is_contiguous():
        raise ValueError(f"slots must be contiguous int64 [{T}]")
    if v.shape[0] != T:
        raise ValueError(f"{T} keys and {v.shape[0]} values")
    args = AppendArgs(T, heads, dim, page_size, n_pages, _dtype(k_pages),
                      k.data_ptr(), *_rows(k, "k", heads, dim, k_pages.dtype),
                      v.data_ptr(), *_rows(v, "v", heads, dim, k_pages.dtype), slots.data_ptr(),
                      k_pages.data_ptr(), *_pages(k_pages, "k_pages"),
                      v_pages.data_ptr(), *_pages(v_pages, "v_pages", k_pages))
    _call("spec_cache_append", args, stream, _status(status), dev)


@_on_stream
def cache_attend(q, k_pages, v_pages, block_table, kv_lens, cu_q, *, max_q=None, scale=None,
                 window=0, sinks=0, out=None, return_lse=False, status=None):
    """Attention of the new tokens ``q`` [T, heads, dim] over their requests'
    pages; returns ``out`` like q, and with ``return_lse`` also the fp32
    logarithm [T, heads] of each row's sum of exponentials.

    Rows cu_q[r] .. cu_q[r + 1] - 1 (int32 [B + 1]) are the last tokens of
    request r, which has kv_lens[r] tokens in all (int32 [B]); each sees the
    tokens up to itself, with ``window`` only the last ``window`` of them and
    the first ``sinks``. ``max_q`` is the most new tokens of one request that
    are expected (speed only). Heads are shared by groups of heads / kv_heads.
    The page size is a power of two from 8, dim a multiple of 8 up to 128.
    """
    import torch
    dev, stream = _on_device(q, (k_pages, v_pages, block_table, kv_lens, cu_q, out, status))
    T, heads, dim = q.shape
    n_pages, page_size, kv_heads, pages_dim = k_pages.shape
    if pages_dim != dim or k_pages.dtype != q.dtype or kv_heads < 1 or heads % kv_heads:
        raise ValueError(f"q {q.dtype} {tuple(q.shape)} does not go with pages {k_pages.dtype} "
                         f"{tuple(k_pages.shape)}")
    B = kv_lens.numel()
    _int32(kv_lens, "kv_lens", (B,))
    _int32(cu_q, "cu_q", (B + 1,))
    stride = _table(block_table, B)
    if out is None:
        out = torch.empty((T, heads, dim), dtype=q.dtype, device=dev)
    elif out.shape[0] != T:
        raise ValueError(f"out has {out.shape[0]} tokens, q {T}")
    lse = torch.empty((T, heads), dtype=torch.float32, device=dev) if return_lse else None
    args = AttendArgs(B, T, T or 1 if max_q is None else max_q, heads, kv_heads, dim, page_size,
                      block_table.shape[1], n_pages, _dtype(q),
                      q.data_ptr(), *_rows(q, "q", heads, dim, q.dtype),
                      k_pages.data_ptr(), *_pages(k_pages, "k_pages"),
                      v_pages.data_ptr(), *_pages(v_pages, "v_pages", k_pages),
                      block_table.data_ptr(), stride, kv_lens.data_ptr(), cu_q.data_ptr(),
                      out.data_ptr(), *_rows(out, "out", heads, dim, q.dtype), _sv._ptr(lse),
                      1.0 / math.sqrt(dim) if scale is None else scale, window, sinks, None, 0)
    need = _sv.lib().spec_cache_attend_workspace(C.byref(args))
    if need < 0:
        raise _sv.SpecVerifyError(need, "spec_cache_attend")
    workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    args.workspace, args.workspace_bytes = _sv._ptr(workspace), need
    _call("spec_cache_attend", args, stream, _status(status), dev)
    return (out, lse) if return_lse else out
