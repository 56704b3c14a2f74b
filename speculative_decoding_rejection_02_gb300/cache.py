"""The paged key/value cache of a verification round: binding of
``include/spec_cache.h``.

``cache_step`` keeps block tables, free pages and slots between two rounds,
``cache_append`` writes new keys and values, ``cache_attend`` reads them. Each
is one call of the C ABI on torch tensors: argument checks here and in the
library raise before anything is enqueued, outputs and workspace come from
torch's allocator on the stream that the call runs on (``stream``, or the
current one), and errors in device data set bits of ``status`` (an int32
tensor of one element, OR-ed).

A call costs the host about as much as its launch, so each check is one
expression over plain attributes; what is wrong is worked out afterwards.
"""
from __future__ import annotations

import ctypes as C
from typing import NamedTuple

import torch

import speculative_decoding_rejection_02_gb300 as _sv

CACHE_NO_PAGES = 0x100
CACHE_BAD_LENGTHS = 0x200
CACHE_BAD_SLOT = 0x400
CACHE_BAD_PAGE = 0x800

_I, _L, _P = C.c_int, C.c_longlong, C.c_void_p
_i32, _i64 = torch.int32, torch.int64
_DTYPES = {torch.bfloat16: 1, torch.float16: 2}
_empty = torch.empty
_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


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
    lens: torch.Tensor        # int32 [B] tokens of each request
    cu_new: torch.Tensor      # int32 [B + 1] offsets of the new tokens
    positions: torch.Tensor   # int32 [num_tokens], -1 past the last new token
    slots: torch.Tensor       # int64 [num_tokens], -1 past the last new token
    free_count: torch.Tensor  # int32 [1]


def _run(fn, name, args, dev, status):
    """One call of the C ABI on the tensors' device and its current stream."""
    if status is not None:
        if status.numel() != 1 or status.element_size() != 4 or status.get_device() != dev:
            raise ValueError("status must be one 32-bit integer beside the other tensors")
        status = status.data_ptr()
    if _device() == dev:
        rc = fn(args, _raw_stream(dev), status)
    else:
        with torch.cuda.device(dev):
            rc = fn(args, _raw_stream(dev), status)
    if rc != 0:
        raise _sv.SpecVerifyError(rc, name)


def _need(ok, what, *tensors):
    if not ok:
        raise ValueError(what + ", not " + ", ".join(
            "none" if t is None else f"{t.dtype} {tuple(t.shape)} on {t.device}"
            for t in tensors))


def _one_device(dev, *tensors):
    if dev < 0:
        raise ValueError("the tensors must be on a CUDA device")
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors on cuda:{dev} and {t.device}")


def _table(t, B):
    """Stride of a block table's rows."""
    shape, stride = t.shape, t.stride()
    if t.dtype is not _i32 or len(shape) != 2 or shape[0] != B or shape[1] < 1 or (
            stride[1] != 1 and shape[1] > 1):
        _need(False, f"block_table must be int32 [{B}, width] with adjacent columns", t)
    return stride[0] if B > 1 else max(stride[0], shape[1])


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
    dev = held_lens.get_device()
    _one_device(dev, new_lens, block_table, free_pages, free_count, cu_num_draft, num_accepted)
    B = held_lens.numel()
    if not (held_lens.dtype is _i32 and new_lens.dtype is _i32 and new_lens.numel() == B
            and held_lens.is_contiguous() and new_lens.is_contiguous()):
        _need(False, "held_lens and new_lens must be contiguous int32 [B]", held_lens, new_lens)
    if not (free_pages.dtype is _i32 and free_pages.is_contiguous()
            and free_count.dtype is _i32 and free_count.numel() == 1):
        _need(False, "free_pages and free_count must be contiguous int32 [pages] and [1]",
              free_pages, free_count)
    drafts = accepted = None
    if cu_num_draft is not None or num_accepted is not None:
        if not (cu_num_draft is not None and num_accepted is not None
                and cu_num_draft.dtype is _i32 and cu_num_draft.numel() == B + 1
                and cu_num_draft.is_contiguous() and num_accepted.dtype is _i32
                and num_accepted.numel() == B and num_accepted.is_contiguous()):
            _need(False, "cu_num_draft and num_accepted must be contiguous int32 [B + 1] and [B]",
                  cu_num_draft, num_accepted)
        drafts, accepted = cu_num_draft.data_ptr(), num_accepted.data_ptr()
    stride = _table(block_table, B)
    place = held_lens.device
    # one allocation for the 32-bit outputs
    ints = _empty(2 * B + 2 + num_tokens, dtype=_i32, device=place)
    at = ints.data_ptr()
    lens, cu_new, count, positions = ints.split_with_sizes((B, B + 1, 1, num_tokens))
    slots = _empty(num_tokens, dtype=_i64, device=place)
    args = StepArgs(B, block_table.shape[1], stride, page_size, free_pages.numel(), num_tokens,
                    held_lens.data_ptr(), new_lens.data_ptr(), drafts, accepted,
                    block_table.data_ptr(), free_pages.data_ptr(), free_count.data_ptr(), at,
                    at + 4 * B, at + 4 * (2 * B + 2), slots.data_ptr(), at + 4 * (2 * B + 1))
    _run(_lib.spec_cache_step, "spec_cache_step", args, dev, status)
    return CacheStep(lens, cu_new, positions, slots, count)


def cache_append(k, v, slots, k_pages, v_pages, *, status=None, stream=None) -> None:
    """Write the keys and values [T, kv_heads, dim] of T tokens to their
    ``slots`` (int64 [T], negative: none) of the pages
    [pages, page_size, kv_heads, dim]. Any strides whose last one is 1."""
    if stream is not None:
        return _on(stream, cache_append, k, v, slots, k_pages, v_pages, status=status)
    dev = k_pages.get_device()
    _one_device(dev, k, v, slots, v_pages)
    shape, dtype = k_pages.shape, k_pages.dtype
    if dtype not in _DTYPES:
        raise TypeError(f"the cache holds bfloat16 or float16, not {dtype}")
    sk, sv, pk, pv = k.stride(), v.stride(), k_pages.stride(), v_pages.stride()
    if not (len(shape) == 4 and v_pages.shape == shape and v_pages.dtype is dtype
            and ((pk[3] == 1 and pv[3] == 1) or shape[3] == 1)):
        _need(False, "k_pages and v_pages must be alike, [pages, page_size, kv_heads, dim] with "
              "adjacent elements", k_pages, v_pages)
    if not (len(sk) == 3 and k.shape[1:] == shape[2:] and v.shape == k.shape
            and k.dtype is dtype and v.dtype is dtype
            and ((sk[2] == 1 and sv[2] == 1) or shape[3] == 1)):
        _need(False, f"k and v must be {dtype} [tokens, {shape[2]}, {shape[3]}] with adjacent "
              "elements", k, v)
    T = k.shape[0]
    if not (slots.dtype is _i64 and slots.numel() == T and slots.is_contiguous()):
        _need(False, f"slots must be contiguous int64 [{T}]", slots)
    args = AppendArgs(T, shape[2], shape[3], shape[1], shape[0], _DTYPES[dtype], k.data_ptr(),
                      sk[0], sk[1], v.data_ptr(), sv[0], sv[1], slots.data_ptr(),
                      k_pages.data_ptr(), pk[0], pk[1], pk[2], v_pages.data_ptr(), pv[0], pv[1],
                      pv[2])
    _run(_lib.spec_cache_append, "spec_cache_append", args, dev, status)


def cache_attend(q, k_pages, v_pages, block_table, kv_lens, cu_q, *, max_q=None, scale=None,
                 window=0, sinks=0, out=None, return_lse=False, status=None, stream=None):
    """Attention of the new tokens ``q`` [T, heads, dim] over their requests'
    pages; returns ``out`` like q, and with ``return_lse`` also the fp32
    logarithm [T, heads] of each row's sum of exponentials.

    Rows cu_q[r] .. cu_q[r + 1] - 1 (int32 [B + 1]) are the last tokens of
    request r, which has kv_lens[r] tokens in all (int32 [B]); each sees the
    tokens up to itself, with ``window`` only the last ``window`` of them and
    the first ``sinks``. ``max_q`` is the most new tokens of one request that
    are expected (speed only). Heads are shared by groups of heads / kv_heads.
    The page size is a power of two from 8, dim a multiple of 8 up to 128;
    addresses and strides are multiples of 16 bytes.
    """
    if stream is not None:
        return _on(stream, cache_attend, q, k_pages, v_pages, block_table, kv_lens, cu_q,
                   max_q=max_q, scale=scale, window=window, sinks=sinks, out=out,
                   return_lse=return_lse, status=status)
    dev = q.get_device()
    _one_device(dev, k_pages, v_pages, block_table, kv_lens, cu_q, out)
    shape, dtype = k_pages.shape, q.dtype
    if dtype not in _DTYPES:
        raise TypeError(f"the cache holds bfloat16 or float16, not {dtype}")
    sq, pk, pv = q.stride(), k_pages.stride(), v_pages.stride()
    if not (len(shape) == 4 and v_pages.shape == shape and v_pages.dtype is dtype
            and k_pages.dtype is dtype and ((pk[3] == 1 and pv[3] == 1) or shape[3] == 1)):
        _need(False, f"k_pages and v_pages must be alike, {dtype} [pages, page_size, kv_heads, "
              "dim] with adjacent elements", k_pages, v_pages)
    n_pages, page_size, kv_heads, dim = shape
    if not (len(sq) == 3 and q.shape[2] == dim and kv_heads > 0 and q.shape[1] % kv_heads == 0
            and (sq[2] == 1 or dim == 1)):
        _need(False, f"q must be [tokens, heads, {dim}] with adjacent elements and heads a "
              f"multiple of {kv_heads}", q)
    T, heads, _ = q.shape
    B = kv_lens.numel()
    if not (kv_lens.dtype is _i32 and cu_q.dtype is _i32 and cu_q.numel() == B + 1
            and kv_lens.is_contiguous() and cu_q.is_contiguous()):
        _need(False, "kv_lens and cu_q must be contiguous int32 [B] and [B + 1]", kv_lens, cu_q)
    stride = _table(block_table, B)
    if out is None:
        out = _empty((T, heads, dim), dtype=dtype, device=q.device)
        so = (heads * dim, dim)
    else:
        so = out.stride()
        if not (out.shape == q.shape and out.dtype is dtype and (so[2] == 1 or dim == 1)):
            _need(False, f"out must be {dtype} {tuple(q.shape)} with adjacent elements", out)
    lse = _empty((T, heads), dtype=torch.float32, device=q.device) if return_lse else None
    args = AttendArgs(B, T, max_q or T or 1, heads, kv_heads, dim, page_size,
                      block_table.shape[1], n_pages, _DTYPES[dtype], q.data_ptr(), sq[0], sq[1],
                      k_pages.data_ptr(), pk[0], pk[1], pk[2], v_pages.data_ptr(), pv[0], pv[1],
                      pv[2], block_table.data_ptr(), stride, kv_lens.data_ptr(), cu_q.data_ptr(),
                      out.data_ptr(), so[0], so[1], lse.data_ptr() if return_lse else None,
                      dim ** -0.5 if scale is None else scale, window, sinks, None, 0)
    need = _lib.spec_cache_attend_workspace(args)
    if need < 0:
        raise _sv.SpecVerifyError(need, "spec_cache_attend")
    workspace = _empty(need, dtype=torch.uint8, device=q.device)
    args.workspace, args.workspace_bytes = workspace.data_ptr(), need
    _run(_lib.spec_cache_attend, "spec_cache_attend", args, dev, status)
    return (out, lse) if return_lse else out


class _Lib:
    """The library, loaded at the first call (the package imports without it)."""

    def __getattr__(self, name):
        lib = _sv.lib()
        for n, kind in (("spec_cache_step", StepArgs), ("spec_cache_append", AppendArgs),
                        ("spec_cache_attend", AttendArgs)):
            # a prototype that takes the structure itself: no pointer object per call
            fn = C.CFUNCTYPE(_I, C.POINTER(kind), _P, _P)((n, lib))
            setattr(self, n, fn)
        self.spec_cache_attend_workspace = C.CFUNCTYPE(_L, C.POINTER(AttendArgs))(
            ("spec_cache_attend_workspace", lib))
        return object.__getattribute__(self, name)


_lib = _Lib()
