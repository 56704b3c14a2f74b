"""Sparse attention and eviction on the paged cache: binding of ``include/spec_sparse.h``.

For contexts that are long, two ways of touching less of the cache than ``cache_attend`` does.

Reading few pages: ``cache_bounds`` finds the extremes of each page's keys after an append,
``cache_score`` bounds each page's scores by them, ``cache_select`` picks the pages for every
new token and kv head, ``cache_attend_selected`` attends to them alone.

Holding few tokens: ``cache_weigh`` adds up the softmax weights that each cached token gets, and
``cache_evict`` keeps the heaviest tokens of every kv head, closes the gaps and gives pages back.

Conventions are those of ``cache.py``: argument checks raise before anything is enqueued, outputs
and workspace come from torch's allocator on the stream that the call runs on (``stream``, or the
current one), errors in device data set bits of ``status`` or are kept for ``cache_status``, and
tensors that require a gradient are refused while gradients are enabled. Page sizes are powers of
two from 8, dim is a multiple of 8 up to 128; addresses and strides of 16-bit tensors are multiples
of 16 bytes; what a call writes may not overlap its other arguments.

``cache_score``, ``cache_select`` and ``cache_evict`` take longer in tables that are wider than
their requests need (scores of a round over up to 30000 tokens: 36 us with 1876 columns, 57 with
8192; its selection 13 and 52): pass a view of the first columns, ``block_table[:, :n]``, as far
as the longest request may reach.
"""
from __future__ import annotations

import ctypes as C
from typing import NamedTuple

import torch

import speculative_decoding_rejection_02_gb300 as _sv

from .cache import _I, _L, _P, _native, _on

CACHE_BAD_SELECTION = 0x1000
CACHE_TEST_WAIT_TIMEOUT = 0x1  # WeighArgs.flags, test only: a wait runs out

_F = C.c_float


class BoundsArgs(C.Structure):
    _fields_ = [("B", _I), ("width", _I), ("table_stride", _L), ("max_q", _I), ("kv_heads", _I),
                ("dim", _I), ("page_size", _I), ("num_pages", _L), ("dtype", _I),
                ("k_pages", _P), ("kp_page", _L), ("kp_token", _L), ("kp_head", _L),
                ("block_table", _P), ("kv_lens", _P), ("cu_q", _P), ("bounds", _P),
                ("b_page", _L), ("b_head", _L), ("b_side", _L)]


class ScoreArgs(C.Structure):
    _fields_ = [("B", _I), ("width", _I), ("table_stride", _L), ("num_tokens", _I),
                ("max_q", _I), ("heads", _I), ("kv_heads", _I), ("dim", _I), ("page_size", _I),
                ("num_pages", _L), ("dtype", _I), ("q", _P), ("q_token", _L), ("q_head", _L),
                ("bounds", _P), ("b_page", _L), ("b_head", _L), ("b_side", _L),
                ("block_table", _P), ("kv_lens", _P), ("cu_q", _P), ("scores", _P),
                ("s_token", _L), ("s_head", _L)]


class SelectArgs(C.Structure):
    _fields_ = [("B", _I), ("num_tokens", _I), ("kv_heads", _I), ("page_size", _I),
                ("width", _I), ("scores", _P), ("s_token", _L), ("s_head", _L),
                ("kv_lens", _P), ("cu_q", _P), ("count", _I), ("first", _I), ("recent", _I),
                ("selected", _P)]


class AttendSelectedArgs(C.Structure):
    _fields_ = [("B", _I), ("width", _I), ("table_stride", _L), ("num_tokens", _I),
                ("heads", _I), ("kv_heads", _I), ("dim", _I), ("page_size", _I),
                ("num_pages", _L), ("dtype", _I), ("q", _P), ("q_token", _L), ("q_head", _L),
                ("k_pages", _P), ("kp_page", _L), ("kp_token", _L), ("kp_head", _L),
                ("v_pages", _P), ("vp_page", _L), ("vp_token", _L), ("vp_head", _L),
                ("block_table", _P), ("kv_lens", _P), ("cu_q", _P), ("count", _I),
                ("selected", _P), ("out", _P), ("out_token", _L), ("out_head", _L),
                ("lse", _P), ("scale", _F)]


class WeighArgs(C.Structure):
    _fields_ = [("B", _I), ("width", _I), ("table_stride", _L), ("num_tokens", _I),
                ("max_q", _I), ("heads", _I), ("kv_heads", _I), ("dim", _I), ("page_size", _I),
                ("num_pages", _L), ("dtype", _I), ("q", _P), ("q_token", _L), ("q_head", _L),
                ("k_pages", _P), ("kp_page", _L), ("kp_token", _L), ("kp_head", _L),
                ("block_table", _P), ("kv_lens", _P), ("cu_q", _P), ("lse", _P),
                ("weights", _P), ("w_page", _L), ("w_head", _L), ("scale", _F), ("decay", _F),
                ("flags", C.c_uint)]


class EvictArgs(C.Structure):
    _fields_ = [("B", _I), ("width", _I), ("table_stride", _L), ("kv_heads", _I), ("dim", _I),
                ("page_size", _I), ("num_pages", _I), ("dtype", _I), ("k_pages", _P),
                ("kp_page", _L), ("kp_token", _L), ("kp_head", _L), ("v_pages", _P),
                ("vp_page", _L), ("vp_token", _L), ("vp_head", _L), ("weights", _P),
                ("w_page", _L), ("w_head", _L), ("block_table", _P), ("lens", _P),
                ("budget", _P), ("first", _I), ("recent", _I), ("free_pages", _P),
                ("free_count", _P), ("lens_out", _P), ("free_count_out", _P),
                ("workspace", _P), ("workspace_bytes", C.c_size_t)]


class CacheEvict(NamedTuple):
    """What ``cache_evict`` computes, besides what it changes in place. Both share a storage."""
    lens: torch.Tensor        # int32 [B] tokens of each request
    free_count: torch.Tensor  # int32 [1]


def cache_bounds(k_pages, block_table, kv_lens, bounds, *, cu_q=None, max_q=None, status=None,
                 stream=None) -> None:
    """Write the least and the largest key of every channel of each page to ``bounds``
    [pages, kv_heads, 2, dim] (the pages' type; 0: least, 1: largest).

    With ``cu_q`` (as in ``cache_attend``) of the pages that hold a request's new tokens, the ones
    that an append has changed; without it of all pages of every request. Only the tokens before
    ``kv_lens`` count, whatever the bounds were before, so dropped drafts leave nothing behind.
    ``max_q`` is the most new tokens of one request that are expected (speed only).
    """
    if stream is not None:
        return _on(stream, cache_bounds, k_pages, block_table, kv_lens, bounds, cu_q=cu_q,
                   max_q=max_q, status=status)
    r = _native.bounds(k_pages, block_table, kv_lens, cu_q, bounds, max_q, status)
    if r is not None:
        raise _sv.SpecVerifyError(r, "spec_cache_bounds")


def cache_score(q, bounds, block_table, kv_lens, cu_q, *, page_size, max_q=None, out=None,
                status=None, stream=None):
    """Upper bounds of the pages' scores: float32 [T, kv_heads, width], for each new token, kv head
    and column of the block table the sum over the head's query heads and the channels of
    max(q lo, q hi); -inf for columns that the token does not see. ``max_q`` as in
    ``cache_attend``."""
    if stream is not None:
        return _on(stream, cache_score, q, bounds, block_table, kv_lens, cu_q,
                   page_size=page_size, max_q=max_q, out=out, status=status)
    r = _native.score(q, bounds, block_table, kv_lens, cu_q, page_size, max_q, out, status)
    if type(r) is int:
        raise _sv.SpecVerifyError(r, "spec_cache_score")
    return r


def cache_select(scores, kv_lens, cu_q, *, page_size, count, first=0, recent=1, out=None,
                 status=None, stream=None):
    """The columns that each new token attends to: int32 [T, kv_heads, count], ascending, -1 past
    the last. Of the visible columns the first ``first``, the last ``recent`` (up to the token's
    own) and those of the highest ``scores`` [T, kv_heads, width] (NaN counts as +inf; of equal
    ones the lowest columns). The scores may be ``cache_score``'s or any others."""
    if stream is not None:
        return _on(stream, cache_select, scores, kv_lens, cu_q, page_size=page_size, count=count,
                   first=first, recent=recent, out=out, status=status)
    r = _native.select(scores, kv_lens, cu_q, page_size, count, first, recent, out, status)
    if type(r) is int:
        raise _sv.SpecVerifyError(r, "spec_cache_select")
    return r


def cache_attend_selected(q, k_pages, v_pages, block_table, kv_lens, cu_q, selected, *, scale=None,
                          out=None, return_lse=False, status=None, stream=None):
    """``cache_attend`` over the pages in ``selected`` (int32 [T, kv_heads, count]) alone: token t
    and the query heads of kv head h see the tokens up to t's own in columns ``selected[t, h]``,
    which ascend and end with -1, as ``cache_select`` leaves them. A value that is not finite may
    reach rows of its request and kv head that do not see it (as 0 times infinity); a key that is
    not finite reaches only those that do."""
    if stream is not None:
        return _on(stream, cache_attend_selected, q, k_pages, v_pages, block_table, kv_lens, cu_q,
                   selected, scale=scale, out=out, return_lse=return_lse, status=status)
    r = _native.attend_selected(q, k_pages, v_pages, block_table, kv_lens, cu_q, selected, scale,
                                out, return_lse, status)
    if type(r) is int:
        raise _sv.SpecVerifyError(r, "spec_cache_attend_selected")
    return r


def cache_weigh(q, k_pages, block_table, kv_lens, cu_q, lse, weights, *, max_q=None, scale=None,
                decay=1.0, status=None, stream=None) -> None:
    """Add to ``weights`` (float32 [pages, kv_heads, page_size]) what the new tokens' queries gave
    every cached token: the sum over the new tokens that see it and the query heads of its kv head
    of e^(scale q . k - lse), with ``lse`` from ``cache_attend`` (without a window). Older sums are
    multiplied by ``decay`` first; the new tokens' own slots start from 0, whatever they held.
    Requests without new tokens stay as they are. ``max_q`` as in ``cache_attend``.

    Drafts give their weight like other tokens, and it stays when they are rejected. To leave it
    out, call after the verification with the rejected rows' lse at -inf; for a round of the last
    token and its drafts, with the row's number in its request::

        rejected = row - cu_q[request] > num_accepted[request]
        cache_weigh(..., lse.masked_fill(rejected[:, None], -math.inf), weights)
    """
    if stream is not None:
        return _on(stream, cache_weigh, q, k_pages, block_table, kv_lens, cu_q, lse, weights,
                   max_q=max_q, scale=scale, decay=decay, status=status)
    r = _native.weigh(q, k_pages, block_table, kv_lens, cu_q, lse, weights, max_q, scale, decay,
                      status)
    if r is not None:
        raise _sv.SpecVerifyError(r, "spec_cache_weigh")


def cache_evict(k_pages, v_pages, weights, block_table, lens, budget, free_pages, free_count, *,
                first=0, recent=0, status=None, stream=None) -> CacheEvict:
    """Bring every request back to ``budget`` (int32 [B]) tokens: each kv head keeps the first
    ``first`` and the last ``recent`` tokens and the heaviest of the others (by ``weights``; of
    equal ones the first), never fewer than first + recent. The kept tokens' keys, values and
    weights move down in their order, the pages past them go on the stack ``free_pages``
    (``free_count`` [1] is read). Requests within their budget stay as they are, and so do table
    entries and slots past the kept tokens.

    A kept token's place is no longer its position: the caller counts positions for rotary
    embeddings itself, and calls ``cache_bounds`` anew (without ``cu_q``) where it uses them.
    Between a round's append and the ``cache_step`` that drops its rejected drafts, ``recent`` must
    be at least the most new tokens of a request in the round: the step drops the last slots,
    whatever stands there, and drafts weigh little, so they would go first. Or drop first, by a
    ``cache_step`` whose ``new_lens`` are 0.

    If a length or budget cannot be, nothing changes and ``status`` gets CACHE_BAD_LENGTHS.
    """
    if stream is not None:
        return _on(stream, cache_evict, k_pages, v_pages, weights, block_table, lens, budget,
                   free_pages, free_count, first=first, recent=recent, status=status)
    r = _native.evict(k_pages, v_pages, weights, block_table, lens, budget, free_pages, free_count,
                      first, recent, status)
    if type(r) is int:
        raise _sv.SpecVerifyError(r, "spec_cache_evict")
    return tuple.__new__(CacheEvict, r)
