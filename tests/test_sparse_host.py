"""Argument checks of the sparse-attention and eviction calls, which need no device: the C ABI's
(before anything is enqueued) and the binding's."""
import ctypes as C
import math

import pytest
import torch

import speculative_decoding_rejection_02_gb300 as sv
from speculative_decoding_rejection_02_gb300 import _build

OK_HERE = 0 if torch.cuda.is_available() else -2  # no sm_103 here: refused after the checks
A = 1 << 32  # addresses that nothing dereferences, far apart


@pytest.fixture(scope="module")
def L():
    _build.build()
    return sv.lib()


TABLE = dict(B=2, width=8, table_stride=8, block_table=8 * A, kv_lens=9 * A, cu_q=10 * A)
SIZES = dict(kv_heads=2, dim=64, page_size=16, num_pages=8, dtype=1)
KEYS = dict(k_pages=A, kp_page=2048, kp_token=128, kp_head=64)
VALUES = dict(v_pages=2 * A, vp_page=2048, vp_token=128, vp_head=64)
QUERY = dict(num_tokens=4, heads=8, q=3 * A, q_token=512, q_head=64)
BOUNDS = dict(bounds=4 * A, b_page=256, b_head=128, b_side=64)
CALLS = {
    "bounds": (sv.BoundsArgs, dict(TABLE, **SIZES, **KEYS, **BOUNDS, max_q=2)),
    "score": (sv.ScoreArgs, dict(TABLE, **SIZES, **QUERY, **BOUNDS, max_q=2, scores=5 * A,
                                 s_token=16, s_head=8)),
    "select": (sv.SelectArgs, dict(B=2, num_tokens=4, kv_heads=2, page_size=16, width=8,
                                   scores=5 * A, s_token=16, s_head=8, kv_lens=9 * A,
                                   cu_q=10 * A, count=4, first=1, recent=2, selected=6 * A)),
    "attend_selected": (sv.AttendSelectedArgs, dict(
        TABLE, **SIZES, **QUERY, **KEYS, **VALUES, count=4, selected=6 * A, out=7 * A,
        out_token=512, out_head=64, lse=11 * A, scale=0.125)),
    "weigh": (sv.WeighArgs, dict(TABLE, **SIZES, **QUERY, **KEYS, max_q=2, lse=11 * A,
                                 weights=12 * A, w_page=32, w_head=16, scale=0.125, decay=1.0)),
    "evict": (sv.EvictArgs, dict(
        B=2, width=8, table_stride=8, block_table=8 * A, **SIZES, **KEYS, **VALUES,
        weights=12 * A, w_page=32, w_head=16, lens=9 * A, budget=13 * A, first=1, recent=2,
        free_pages=14 * A, free_count=15 * A, lens_out=16 * A, free_count_out=17 * A,
        workspace=18 * A, workspace_bytes=1 << 20)),
}


def call(L, name, **kw):
    kind, base = CALLS[name]
    assert set(kw) <= {f for f, _ in kind._fields_}, kw
    return getattr(L, "spec_cache_" + name)(C.byref(kind(**dict(base, **kw))), None, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on addresses that are not")
@pytest.mark.parametrize("name", CALLS)
def test_complete_arguments_pass_the_checks(L, name):
    assert call(L, name) == -2


SIZE_CASES = [(dict(B=-1), -1), (dict(width=0), -1), (dict(kv_heads=0), -1),
              (dict(page_size=0), -1), (dict(page_size=4), -2), (dict(page_size=24), -2),
              (dict(page_size=1 << 21), -2)]
POOL_CASES = [(dict(dim=0), -1), (dict(dim=60), -2), (dict(dim=136), -2), (dict(dtype=0), -1),
              (dict(dtype=3), -1), (dict(num_pages=0), -1), (dict(table_stride=7), -1),
              (dict(block_table=None), -1)]
QUERY_CASES = [(dict(heads=7), -1), (dict(heads=0), -1), (dict(heads=258), -2),
               (dict(num_tokens=-1), -1), (dict(q=None), -1), (dict(q=3 * A + 8), -1),
               (dict(q_token=515), -1), (dict(q_head=-64), -1), (dict(kv_lens=None), -1),
               (dict(cu_q=None), -1)]
KEY_CASES = [(dict(k_pages=None), -1), (dict(k_pages=A + 2), -1), (dict(kp_token=60), -1),
             (dict(kp_page=0), -1)]
REFUSED = {
    "bounds": SIZE_CASES + POOL_CASES + KEY_CASES + [
        (dict(max_q=0), -1), (dict(bounds=None), -1), (dict(bounds=4 * A + 8), -1),
        (dict(b_side=4), -1), (dict(kv_lens=None), -1), (dict(bounds=A), -1),
        (dict(bounds=9 * A), -1)],
    "score": SIZE_CASES + POOL_CASES + QUERY_CASES + [
        (dict(max_q=0), -1), (dict(bounds=None), -1), (dict(scores=None), -1),
        (dict(scores=5 * A + 2), -1), (dict(s_token=0), -1), (dict(scores=3 * A), -1),
        (dict(scores=10 * A), -1)],
    "select": SIZE_CASES + [
        (dict(count=0), -1), (dict(first=-1), -1), (dict(recent=-1), -1),
        (dict(first=3, recent=2), -1), (dict(first=2 ** 31 - 1, recent=2 ** 31 - 1), -1),
        (dict(scores=None), -1), (dict(selected=None), -1), (dict(selected=5 * A), -1),
        (dict(selected=9 * A), -1), (dict(kv_lens=None), -1), (dict(cu_q=None), -1)],
    "attend_selected": SIZE_CASES + POOL_CASES + QUERY_CASES + KEY_CASES + [
        (dict(v_pages=None), -1), (dict(vp_head=4), -1), (dict(out=None), -1),
        (dict(out=7 * A + 8), -1), (dict(out_token=4), -1), (dict(selected=None), -1),
        (dict(count=0), -1), (dict(scale=float("nan")), -1), (dict(scale=3e38), -1),
        (dict(out=3 * A), -1), (dict(lse=6 * A), -1), (dict(out=2 * A), -1)],
    "weigh": SIZE_CASES + POOL_CASES + QUERY_CASES + KEY_CASES + [
        (dict(max_q=0), -1), (dict(lse=None), -1), (dict(lse=11 * A + 2), -1),
        (dict(weights=None), -1), (dict(weights=12 * A + 2), -1), (dict(w_page=0), -1),
        (dict(scale=float("inf")), -1), (dict(decay=float("nan")), -1), (dict(weights=A), -1),
        (dict(weights=11 * A), -1)],
    "evict": SIZE_CASES + POOL_CASES + KEY_CASES + [
        (dict(v_pages=None), -1), (dict(v_pages=A), -1), (dict(weights=None), -1),
        (dict(weights=A), -1), (dict(lens=None), -1), (dict(budget=None), -1),
        (dict(first=-1), -1), (dict(recent=-1), -1), (dict(free_pages=None), -1),
        (dict(free_count=None), -1), (dict(lens_out=None), -1), (dict(free_count_out=None), -1),
        (dict(lens_out=9 * A), -1), (dict(free_count_out=15 * A), -1),
        (dict(free_pages=8 * A), -1)],
}


@pytest.mark.parametrize("name,kw,rc", [(n, kw, rc) for n, cases in REFUSED.items()
                                        for kw, rc in cases])
def test_refuses(L, name, kw, rc):
    assert call(L, name, **kw) == rc


@pytest.mark.parametrize("name", CALLS)
def test_null_structures(L, name):
    assert getattr(L, "spec_cache_" + name)(None, None, None) == -1
    assert L.spec_cache_evict_workspace(None) == -1


def test_evict_workspace_by_the_sizes_alone(L):
    kind, base = CALLS["evict"]
    need = L.spec_cache_evict_workspace(C.byref(kind(**dict(base, k_pages=None, weights=None))))
    assert need == 256 + 2 * 8 * 2 * 16 * 4  # by columns
    few = L.spec_cache_evict_workspace(C.byref(kind(**dict(base, num_pages=3))))
    assert few == 256 + 3 * 2 * 16 * 4  # by pages of the pool
    assert L.spec_cache_evict_workspace(C.byref(kind(**dict(base, dim=4)))) == -2


@pytest.mark.skipif(not torch.cuda.is_available(), reason="found after the device")
def test_evict_workspace_too_small(L):
    assert call(L, "evict", workspace_bytes=100) == -5
    assert call(L, "evict", workspace=18 * A + 64) == -1


def test_keys_and_values_between_one_another(L):
    """Views of one pool [pages, 2, page, heads, dim]."""
    for name in ("attend_selected", "evict"):
        rc = call(L, name, kp_page=4096, vp_page=4096, v_pages=A + 4096, num_pages=0)
        assert rc == -1  # (the size, to stop before the device)
        if not torch.cuda.is_available():
            assert call(L, name, kp_page=4096, vp_page=4096, v_pages=A + 4096) == -2


def test_nothing_to_do_is_no_launch(L):
    assert call(L, "bounds", B=0, k_pages=None, bounds=None) == OK_HERE
    assert call(L, "score", num_tokens=0, q=None, scores=None) == OK_HERE
    assert call(L, "select", num_tokens=0, scores=None, selected=None) == OK_HERE
    assert call(L, "attend_selected", num_tokens=0, q=None, out=None) == OK_HERE
    assert call(L, "weigh", num_tokens=0, q=None, weights=None) == OK_HERE
    assert call(L, "weigh", B=0, kv_lens=None, weights=None) == OK_HERE


def test_declared_calls_are_exported(L):
    for name in sv.SPARSE_ENTRY_POINTS:
        assert hasattr(L, name), name
    assert {"spec_cache_" + n for n in CALLS} < set(sv.SPARSE_ENTRY_POINTS)


# ---------------------------------------------------------------- the binding

def tensors(device="cpu"):
    bf, i32 = dict(dtype=torch.bfloat16, device=device), dict(dtype=torch.int32, device=device)
    return dict(k_pages=torch.zeros((4, 16, 2, 64), **bf), v_pages=torch.zeros((4, 16, 2, 64), **bf),
                block_table=torch.zeros((1, 4), **i32), kv_lens=torch.full((1,), 20, **i32),
                cu_q=torch.tensor([0, 3], **i32), q=torch.zeros((3, 4, 64), **bf),
                bounds=torch.zeros((4, 2, 2, 64), **bf), scores=torch.zeros((3, 2, 4), device=device),
                selected=torch.zeros((3, 2, 2), **i32), lse=torch.zeros((3, 4), device=device),
                weights=torch.zeros((4, 2, 16), device=device), lens=torch.full((1,), 20, **i32),
                budget=torch.full((1,), 8, **i32), free_pages=torch.zeros(4, **i32),
                free_count=torch.zeros(1, **i32))


PYTHON = {
    "cache_bounds": (["k_pages", "block_table", "kv_lens", "bounds"], {}),
    "cache_score": (["q", "bounds", "block_table", "kv_lens", "cu_q"], dict(page_size=16)),
    "cache_select": (["scores", "kv_lens", "cu_q"], dict(page_size=16, count=2)),
    "cache_attend_selected": (["q", "k_pages", "v_pages", "block_table", "kv_lens", "cu_q",
                               "selected"], {}),
    "cache_weigh": (["q", "k_pages", "block_table", "kv_lens", "cu_q", "lse", "weights"], {}),
    "cache_evict": (["k_pages", "v_pages", "weights", "block_table", "lens", "budget",
                     "free_pages", "free_count"], {}),
}
FLOATS = {"k_pages", "v_pages", "q", "bounds", "scores", "lse", "weights"}


@pytest.mark.parametrize("name", PYTHON)
def test_binding_refuses_host_tensors(L, name):
    args, kw = PYTHON[name]
    x = tensors()
    with pytest.raises(ValueError, match="CUDA device"):
        getattr(sv, name)(*(x[a] for a in args), **kw)
    with pytest.raises(TypeError, match="must be a tensor"):
        getattr(sv, name)(None, *(x[a] for a in args[1:]), **kw)


@pytest.mark.parametrize("name,which", [(n, a) for n, (args, _) in PYTHON.items() for a in args
                                        if a in FLOATS and a == args[0]])
def test_binding_refuses_gradients(L, name, which):
    args, kw = PYTHON[name]
    x = tensors()
    x[which].requires_grad_()
    with pytest.raises(ValueError, match=f"{which} .*gradient"):
        getattr(sv, name)(*(x[a] for a in args), **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("name,which", [(n, a) for n, (args, _) in PYTHON.items() for a in args
                                        if a in FLOATS])
def test_binding_takes_tensors_of_gradients_without_them(L, name, which):
    args, kw = PYTHON[name]
    x = tensors("cuda:0")
    x[which].requires_grad_()
    with pytest.raises(ValueError, match=f"{which} .*gradient"):
        getattr(sv, name)(*(x[a] for a in args), **kw)
    with torch.no_grad():
        getattr(sv, name)(*(x[a] for a in args), **kw)


BAD = {  # of each argument something that it cannot be
    "k_pages": lambda t: [t[0], t.float(), t[..., ::2], t[:, :, :1]],
    "v_pages": lambda t: [t[:3], t.half(), t[..., ::2]],
    "block_table": lambda t: [t[0], t.long(), t.expand(2, 4), t[:, :0]],
    "kv_lens": lambda t: [t.long(), t.expand(2)],
    "lens": lambda t: [t.long(), t.expand(2)],
    "cu_q": lambda t: [t.long(), t[:1]],
    "q": lambda t: [t[0], t.half(), t[:, :3], t[..., :32], t.expand(1, 3, 4, 64)],
    "bounds": lambda t: [t[0], t.half(), t[:, :, :1], t[..., ::2]],
    "scores": lambda t: [t[0], t.half(), t[..., ::2]],
    "selected": lambda t: [t[:2], t.long(), t[:, :1], t[..., :0], t[..., ::2]],
    "lse": lambda t: [t[:2], t.double(), t[:, :3], t.t()],
    "weights": lambda t: [t[:3], t.double(), t[:, :1], t[..., ::2], t[0]],
    "budget": lambda t: [t.long(), t.expand(2)],
    "free_pages": lambda t: [t[:3], t.long()],
    "free_count": lambda t: [t.long(), t.expand(2)],
}


@pytest.mark.gpu
@pytest.mark.parametrize("name,which", [(n, a) for n, (args, _) in PYTHON.items() for a in args])
def test_binding_refuses(L, name, which):
    args, kw = PYTHON[name]
    good = tensors("cuda:0")
    getattr(sv, name)(*(good[a] for a in args), **kw)
    for bad in BAD[which](good[which]):
        x = dict(good, **{which: bad})
        with pytest.raises((ValueError, TypeError, sv.SpecVerifyError)):
            getattr(sv, name)(*(x[a] for a in args), **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("name,kw", [
    ("cache_bounds", dict(max_q=0)), ("cache_bounds", dict(max_q=1.5)),
    ("cache_bounds", dict(cu_q=torch.zeros(3))), ("cache_score", dict(page_size=5)),
    ("cache_score", dict(page_size=None)), ("cache_score", dict(max_q=-1)),
    ("cache_score", dict(out=torch.zeros((3, 2, 4)))), ("cache_select", dict(count=0)),
    ("cache_select", dict(first=2, recent=1)), ("cache_select", dict(first=-1)),
    ("cache_select", dict(page_size=0)), ("cache_attend_selected", dict(scale="1")),
    ("cache_attend_selected", dict(scale=math.nan)),
    ("cache_weigh", dict(decay=math.nan)), ("cache_weigh", dict(max_q=0)),
    ("cache_weigh", dict(scale=float("inf"))), ("cache_evict", dict(first=-1)),
    ("cache_evict", dict(recent=2 ** 40)), ("cache_evict", dict(status=torch.zeros(1)))])
def test_binding_refuses_numbers(L, name, kw):
    args, base = PYTHON[name]
    x = tensors("cuda:0")
    with pytest.raises((ValueError, TypeError, sv.SpecVerifyError)):
        getattr(sv, name)(*(x[a] for a in args), **dict(base, **kw))


@pytest.mark.gpu
def test_binding_refuses_overlaps(L):
    x = tensors("cuda:0")
    args = {n: [x[a] for a in a_] for n, (a_, _) in PYTHON.items()}
    with pytest.raises(sv.SpecVerifyError):
        sv.cache_attend_selected(*args["cache_attend_selected"], out=x["q"])
    with pytest.raises(sv.SpecVerifyError):
        sv.cache_evict(x["k_pages"], x["k_pages"], *args["cache_evict"][2:])
    with pytest.raises(sv.SpecVerifyError):
        sv.cache_select(*args["cache_select"], page_size=16, count=4,
                        out=x["scores"].view(torch.int32))
