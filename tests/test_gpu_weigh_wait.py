"""A wait of cache_weigh that runs out."""
import ctypes as C

import pytest
import torch

import cache_ref
import sparse_ref as ref
import speculative_decoding_rejection_02_gb300 as sv
from test_gpu_sparse import BF, DEV, FP, ints, spread_weights, starts, status_word


def c_args(q, kp, table, lens, cu, lse, w, max_q, flags):
    """The C ABI's structure for these tensors."""
    a = sv.WeighArgs(B=lens.numel(), width=table.shape[1], table_stride=table.stride(0),
                     num_tokens=q.shape[0], max_q=max_q, heads=q.shape[1], kv_heads=kp.shape[2],
                     dim=q.shape[2], page_size=kp.shape[1], num_pages=kp.shape[0],
                     dtype=1 if q.dtype == BF else 2, scale=q.shape[2] ** -0.5, decay=1.0,
                     flags=flags)
    a.q, a.q_token, a.q_head = q.data_ptr(), q.stride(0), q.stride(1)
    a.k_pages, a.kp_page, a.kp_token, a.kp_head = (kp.data_ptr(), kp.stride(0), kp.stride(1),
                                                   kp.stride(2))
    a.block_table, a.kv_lens, a.cu_q = table.data_ptr(), lens.data_ptr(), cu.data_ptr()
    a.lse, a.weights, a.w_page, a.w_head = lse.data_ptr(), w.data_ptr(), w.stride(0), w.stride(1)
    return a


def test_unknown_flags_are_refused():
    zero = torch.zeros(1, dtype=torch.int32)
    x = torch.zeros((1, 1, 64), dtype=BF)
    for flags, rc in ((2, -1), (3, -1), (1 << 31, -1), (0, -2), (1, -2)):  # (-2: pages of one token)
        a = c_args(x, x[None], zero[None], zero, zero, torch.zeros(1, 1), torch.zeros(1, 1, 1), 1,
                   flags)
        assert sv.lib().spec_cache_weigh(C.byref(a), None, None) == rc


@pytest.mark.gpu
@pytest.mark.parametrize("q_lens,kv_lens,max_q,dim,dtype", [
    ([1, 3], [700, 40], 3, 128, BF),                   # one column tile, keys loaded by two warps
    ([300, 1, 64], [2500, 9000, 64], 300, 64, FP),     # many column tiles
    ([1] * 40, [5000] * 40, 1, 128, BF)])              # parts of many pairs
def test_a_wait_that_runs_out(q_lens, kv_lens, max_q, dim, dtype):
    """The sums wait for a signal that never comes: every role of the kernel gives up, what it has
    in flight lands, and the next call, on the same multiprocessors, is right."""
    g = torch.Generator().manual_seed(51)
    kp, vp, table, ks, vs = cache_ref.cache(kv_lens, 16, 2, dim, dtype, g)
    q = torch.randn((sum(q_lens), 8, dim), generator=g).to(dtype)
    _, lse, _, _ = cache_ref.attend(q, ks, vs, q_lens)
    lse = lse.float()
    before = [torch.rand((2, n), generator=g) for n in kv_lens]
    weights = torch.zeros((kp.shape[0], 2, 16))
    spread_weights(weights, before, table, 16)
    want, tol = ref.weigh(q, ks, q_lens, lse, before)
    dev = [x.to(DEV) for x in (q, kp, table, ints(kv_lens), starts(q_lens), lse)]
    stream = torch.cuda.current_stream().cuda_stream
    for _ in range(2):
        w, status = weights.to(DEV), status_word()
        a = c_args(*dev, w, max_q, sv.CACHE_TEST_WAIT_TIMEOUT)
        assert sv.lib().spec_cache_weigh(C.byref(a), stream, status.data_ptr()) == 0
        assert int(status) == sv.STATUS_TIMEOUT
        w, status = weights.to(DEV), status_word()
        sv.cache_weigh(*dev, w, max_q=max_q, status=status)
        assert int(status) == 0
        w = w.double().cpu()
        for r, (x, off) in enumerate(zip(want, tol)):
            rows = [w[table[r, c]] for c in range(-(-kv_lens[r] // 16))]
            assert ((torch.cat(rows, 1)[:, : kv_lens[r]] - x).abs() <= off).all(), r
