"""The paged-cache operators on the GPU against their plain forms."""
import math

import pytest
import torch

import cache_ref as ref
import speculative_decoding_rejection_02_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def status_word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- step

def step_case(B, page, seed, gamma=7, new_hi=9, ctx_hi=300, spare=40):
    g = torch.Generator().manual_seed(seed)

    def pick(lo, hi):
        return torch.randint(lo, hi + 1, (B,), generator=g).tolist()
    drafts = pick(0, gamma)
    accepted = [min(a, d) for a, d in zip(pick(0, gamma), drafts)]
    held = [c + d for c, d in zip(pick(0, ctx_hi), drafts)]
    new = pick(0, new_hi)
    width = max([-(-(h + n) // page) for h, n in zip(held, new)] + [1]) + 1
    have = [-(-h // page) for h in held]
    pages = sum(have) + sum(-(-n // page) + 1 for n in new) + spare
    order = torch.randperm(pages, generator=g).tolist()
    table = [[order.pop() for _ in range(n)] + [-1] * (width - n) for n in have]
    free = order + [-7] * (pages - len(order))
    return dict(held=held, new=new, table=table, free=free, count=len(order), page=page,
                tokens=sum(new) + 5, drafts=drafts, accepted=accepted)


def run_step(c):
    starts = None
    if c["drafts"] is not None:
        starts = ints([sum(c["drafts"][:r]) for r in range(len(c["drafts"]) + 1)])
    width = len(c["table"][0]) if c["table"] else 1
    table = ints(c["table"]).reshape(len(c["held"]), width)
    free, status = ints(c["free"]), status_word()
    r = sv.cache_step(ints(c["held"]), ints(c["new"]), table, free, ints([c["count"]]),
                      page_size=c["page"], num_tokens=c["tokens"], cu_num_draft=starts,
                      num_accepted=None if starts is None else ints(c["accepted"]),
                      status=status)
    return dict(lens=r.lens.tolist(), cu_new=r.cu_new.tolist(), positions=r.positions.tolist(),
                slots=r.slots.tolist(), table=table.tolist(), free=free.tolist(),
                free_count=int(r.free_count)), int(status)


@pytest.mark.parametrize("B,page,kw", [
    (1, 16, {}), (1, 1, {}), (3, 8, dict(gamma=0)), (7, 16, {}), (64, 3, {}), (511, 16, {}),
    (512, 16, {}), (513, 16, {}), (1700, 32, dict(ctx_hi=60)), (40, 16, dict(new_hi=700)),
    (5, 64, dict(new_hi=0)), (2100, 5, dict(ctx_hi=30, new_hi=30))])
def test_step(B, page, kw):
    c = step_case(B, page, 11 + B, **kw)
    want = ref.step(**c)
    assert want is not None
    got, status = run_step(c)
    assert status == 0
    assert got == want


def test_step_without_drafts_and_without_requests():
    c = step_case(9, 16, 3)
    c.update(drafts=None, accepted=None)
    got, status = run_step(c)
    assert status == 0 and got == ref.step(**c)
    c = dict(held=[], new=[], table=[], free=[4, 5, 6], count=2, page=16, tokens=3, drafts=[],
             accepted=[])
    got, status = run_step(c)
    assert status == 0
    assert got == dict(lens=[], cu_new=[0], positions=[-1] * 3, slots=[-1] * 3, table=[],
                       free=[4, 5, 6], free_count=2)


def test_step_pages_given_back_are_taken_in_the_same_call():
    # an empty stack: every page taken is one that another request gives up
    c = dict(held=[64, 1, 40], new=[0, 60, 1], table=[[9, 8, 7, 6], [5, -1, -1, -1],
             [4, 3, 2, -1]], free=[-1] * 10, count=0, page=16, tokens=64,
             drafts=[50, 0, 30], accepted=[0, 0, 0])
    want = ref.step(**c)
    got, status = run_step(c)
    assert status == 0 and got == want
    assert want["table"][1] == [5, 2, 3, 6]


@pytest.mark.parametrize("change,bit", [
    (dict(count=3), sv.CACHE_NO_PAGES),
    (dict(tokens=10), sv.CACHE_BAD_LENGTHS),
    (dict(new=[-1] + [2] * 599), sv.CACHE_BAD_LENGTHS),
    (dict(held=[-5] * 600), sv.CACHE_BAD_LENGTHS),
    (dict(accepted=[0] * 599 + [8]), sv.CACHE_BAD_LENGTHS),
    (dict(new=[2] * 599 + [100000], tokens=200000), sv.CACHE_BAD_LENGTHS),
    (dict(count=-1), sv.CACHE_BAD_LENGTHS),
    (dict(count=10 ** 6), sv.CACHE_BAD_LENGTHS)])
def test_step_refuses_as_a_whole(change, bit):
    c = step_case(600, 16, 5)
    c.update(change)
    got, status = run_step(c)
    assert status == bit
    assert got == dict(lens=c["held"], cu_new=[0] * 601, positions=[-1] * c["tokens"],
                       slots=[-1] * c["tokens"], table=c["table"], free=c["free"],
                       free_count=c["count"])


def test_step_repeats():
    """The same inputs again give the same result: only the pages' owners changed."""
    c = step_case(300, 16, 8)
    first, _ = run_step(c)
    again = dict(c, table=first["table"], free=first["free"])
    assert run_step(again)[0] == first


def test_step_slots_past_32_bits():
    c = dict(held=[16], new=[2], table=[[5, -1]], free=[2 ** 31 - 1, 7], count=1,
             page=16, tokens=2, drafts=None, accepted=None)
    got, status = run_step(c)
    assert status == 0
    assert got["slots"] == [(2 ** 31 - 1) * 16, (2 ** 31 - 1) * 16 + 1]


def test_step_table_with_a_stride():
    c = step_case(20, 16, 21)
    want = ref.step(**c)
    width = len(c["table"][0])
    wide = torch.full((20, width + 3), -9, dtype=torch.int32, device=DEV)
    wide[:, :width] = ints(c["table"])
    starts = ints([sum(c["drafts"][:r]) for r in range(21)])
    r = sv.cache_step(ints(c["held"]), ints(c["new"]), wide[:, :width], ints(c["free"]),
                      ints([c["count"]]), page_size=16, num_tokens=c["tokens"],
                      cu_num_draft=starts, num_accepted=ints(c["accepted"]))
    assert wide[:, :width].tolist() == want["table"] and r.slots.tolist() == want["slots"]
    assert (wide[:, width:] == -9).all()


# -------------------------------------------------------------- append

@pytest.mark.parametrize("T,heads,dim,page,dtype,layout,shift", [
    (1, 8, 128, 16, torch.bfloat16, "token", 0), (37, 3, 80, 16, torch.float16, "head", 0),
    (300, 8, 128, 64, torch.bfloat16, "head", 0), (2000, 2, 96, 16, torch.float16, "token", 0),
    (19, 1, 7, 5, torch.bfloat16, "token", 0), (1300, 4, 64, 16, torch.float16, "token", 3),
    (65, 40, 128, 32, torch.bfloat16, "token", 0)])
def test_append(T, heads, dim, page, dtype, layout, shift):
    g = torch.Generator().manual_seed(T)
    pages = -(-T // page) + 3
    shape = (pages, heads, page, dim) if layout == "head" else (pages, page, heads, dim)
    kp, vp = torch.randn(shape, generator=g).to(dtype), torch.randn(shape, generator=g).to(dtype)
    if layout == "head":
        kp, vp = kp.transpose(1, 2), vp.transpose(1, 2)
    qkv = torch.randn((T, 3 * heads * dim + shift), generator=g).to(dtype)
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[::7] = -1
    if T > 8:
        slots[1] = -(2 ** 40)

    def heads_of(x, i):  # a slice of a fused projection, off its alignment by `shift`
        at = shift + i * heads * dim
        return x[:, at: at + heads * dim].view(T, heads, dim) if T == 1 else (
            x[:, at: at + heads * dim].unflatten(1, (heads, dim)))
    want_k, want_v = kp.clone(), vp.clone()
    for t in range(T):
        if slots[t] >= 0:
            want_k[slots[t] // page, slots[t] % page] = heads_of(qkv, 1)[t]
            want_v[slots[t] // page, slots[t] % page] = heads_of(qkv, 2)[t]
    gk, gv, x, status = kp.to(DEV), vp.to(DEV), qkv.to(DEV), status_word()
    assert gk.stride() == kp.stride()
    sv.cache_append(heads_of(x, 1), heads_of(x, 2), slots.to(DEV), gk, gv, status=status)
    assert int(status) == 0
    assert torch.equal(gk.cpu(), want_k) and torch.equal(gv.cpu(), want_v)


def test_append_skips_slots_past_the_pool():
    pages = torch.zeros((2, 16, 1, 64), dtype=torch.bfloat16, device=DEV)
    v_pages, status = pages.clone(), status_word()
    x = torch.ones((4, 1, 64), dtype=torch.bfloat16, device=DEV)
    slots = torch.tensor([31, 32, 2 ** 40, -1], device=DEV)
    sv.cache_append(x, x, slots, pages, v_pages, status=status)
    assert int(status) == sv.CACHE_BAD_SLOT
    want = torch.zeros((2, 16, 1, 64))
    want[1, 15] = 1
    assert torch.equal(pages.float().cpu(), want) and torch.equal(v_pages.float().cpu(), want)


# -------------------------------------------------------------- attend

def attend_case(q_lens, kv_lens, heads, kv_heads, dim, page, dtype, layout="token", seed=1,
                pad=0, loud=1.5, **kw):
    g = torch.Generator().manual_seed(seed)
    kp, vp, table, ks, vs = ref.cache(kv_lens, page, kv_heads, dim, dtype, g, layout, **kw)
    T = sum(q_lens)
    # queries as the front heads of a fused projection
    qkv = (torch.randn((T + pad, heads + 2 * kv_heads, dim), generator=g) * loud).to(dtype)
    starts = [0]
    for n in q_lens:
        starts.append(starts[-1] + n)
    gpu = dict(q=qkv.to(DEV)[:, :heads], k_pages=kp.to(DEV), v_pages=vp.to(DEV),
               block_table=table.to(DEV), kv_lens=ints(kv_lens), cu_q=ints(starts))
    return gpu, (qkv[:, :heads], ks, vs, q_lens)


def check_attend(q_lens, kv_lens, *args, window=0, sinks=0, scale=None, max_q=None, **kw):
    gpu, host = attend_case(q_lens, kv_lens, *args, **kw)
    status = status_word()
    got, lse = sv.cache_attend(**gpu, window=window, sinks=sinks, scale=scale, max_q=max_q,
                               return_lse=True, status=status)
    assert int(status) == 0
    ref.assert_attend(got, lse, ref.attend(*host, scale=scale, window=window, sinks=sinks))
    return gpu, got, lse


BF, FP = torch.bfloat16, torch.float16
SHAPES = [
    # q lengths, kv lengths, heads, kv heads, dim, page, type, layout
    ([1], [1], 1, 1, 64, 16, BF, "token"),
    ([1], [129], 8, 2, 128, 16, BF, "token"),
    ([1], [4097], 32, 8, 128, 16, FP, "head"),
    ([1] * 5, [1, 127, 128, 129, 700], 8, 8, 128, 32, BF, "token"),
    ([1, 2, 3, 4, 5], [500, 40, 3, 260, 5], 14, 2, 64, 16, FP, "token"),
    ([5, 0, 1, 0, 8], [70, 33, 0, 0, 1000], 12, 4, 96, 8, BF, "head"),
    ([130], [130], 4, 1, 128, 64, BF, "token"),
    ([257, 3], [300, 1111], 6, 2, 80, 16, FP, "token"),
    ([40], [2000], 71, 1, 64, 16, BF, "token"),
    ([3], [900], 128, 1, 128, 128, FP, "token"),
    ([2], [650], 4, 4, 8, 256, BF, "head"),
    ([9], [77], 5, 1, 72, 8, FP, "token"),
    ([64, 64, 64], [64, 1000, 192], 8, 2, 128, 16, BF, "token"),
    ([1] * 300, [1 + 3 * i for i in range(300)], 2, 1, 64, 16, FP, "token"),
    ([600], [900], 3, 3, 128, 16, BF, "token"),
]


@pytest.mark.parametrize("shape", SHAPES, ids=range(len(SHAPES)))
def test_attend(shape):
    check_attend(*shape[:-1], layout=shape[-1])


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 4), (64, 0), (128, 128), (100, 3),
                                          (1000, 16), (5, 4000), (10 ** 6, 4), (129, 130)])
@pytest.mark.parametrize("shape", [SHAPES[2], SHAPES[4], SHAPES[5], SHAPES[7], SHAPES[12]],
                         ids=[2, 4, 5, 7, 12])
def test_attend_window(shape, window, sinks):
    check_attend(*shape[:-1], layout=shape[-1], window=window, sinks=sinks)


def test_attend_rows_that_see_nothing():
    # fewer cached tokens than new ones: the first rows stand before position 0
    check_attend([5, 4, 300], [2, 0, 131], 8, 2, 128, 16, BF)
    check_attend([5, 4, 300], [2, 0, 131], 8, 2, 64, 16, FP, window=3, sinks=1)


def test_attend_padding_rows():
    """Rows past the last request give zeros."""
    gpu, host = attend_case([2, 3], [50, 60], 8, 2, 128, 16, BF, pad=4)
    got, lse = sv.cache_attend(**gpu, return_lse=True)
    want = ref.attend(*host)
    ref.assert_attend(got, lse, want)
    assert (got[5:] == 0).all() and torch.isinf(lse[5:]).all()


def test_attend_no_requests():
    gpu, _ = attend_case([2], [50], 8, 2, 128, 16, BF)
    gpu.update(block_table=gpu["block_table"][:0], kv_lens=gpu["kv_lens"][:0], cu_q=ints([0]))
    got, lse = sv.cache_attend(**gpu, return_lse=True)
    assert (got == 0).all() and torch.isinf(lse).all()
    gpu["q"] = gpu["q"][:0]
    assert sv.cache_attend(**gpu).shape == (0, 8, 128)


def test_attend_infinite_rubbish_and_given_away_pages():
    check_attend([1, 6], [200, 333], 8, 2, 128, 16, FP, rubbish=float("inf"))
    # pages before the window hold NaN now: no row sees them
    gpu, host = attend_case([3, 1], [1500, 700], 8, 2, 128, 16, BF)
    window, sinks = 100, 5
    for r, n in enumerate([1500, 700]):
        first = n - host[3][r] - window + 1  # of the first row's window
        for c in range(1, first // 16):
            page = int(gpu["block_table"][r, c])
            gpu["k_pages"][page] = float("nan")
            gpu["v_pages"][page] = float("nan")
        gpu["block_table"][r, 2: first // 16] = -1
        # and the tokens beside the sinks in the first page, and before the window in its page
        page = int(gpu["block_table"][r, 0])
        gpu["k_pages"][page, sinks:] = float("nan")
        gpu["v_pages"][page, sinks:] = float("nan")
        page = int(gpu["block_table"][r, first // 16])
        gpu["v_pages"][page, : first % 16] = float("nan")
        gpu["k_pages"][page, : first % 16] = float("inf")
    status = status_word()
    got, lse = sv.cache_attend(**gpu, window=window, sinks=sinks, return_lse=True, status=status)
    assert int(status) == 0
    ref.assert_attend(got, lse, ref.attend(*host, window=window, sinks=sinks))


@pytest.mark.parametrize("dtype", [BF, FP])
def test_attend_extreme_scores(dtype):
    # scores of a few hundred either way: one token carries each row
    check_attend([7, 1], [400, 260], 8, 2, 64, 16, dtype, loud=40.0)
    # a rising row: every tile brings a new maximum
    gpu, host = attend_case([4], [2000], 4, 1, 64, 16, dtype)
    for j in range(2000):
        k = torch.full((1, 64), j / 256.0).to(dtype)
        host[1][0][j] = k
        gpu["k_pages"][int(gpu["block_table"][0, j // 16]), j % 16] = k.to(DEV)
    gpu["q"][:] = 1.0
    host[0][:] = 1.0
    got, lse = sv.cache_attend(**gpu, scale=0.5, return_lse=True)
    ref.assert_attend(got, lse, ref.attend(*host, scale=0.5))


@pytest.mark.parametrize("seed", range(16))
def test_attend_random(seed):
    """Ragged batches of any make-up: empty requests, single tokens and chunks side by side."""
    g = torch.Generator().manual_seed(100 + seed)

    def pick(lo, hi):
        return int(torch.randint(lo, hi + 1, (1,), generator=g))
    B = pick(1, 30)
    kv_heads = pick(1, 3)
    heads = kv_heads * pick(1, 9)
    dim = 8 * pick(1, 16)
    q_lens = [pick(0, 1) * pick(0, (3, 40, 200)[pick(0, 2)]) for _ in range(B)]
    kv_lens = [max(0, n + pick(-3, (10, 300, 1500)[pick(0, 2)])) for n in q_lens]
    window = pick(0, 1) * pick(1, 400)
    check_attend(q_lens, kv_lens, heads, kv_heads, dim, 8 << pick(0, 5), (BF, FP)[seed % 2],
                 layout=("token", "head")[pick(0, 1)], seed=seed, window=window,
                 sinks=pick(0, 1) * pick(0, 200), max_q=pick(0, 1) * pick(1, 50) or None)


def test_attend_more_requests_than_threads():
    """The list's head is found in runs of requests; many of them have no rows."""
    q_lens = [(r * 7) % 3 if r % 5 else 0 for r in range(700)]
    check_attend(q_lens, [n + (r * 31) % 150 for r, n in enumerate(q_lens)], 4, 2, 64, 16, BF)
    check_attend([0] * 400 + [3], [20] * 400 + [500], 4, 2, 64, 16, FP)


def test_attend_scale_and_negative_scale():
    check_attend([3], [300], 8, 2, 128, 16, BF, scale=0.02)
    check_attend([3], [300], 8, 2, 128, 16, BF, scale=-0.11)
    check_attend([3], [300], 8, 2, 128, 16, FP, scale=0.0)


@pytest.mark.parametrize("max_q", [1, 4, 1000])
def test_attend_max_q_is_speed_only(max_q):
    _, got, lse = check_attend([1, 70, 6], [500, 900, 30], 8, 2, 128, 16, BF, max_q=max_q)
    _, base, base_lse = check_attend([1, 70, 6], [500, 900, 30], 8, 2, 128, 16, BF)
    assert torch.allclose(got.float(), base.float(), atol=0.02)


def test_attend_long_context_and_split():
    """Few rows over a long context: the work is split over the tokens."""
    check_attend([2], [70001], 8, 2, 128, 64, BF)
    check_attend([1, 1], [50000, 3], 4, 1, 64, 16, FP)
    check_attend([200], [20000], 4, 1, 128, 64, BF)


def test_attend_is_reproducible():
    """Equal to the bit whatever ran on the SMs before and lies in the workspace, with
    units of one and of two tiles of rows side by side in a block's part of the work."""
    gpu, host = attend_case([3, 40, 1], [5000, 900, 20000], 16, 4, 128, 16, BF)
    other, _ = attend_case([7, 50], [700, 3000], 16, 4, 128, 16, FP, seed=9, loud=3.0)
    a, al = sv.cache_attend(**gpu, return_lse=True)
    ref.assert_attend(a, al, ref.attend(*host))
    for k in range(12):
        if k % 3 == 0:
            rubbish = torch.full((10 ** 7,), math.nan if k % 2 else 7.0, device=DEV)
            del rubbish
        elif k % 3 == 1:
            sv.cache_attend(**other, max_q=5 + k)
        b, bl = sv.cache_attend(**gpu, return_lse=True)
        assert torch.equal(a, b) and torch.equal(al, bl), k


def test_attend_offsets_past_32_bits():
    """Pages whose elements lie past 2^31 from the pool's start."""
    page, heads, dim = 16, 8, 128
    pages = 2 ** 31 // (page * heads * dim) + 40
    gpu, host = attend_case([5], [100], 32, 8, 128, 16, BF)
    far = torch.arange(pages - 7, pages, dtype=torch.int32, device=DEV)
    big_k = torch.empty((pages, page, heads, dim), dtype=BF, device=DEV)
    big_v = torch.empty_like(big_k)
    used = gpu["block_table"][0, :7].long()
    big_k[far.long()] = gpu["k_pages"][used]
    big_v[far.long()] = gpu["v_pages"][used]
    table = far.flip(0).reshape(1, 7).contiguous()
    big_k[far.long().flip(0)] = gpu["k_pages"][used]
    big_v[far.long().flip(0)] = gpu["v_pages"][used]
    got, lse = sv.cache_attend(gpu["q"], big_k, big_v, table, gpu["kv_lens"], gpu["cu_q"],
                               return_lse=True)
    ref.assert_attend(got, lse, ref.attend(*host))
    # and an append there
    x = torch.randn((2, 8, 128), device=DEV).to(BF)
    slots = torch.tensor([pages * page - 1, (pages - 3) * page], device=DEV)
    sv.cache_append(x, x, slots, big_k, big_v)
    assert torch.equal(big_k[pages - 1, 15], x[0]) and torch.equal(big_v[pages - 3, 0], x[1])


def test_attend_strided_output_and_other_stream():
    gpu, host = attend_case([3, 9], [333, 50], 8, 2, 128, 16, BF)
    side = torch.cuda.Stream()
    wide = torch.zeros((12, 10, 128), dtype=BF, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    got, lse = sv.cache_attend(**gpu, out=wide[:, 1:9], return_lse=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    ref.assert_attend(wide[:, 1:9], lse, ref.attend(*host))
    assert (wide[:, 0] == 0).all() and (wide[:, 9] == 0).all()


def test_attend_bad_device_data_sets_bits():
    gpu, host = attend_case([2, 3], [50, 60], 8, 2, 128, 16, BF)
    for name, value, bit in (("kv_lens", [50, -1], sv.CACHE_BAD_LENGTHS),
                             ("kv_lens", [50, 10 ** 6], sv.CACHE_BAD_LENGTHS),
                             ("cu_q", [0, 2, 1], sv.CACHE_BAD_LENGTHS),
                             ("cu_q", [0, 2, 99], sv.CACHE_BAD_LENGTHS)):
        bad, status = dict(gpu), status_word()
        bad[name] = ints(value)
        got = sv.cache_attend(**bad, status=status)
        assert int(status) == bit, name
        # the request beside it is as ever
        want, _, tol, _ = ref.attend(*host)
        assert ((got.double().cpu() - want).abs() <= tol)[:2].all()
    table, status = gpu["block_table"].clone(), status_word()
    table[1, 0], table[1, 1] = -3, 10 ** 6
    sv.cache_attend(**dict(gpu, block_table=table), status=status)
    assert int(status) == sv.CACHE_BAD_PAGE


def test_attend_binding_refusals():
    gpu, _ = attend_case([2], [50], 8, 2, 128, 16, BF)
    for kw in (dict(q=gpu["q"][:, :7]), dict(q=gpu["q"].half()), dict(kv_lens=ints([50, 1])),
               dict(kv_lens=gpu["kv_lens"].long()), dict(block_table=gpu["block_table"].long()),
               dict(v_pages=gpu["v_pages"][:, :8]), dict(out=gpu["q"][:1])):
        with pytest.raises((ValueError, TypeError)):
            sv.cache_attend(**dict(gpu, **kw))
    with pytest.raises(sv.SpecVerifyError):
        sv.cache_attend(**gpu, window=-1)
    odd = torch.zeros((2, 8, 132), dtype=BF, device=DEV)[:, :, 4:]
    with pytest.raises(sv.SpecVerifyError):
        sv.cache_attend(**dict(gpu, q=odd))
    with pytest.raises(TypeError):
        sv.cache_attend(**{k: v.float() if v.is_floating_point() else v for k, v in gpu.items()})


def test_calls_in_a_graph():
    """The three calls allocate nothing of their own and can be captured."""
    gpu, host = attend_case([3, 9], [333, 50], 8, 2, 128, 16, BF)
    sv.cache_attend(**gpu)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out, lse = sv.cache_attend(**gpu, return_lse=True)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    ref.assert_attend(out, lse, ref.attend(*host))
    assert math.isfinite(float(lse.sum()))
