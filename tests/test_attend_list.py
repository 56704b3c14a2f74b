"""The attention's list of key tiles and the blocks' walk over it, compiled for the
host: every key tile of every unit is met once, by the block whose part it lies in."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
TILE, COST, PAIR_COST = 128, 2, 4
SEG = np.dtype([(n, "<i4") for n in (
    "n", "i0", "b", "head", "token", "tokens", "pos", "lo", "hi", "gap_at", "gap", "pair", "q_at",
    "ring", "slot")])
JOIN = np.dtype([(n, "<i4") for n in ("last", "head", "token", "tokens")])


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("list") / "attend_list.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-fPIC", "-shared", "-o", so,
                    os.path.join(HERE, "attend_list.cpp")], check=True)
    lib = C.CDLL(so)
    lib.list_before.restype = C.c_longlong
    return lib


def units_of(cu, kv, kv_heads, tile_tokens, window, sinks):
    """The list's units in order, from the definition: what each sees and takes."""
    step, sink_tiles, rows = 2 * tile_tokens, -(-sinks // TILE), []
    for b, length in enumerate(kv):
        q = cu[b + 1] - cu[b]
        u = np.arange(-(-q // step), dtype=np.int64)
        first = length - q + u * step                       # position of the first row
        end = np.minimum(first + step, length)
        lo = np.maximum(first + 1 - window, 0) if window else 0 * u
        # tiles [0, sinks' tiles) and [lo's tile, the last row's]
        from_tile, to_tile = lo // TILE, np.maximum(end - 1, 0) // TILE + 1
        gap = np.maximum(from_tile - sink_tiles, 0)
        rec = np.zeros(len(u), dtype=[(n, "<i8") for n in (
            "b", "head", "token", "tokens", "pos", "lo", "hi", "gap", "tiles", "cost")])
        rec["b"], rec["token"] = b, cu[b] + u * step
        rec["tokens"] = np.minimum(step, q - u * step)
        rec["pos"], rec["lo"], rec["hi"] = first, lo, np.maximum(end, 0)
        rec["gap"] = np.where(end > 0, gap, 0)
        rec["tiles"] = np.where(end > 0, to_tile - gap, 1)
        rec["cost"] = PAIR_COST if q > tile_tokens else COST
        for h in range(kv_heads):
            rec["head"] = h
            rows.append(rec.copy())
    return np.concatenate(rows)


def check_walk(L, q_lens, kv, kv_heads, tile_tokens, window=0, sinks=0, grid=152):
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    kv = np.asarray(kv, dtype=np.int32)
    units = units_of(cu.tolist(), kv.tolist(), kv_heads, tile_tokens, window, sinks)
    places = units["tiles"] + units["cost"]
    start = np.cumsum(places) - places
    total = int(places.sum())
    blocks = min(grid, total)
    most = len(units) + 2 * grid + 1
    segs, first = np.zeros(most, SEG), np.zeros(grid + 1, np.int64)
    joins = np.zeros(grid, JOIN)

    def ptr(x):
        return C.c_void_p(x.ctypes.data)
    got = L.list_walk(ptr(cu), ptr(kv), len(kv), kv_heads, tile_tokens, window, sinks, grid,
                      ptr(segs), C.c_longlong(most), ptr(first), ptr(joins))
    assert got == blocks
    segs = segs[: first[blocks]].astype(
        [(n, "<u4" if n == "ring" else "<i4") for n in SEG.names])
    # what is expected: cut the places at the units' starts and the parts' ends
    part, more = divmod(total, blocks)
    begins = np.arange(blocks, dtype=np.int64) * part + np.minimum(np.arange(blocks), more)
    cuts = np.unique(np.concatenate([start, begins]))
    u = np.searchsorted(start, cuts, side="right") - 1
    c = np.searchsorted(begins, cuts, side="right") - 1
    i0 = cuts - start[u]
    n = np.minimum(np.append(cuts[1:], total) - start[u], units["tiles"][u]) - i0
    live = n > 0
    u, c, i0, n = u[live], c[live], i0[live], n[live]
    assert len(segs) == len(u)
    x = units[u]
    assert np.array_equal(segs["n"], n) and np.array_equal(segs["i0"], i0)
    for name in ("b", "head", "token", "tokens", "pos", "lo", "hi"):
        assert np.array_equal(segs[name], x[name]), name
    pair = x["tokens"] > tile_tokens
    assert np.array_equal(segs["pair"] != 0, pair)
    whole, starts = (i0 == 0) & (n == x["tiles"]), i0 == 0
    assert np.array_equal(segs["slot"], np.where(whole, -1, np.where(starts, 1, 0)))
    for k in (0 * n, n - 1):  # an entry's first and last tile
        place = i0 + k
        tile = np.where(place < segs["gap_at"], place, place + segs["gap"])
        sink_tiles = -(-sinks // TILE)
        want = np.where(place < np.where(x["gap"] > 0, sink_tiles, place + 1), place,
                        place + x["gap"])
        assert np.array_equal(tile, want)
    for block in np.unique(c):
        mine = c == block
        assert first[block + 1] - first[block] == mine.sum()
        at = np.cumsum(np.where(pair[mine], 2, 1)) - np.where(pair[mine], 2, 1)
        assert np.array_equal(segs["q_at"][mine], at)
        ring = 2 * (np.cumsum(n[mine]) - n[mine])
        assert np.array_equal(segs["ring"][mine], ring)
    # units that end in a later block than they start in
    last_c = np.full(len(units), -1)
    first_c = np.full(len(units), blocks)
    np.maximum.at(last_c, u, c)
    np.minimum.at(first_c, u, c)
    split = np.flatnonzero(first_c < last_c)
    want = np.full(blocks, -1)
    want[first_c[split]] = last_c[split]
    assert np.array_equal(joins["last"][:blocks], want)
    for name in ("head", "token", "tokens"):
        assert np.array_equal(joins[name][first_c[split]], units[name][split])


@pytest.mark.parametrize("seed", range(60))
def test_every_tile_once(L, seed):
    r = np.random.default_rng(seed)
    B = int(r.integers(1, 200 if seed % 4 == 0 else 12))
    q = np.where(r.random(B) < 0.2, 0, r.integers(1, 300 if seed % 3 == 0 else 7, B))
    if q.sum() == 0:
        q[0] = 1
    kv = q + r.integers(0, 500 if seed % 2 else 6000, B)
    kv = np.where(r.random(B) < 0.1, r.integers(0, q + 3), kv)  # rows before position 0
    window = int(r.integers(0, 2) * r.integers(1, 700))
    check_walk(L, q.tolist(), kv.tolist(), int(r.integers(1, 5)), int(r.integers(1, 41)), window,
               int(r.integers(0, 300)) if window else 0, 152 if seed % 2 else 7)


@pytest.mark.parametrize("window,sinks", [(0, 0), (2000, 16), (1, 0), (130, 100000)])
def test_units_before_in_closed_form(L, window, sinks):
    r = np.random.default_rng(window)
    for _ in range(300):
        q, step = int(r.integers(1, 5000)), 2 * int(r.integers(1, 129))
        length = int(max(0, q + r.integers(-300, 40000)))
        x = units_of([0, q], [length], 1, step // 2, window, sinks)
        want = np.concatenate([[0], np.cumsum(x["tiles"] + x["cost"])])
        for k in {0, len(x), int(r.integers(0, len(x) + 1))}:
            assert L.list_before(length, q, step, window, sinks, k) == want[k]


LONG = [
    # new tokens, length, kv heads, new tokens of a tile of rows, window, sinks
    (1600000, 1600000, 1, 1, 0, 0),   # 5.0e9 places
    (1 << 20, 1 << 20, 8, 8, 0, 0),   # 2.1e9
    (400000, 400000, 8, 1, 0, 0),     # 2.5e9
    (1500000, 1400000, 1, 1, 0, 0),   # rows before position 0
    (3000000, 3000000, 2, 1, 2000000, 300),
    (300000, 0x7fff0000, 1, 128, 0, 0),
    (5, 0x7fff0000, 64, 5, 0, 0),
]


@pytest.mark.parametrize("q,length,kv_heads,tile_tokens,window,sinks", LONG)
def test_lists_past_32_bits(L, q, length, kv_heads, tile_tokens, window, sinks):
    x = units_of([0, q], [length], 1, tile_tokens, window, sinks)
    want = np.concatenate([[0], np.cumsum(x["tiles"] + x["cost"])])
    for k in (0, 1, len(x) // 3, len(x) - 1, len(x)):
        if k >= 0:
            assert L.list_before(length, q, 2 * tile_tokens, window, sinks, k) == want[k]
    check_walk(L, [3, q, 7], [2000, length, 9], kv_heads, tile_tokens, window, sinks)


def test_longest_request(L):
    """The most places that one request's lengths give: far from 64 bits."""
    length, q, step = 2 ** 31 - 2 ** 16, 2 ** 22, 2
    first = length - q + np.arange(q // step, dtype=np.int64) * step
    tiles = (first + step - 1) // TILE + 1
    want = int(tiles.sum()) + PAIR_COST * (q // step)
    assert L.list_before(length, q, step, 0, 0, q // step) == want > 2 ** 45 - 2 ** 43
    # units of two, as many as q can have: the formula stays exact
    q = 2 ** 31 - 2 ** 17
    n = q // step
    at = length - q + step - 1  # of unit 0's last row; tiles (at + 2 u) / 128 + 1
    total = sum((at % TILE + step * v) // TILE for v in range(TILE))
    h = n // TILE
    want = n * (at // TILE) + h * total + step * TILE * (h * (h - 1) // 2) + n * (1 + PAIR_COST)
    assert n % TILE == 0
    assert L.list_before(length, q, step, 0, 0, n) == want
