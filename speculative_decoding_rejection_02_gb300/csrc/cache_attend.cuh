// Attention of a round's new tokens over the paged cache (spec_cache_attend).
//
// The rows of one kv head are the new tokens times the G query heads that
// share it: a tile of 128 rows is floor(128 / G) tokens (or as many as a
// request is expected to have), so a round's few tokens still read each key
// and value once for all their heads. Keys come in tiles of 128 tokens:
//
//   S = Q K^T       tcgen05, Q and K in shared memory, S (fp32) in TMEM
//   P = 2^(c S - m) one thread per row: running maximum m and sum l in fp32,
//                   P rounded to the cache's type and written over S
//   O += P V        tcgen05, P from TMEM, V in shared memory, O (fp32) in TMEM
//
// with c = scale * log2(e). P's rounding is the one step below 32 bits before
// the result's own: the tensor cores take 16-bit operands. l sums P unrounded.
// m and O follow a higher maximum only when it has passed m by 2^8: until then P
// may exceed 1, which costs no precision (bf16 and fp32 have the range; fp16's P
// starts at 2^7, may reach 2^15 and goes down to 2^-31 of it).
//
// Two streams of S and O run side by side in one block, so that one's products
// cover the other's softmax: two tiles of rows over the same keys where a unit
// has more than one tile of rows, else the even and the odd key tiles of the
// one tile of rows, joined at the end.
//
// Work is one list of key tiles over (request, kv head, tiles of rows), cut
// into equal parts, one for each block (one block per SM): ragged batches
// balance without a plan on the host, and a unit that a cut crosses leaves
// partial (m, l, O) in the workspace, which k_attend_join joins. Tiles that no
// row of a unit sees are not in the list.
//
// Warps: 0-3 and 4-7 the softmax of stream 0 and 1, 8 and 11 the loaders (TMA,
// through the block table; 11 also walks over the list), 9 and 10 the issuers of
// the two streams' products; the last four give registers to the softmax warps.
//
// What bounds it, on one GB300 (6792 GB/s, 1876 TFLOP/s bf16 measured):
//  - long contexts and few rows: HBM. 64 requests of 2-8 tokens over 1000-30000
//    (heads of 128): 0.346 ms, 6.48 TB/s; 128 single tokens over 150-9000: 0.188 ms,
//    6.04 TB/s, the rest a unit's start and results (about 4000 clocks each, partly
//    behind its successor's loads).
//  - prompt chunks: the chain softmax -> PV -> QK of one stream against the other's.
//    Two chunks of 2048 over 11000-14000: 0.58 ms (1560 TFLOP/s) in a short run, 0.66 ms
//    (1370) when the clocks follow the power limit.
//  - small calls: the chain from launch to the first result and the join (one token over
//    one cached token 12.1 us, over 4097 15.3).
//  - windows: many short units, each with its start and its results (64 requests of 1-6
//    tokens in a window of 1024: 66.5 us; over 1024 tokens without a window 61.5).
// Code size counts: the warps' loops together overflow the instruction cache, and
// rolling the softmax's, shortening the waits' and moving rare paths out of the way
// took the chunks from 1.13 ms to 0.58.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/spec_cache.h"
#include "attend_list.cuh"
#include "pipe.cuh"
#include "tcgen05.cuh"

namespace sv {

constexpr int kAttThreads = 384;  // 12 warps, at most 168 registers each at launch
constexpr int kAttScan = 128;     // threads that scan the requests
constexpr int kAttRegsMany = 208, kAttRegsFew = 88;  // 2 * 208 + 88 = 3 * 168
constexpr int kAttSegs = 4;       // list entries ahead of the slowest warp
constexpr long long kAttPatience = 2000000000;  // clocks that a wait may take
constexpr float kAttGrow = 8.f;   // log2 of how far a row's maximum may grow unscaled

template <int DP>
struct AttCfg {
  static constexpr int kTileBytes = kAttTile * DP * 2;
  static constexpr int kStages = DP == 128 ? 5 : 10;  // of one K or V tile each
  // Barriers go by a longer ring than the tiles: no warp is ever kRing loads behind another,
  // so a phase's parity says which load is meant, whichever of them a warp waits for.
  static constexpr int kRing = DP == 128 ? 16 : 32;
  static constexpr int kSmem = (2 + kStages) * kTileBytes + (DP == 128 ? 3 : 4) * 1024;
};

struct AttendParams {
  CUtensorMap q_map, k_map, v_map;
  int B, T, heads, kv_heads, G, dim;
  int page_shift, width;
  long long num_pages, table_stride;
  const int* table;
  const int* kv_lens;
  const int* cu_q;
  char* out;
  long long out_token, out_head;  // bytes
  float* lse;
  float c;       // scale * log2(e)
  float hidden;  // score that c takes to -inf
  int window, sinks;
  int tile_tokens;  // new tokens of a tile of rows
  unsigned* status;
  float4* part_o;   // [blocks][2][2 tiles][DP / 4][128] partial outputs
  float2* part_ml;  // [blocks][2][2][128] their maxima and sums
  AttJoin* join;  // [blocks]

  // The new tokens of request b as rows [lo, hi) of q, and its length. Offsets
  // that cannot be give no rows (lo = hi = -1), a length that cannot be length 0.
  __device__ __forceinline__ int request(int b, int& lo, int& hi) const {
    lo = cu_q[b];
    hi = cu_q[b + 1];
    int len = kv_lens[b];
    const bool bad_rows = lo < 0 || hi < lo || hi > T;
    // (the last key tiles' ends stay below 2^31)
    const bool bad_len = len < 0 || len > ((long long)width << page_shift) || len > 0x7fff0000;
    if (bad_rows || bad_len) {
      atomicOr(status, SPEC_CACHE_BAD_LENGTHS);
      if (bad_rows) lo = hi = -1;
      len = 0;
    }
    return len;
  }
};

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

struct AttBase {
  uint64_t q_full[4], q_empty[2];
  uint64_t s_full[2], p_half[2], p_full[2];
  uint64_t turn[2], warm;
  uint64_t o_full, o_free, ml_full, edge_full, drain[2];
  uint64_t seg_full[kAttSegs], seg_empty[kAttSegs];
  AttSeg seg[kAttSegs];
  float2 ml[2][kAttTile];
  long long scan[kAttScan / 32];
  int pad[kAttScan / 32], pad_all;
  int gaps;  // some rows before pad_all may belong to no request
  AttWalk walk;
  int entry;  // the walk's next
  uint32_t tmem;
  int stop;
};
template <int DP>
struct AttShared : AttBase {
  uint64_t kv_full[AttCfg<DP>::kRing], kv_empty[AttCfg<DP>::kRing];
};
static_assert(sizeof(AttShared<128>) <= 3 * 1024 && sizeof(AttShared<64>) <= 4 * 1024,
              "shared memory beside the tiles");

// A bounded wait (about a second); once one has run out every later one returns at once. The
// probes carry no time limit of their own: one with a limit costs three times as much.
__device__ __forceinline__ bool att_wait(AttBase& sh, const AttendParams& p, uint64_t* bar,
                                         uint32_t parity) {
  if (__builtin_expect(mbar_poll(bar, parity & 1), 1)) return true;
  const long long from = clock64();
  do {
    if (mbar_poll(bar, parity & 1)) return true;
  } while (!*(volatile int*)&sh.stop && clock64() - from < kAttPatience);
  *(volatile int*)&sh.stop = 1;
  atomicOr(p.status, SPEC_STATUS_TIMEOUT);
  return false;
}

// The wait for what a warp has in flight when it ends: 20 ms at most (one for what was never
// issued takes its limit).
__device__ __forceinline__ void att_land(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < 1024; ++i)
    if (mbar_try(bar, parity & 1)) break;
}

// att_wait for a whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool att_wait_warp(AttBase& sh, const AttendParams& p, uint64_t* bar,
                                              uint32_t parity) {
  return __all_sync(~0u, att_wait(sh, p, bar, parity));
}

// Place of key tile i's K and V among the 2 n loads of a segment: in the order
// in which the products use them.
__device__ __forceinline__ int att_k_at(bool pair, int i) {
  return pair ? 2 * i : i ? 2 * i - 1 : 0;
}
__device__ __forceinline__ int att_v_at(bool pair, int i, int n) {
  return pair ? 2 * i + 1 : min(2 * i + 2, 2 * n - 1);
}

// ---- the walk over this block's part of the list: begun by the thread whose run of requests
// the part starts in, carried on by one of the V loader's

// Puts the walk's next entry, or the end mark, into the ring; nothing once that is there.
__device__ __forceinline__ bool att_publish(AttWalk& walk, int& entry, AttBase& sh,
                                            const AttendParams& p) {
  if (entry < 0) return true;
  const int at = entry % kAttSegs;
  AttSeg g;
  walk.next(p, g);
  if (g.n == 0) p.join[blockIdx.x] = walk.join;
  if (!att_wait(sh, p, &sh.seg_empty[at], (entry / kAttSegs + 1) & 1)) return false;
  sh.seg[at] = g;
  mbar_arrive(&sh.seg_full[at]);
  entry = g.n ? entry + 1 : -1;
  return true;
}

// Lets the last tiles' loads land: none outlives the block, whether all went well or a wait ran
// out. (A call: inlined, this code moves the tile loops, and two chunks of 2048 take 667 us
// instead of 648.)
template <int DP>
__device__ __noinline__ void att_drain(AttShared<DP>& sh, unsigned issued, unsigned q_issued) {
  using Cfg = AttCfg<DP>;
  for (unsigned r = issued > Cfg::kStages ? issued - Cfg::kStages : 0; r < issued; ++r)
    att_land(&sh.kv_full[r % Cfg::kRing], r / Cfg::kRing);
  for (unsigned x = q_issued > 2 ? q_issued - 2 : 0; x < q_issued; ++x)
    att_land(&sh.q_full[x & 3], x / 4);
}

// ---- warps 8 and 11: Q and K, and V tiles by TMA (two warps: with small pages it is the
// issue of the loads that takes the time). The one for V also does the walk, two entries
// ahead of its loads.

template <int DP, bool V>
__device__ __forceinline__ void att_load(AttShared<DP>& sh, const AttendParams& p, char* q_smem,
                                         char* kv_smem, int lane, AttWalk* walk) {
  using Cfg = AttCfg<DP>;
  constexpr int kBlocks = DP / 64, kBlockBytes = kAttTile * 128;
  const int page = 1 << p.page_shift;
  const int box = min(page, kAttTile);         // tokens of one load
  const int boxes = kAttTile / box;            // of a tile
  unsigned issued = 0, q_issued = 0, edges = 0;
  int entry = V ? sh.entry : 0;
  auto load_q = [&](const AttSeg& g) {
    for (int s = 0; s <= g.pair; ++s) {
      const int x = g.q_at + s, slot = x & 1;
      if (!att_wait_warp(sh, p, &sh.q_empty[slot], (x / 2 + 1) & 1)) return false;
      if (lane == 0) {
        mbar_arrive_expect_tx(&sh.q_full[x & 3], kBlocks * p.tile_tokens * p.G * 128);
        for (int k = 0; k < kBlocks; ++k)
          tma_load_4d(q_smem + slot * Cfg::kTileBytes + k * kBlockBytes, &p.q_map, 64 * k, 0,
                      g.head, g.token + s * p.tile_tokens, &sh.q_full[x & 3]);
      }
      __syncwarp();
      q_issued = x + 1;
    }
    return true;
  };
  for (int e = 0;; ++e) {
    const int at = e % kAttSegs;
    if (!att_wait_warp(sh, p, &sh.seg_full[at], e / kAttSegs)) break;
    const AttSeg g = sh.seg[at];
    if (g.n == 0) break;
    bool ok = true;
    const int* table = p.table + g.b * p.table_stride;
    const int sinks = min(p.sinks, g.lo);
    // The lane's first token of tile i, and the number of its page (-1: no row sees it).
    auto place = [&](int i) { return att_tile(g, i) * kAttTile + lane * box; };
    auto page_of = [&](int j) {
      const bool seen = lane < boxes && j < g.hi && (j + box > g.lo || j < sinks);
      // (an ordinary load: the kernel before this one may still be writing the table when this
      // one starts, which loads through the read-only path do not allow)
      return seen ? table[j >> p.page_shift] : -1;
    };
    int number = page_of(place(0));
    // Q of the first segment while that comes; later ones' after their first tile, which need
    // not wait for Q's place
    if (!V && e == 0) ok = load_q(g);
    for (int i = 0; ok && i < g.n; ++i) {
      const int j = place(i), j0 = j - lane * box, this_page = number;
      // the next tile's pages, read while this one is loaded
      if (i + 1 < g.n) number = page_of(place(i + 1));
      const bool live = this_page >= 0 && this_page < p.num_pages;
      if (__builtin_expect(!live && lane < boxes && j < g.hi && (j + box > g.lo || j < sinks), 0))
        atomicOr(p.status, SPEC_CACHE_BAD_PAGE);
      const int count = __popc(__ballot_sync(~0u, live));
      const unsigned r = g.ring + (V ? att_v_at(g.pair, i, g.n) : att_k_at(g.pair, i));
      char* tile = kv_smem + (r % Cfg::kStages) * Cfg::kTileBytes;
      uint64_t* full = &sh.kv_full[r % Cfg::kRing];
      if (r >= Cfg::kStages) {  // what the tile's place held has been used
        const unsigned x = r - Cfg::kStages;
        ok = att_wait_warp(sh, p, &sh.kv_empty[x % Cfg::kRing], x / Cfg::kRing);
        if (!ok) break;
      }
      const bool clear = V && j0 + kAttTile > sinks && !(j0 >= g.lo && j0 + kAttTile <= g.hi);
      uint64_t* landed = clear ? &sh.edge_full : full;
      if (lane == 0) mbar_arrive_expect_tx(landed, count * kBlocks * box * 128);
      __syncwarp();
      if (live) {
        char* dst = tile + lane * box * 128;
        for (int k = 0; k < kBlocks; ++k)
          tma_load_4d(dst + k * kBlockBytes, V ? &p.v_map : &p.k_map, 64 * k, j & (page - 1),
                      g.head, this_page, landed);
      }
      __syncwarp();
      issued = r + 1;
      if (V) {
        // the list's next entry, in the shadow of this load; and the second one at the start
        if (__builtin_expect(i == g.n - 1 || (e == 0 && i == 0), 0)) {
          for (int x = (i == g.n - 1) + (e == 0 && i == 0); x > 0; --x)
            if (lane == 0) att_publish(*walk, entry, sh, p);
          __syncwarp();
        }
        if (__builtin_expect(clear, 0)) {
          // V's rows that no row of the unit sees may hold anything, and P is 0 there: they are
          // zeroed before the tile counts as loaded.
          ok = att_wait_warp(sh, p, &sh.edge_full, edges);
          if (!ok) {
            att_land(&sh.edge_full, edges);
            break;
          }
          ++edges;
#pragma unroll 1
          for (int y = lane; y < kAttTile * kBlocks; y += 32) {
            const int j = j0 + (y & (kAttTile - 1));
            if (j < sinks || (j >= g.lo && j < g.hi)) continue;
#pragma unroll
            for (int x = 0; x < 8; ++x)
              *(uint4*)(tile + y * 128 + 16 * x) = make_uint4(0, 0, 0, 0);
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(full);
        }
      } else if (__builtin_expect(i == 0 && e > 0, 0)) {
        ok = load_q(g);
      }
    }
    if (!ok) break;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.seg_empty[at]);
  }
  att_drain<DP>(sh, issued, q_issued);
}

// ---- warps 9 and 10: the products of stream 0 and 1, issued by one thread of each.
// A thread that issues is held until the tensor cores have all but caught up, so a warp for
// each stream does its waiting for P, K and V while the other's products run. They take
// turns (PV of a tile and QK of the stream's next), which keeps the streams half a period
// apart: left to themselves they fall into step, and the tensor cores idle through both
// softmaxes. A commit is dear, so there is one for each tile: S of tile i tells that K of
// tile i and V of the stream's tile before have been used too.

// A tile of K or V is free after both streams' products, or twice after the one's.
template <int DP>
__device__ __forceinline__ void att_release(AttShared<DP>& sh, unsigned r, bool pair) {
  mbar_arrive(&sh.kv_empty[r % AttCfg<DP>::kRing]);
  if (!pair) mbar_arrive(&sh.kv_empty[r % AttCfg<DP>::kRing]);
}

template <int DP, bool BF16>
__device__ __forceinline__ void att_products(AttShared<DP>& sh, const AttendParams& p,
                                             char* q_smem, char* kv_smem, const int s) {
  using Cfg = AttCfg<DP>;
  constexpr uint32_t kQK = mma_kind(BF16, false, kAttTile, kAttTile);
  // Head sizes between the tiles' have fewer steps in QK and fewer columns in PV.
  const uint32_t kind_pv = mma_kind(BF16, true, kAttTile, (p.dim + 15) / 16 * 16);
  const int steps = (p.dim + 15) / 16;
  const uint32_t tmem_s = __shfl_sync(~0u, sh.tmem, 0) + s * 128, tmem_o = tmem_s + 256;
  const bool one = elect_one();
  // descriptors of the first tiles; others by what is added to their addresses (in 16 bytes)
  const uint64_t q0 = mma_desc(smem_addr(q_smem), 16), k0 = mma_desc(smem_addr(kv_smem), 16);
  const uint64_t v0 = mma_desc(smem_addr(kv_smem), kAttTile * 128);
  constexpr unsigned kTile = Cfg::kTileBytes / 16;
  unsigned p_count = 0, turn = 0;
  if (!att_wait_warp(sh, p, &sh.warm, 0)) return;  // the softmax warps' dry run
  auto loaded = [&](unsigned r) {
    return att_wait_warp(sh, p, &sh.kv_full[r % Cfg::kRing], r / Cfg::kRing);
  };
  for (int e = 0;; ++e) {
    const int at = e % kAttSegs;
    if (!att_wait_warp(sh, p, &sh.seg_full[at], e / kAttSegs)) return;
    const int n = __shfl_sync(~0u, sh.seg[at].n, 0);
    if (n == 0) return;
    const bool pair = __shfl_sync(~0u, sh.seg[at].pair, 0);
    const int q_at = __shfl_sync(~0u, sh.seg[at].q_at, 0) + (pair ? s : 0);
    const unsigned ring = __shfl_sync(~0u, sh.seg[at].ring, 0);
    if (!att_wait_warp(sh, p, &sh.q_full[q_at & 3], q_at / 4)) return;
    const int step = pair ? 1 : 2, first = pair ? 0 : s;
    // The same number of turns for both streams, whether they have a tile for it or not.
    const int turns = pair ? n + 1 : (n + 3) / 2;
#pragma unroll 1
    for (int t = 0; t < turns; ++t) {
      const int next = first + t * step, last = next - step;  // QK of the one, PV of the other
      const unsigned k = ring + att_k_at(pair, next), v = ring + att_v_at(pair, last, n);
      const bool has_pv = t > 0 && last < n, has_qk = next < n;
      // the results of the segment before (e > 0) have been read by all
      if (t == 1 && !att_wait_warp(sh, p, &sh.o_free, e + 1)) return;
      if (has_pv) {
        // S of the turn before is there: what its products read is free (and the loads below
        // may be waiting for that)
        if (!att_wait_warp(sh, p, &sh.s_full[s], p_count)) return;
        if (one) {
          att_release<DP>(sh, ring + att_k_at(pair, last), pair);
          if (t > 1) att_release<DP>(sh, ring + att_v_at(pair, last - step, n), pair);
        }
        __syncwarp();
      }
      if (has_qk && !loaded(k)) return;
      if (has_pv && (!loaded(v) || !att_wait_warp(sh, p, &sh.p_half[s], p_count))) return;
      if (!att_wait_warp(sh, p, &sh.turn[s], turn + 1 - s)) return;
      ++turn;
      tmem_fence_after();
      if (has_pv) {
        const uint64_t vd = v0 + (v % Cfg::kStages) * kTile;
#pragma unroll
        for (int x = 0; x < kAttTile / 16; ++x) {
          if (x == kAttTile / 32) {  // half of P at a time, as it comes
            if (!att_wait_warp(sh, p, &sh.p_full[s], p_count)) return;
            tmem_fence_after();
          }
          mma_ts(tmem_o, tmem_s + 8 * x, vd + x * (16 * 128 / 16), kind_pv, t > 1 || x > 0,
                 one);
        }
        ++p_count;
      }
      if (has_qk) {
        const uint64_t qd = q0 + (q_at & 1) * kTile, kd = k0 + (k % Cfg::kStages) * kTile;
#pragma unroll
        for (int x = 0; x < DP / 16; ++x) {
          const unsigned y = ((x / 4) * (kAttTile * 128) + (x % 4) * 32) / 16;
          if (x < steps) mma_ss(tmem_s, qd + y, kd + y, kQK, x > 0, one);
        }
      }
      if (one) mbar_arrive(&sh.turn[s ^ 1]);
      if (has_qk) mma_commit(&sh.s_full[s], one);
      __syncwarp();
    }
    // The stream's last V, and Q: read by both streams, or each stream's own.
    if (first < n) {
      const int last = first + (n - 1 - first) / step * step;
      const unsigned v = ring + att_v_at(pair, last, n);
      for (int x = 0; x <= !pair; ++x) mma_commit(&sh.kv_empty[v % Cfg::kRing], one);
    }
    for (int x = 0; x <= pair; ++x) mma_commit(&sh.q_empty[q_at & 1], one);
    mma_commit(&sh.o_full, one);
    if (one) mbar_arrive(&sh.seg_empty[at]);
    __syncwarp();
  }
}

// ---- warps 0-7: softmax, rescaling, results

// Overwrite the scores that the row at `pos` does not see, 32 columns at a time
// in a rolled loop: edge tiles are few, and the code of the others stays short.
__device__ __forceinline__ void att_hide(uint32_t tmem_s, int pos, int j0, int window, int sinks,
                                      float hidden) {
  const int end = min(pos - j0 + 1, kAttTile);
  const int from = window && pos >= window ? pos - window + 1 - j0 : -j0;
  const int sink_end = sinks - j0;
#pragma unroll 1
  for (int k = 0; k < kAttTile; k += 32) {
    // columns [0, sink_end) and [from, end) of these 32, as bits
    auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; };
    const uint32_t seen = below(end - k) & (~below(from - k) | below(sink_end - k));
    if (__all_sync(~0u, seen == ~0u)) continue;
    float x[32];
    tmem_ld32(tmem_s + k, x);
    tmem_wait_ld(x);
#pragma unroll
    for (int y = 0; y < 32; ++y)
      if (!(seen >> y & 1)) x[y] = hidden;
    tmem_st32(tmem_s + k, x);
  }
  tmem_wait_st();
}

template <int DP>
__device__ __forceinline__ void att_rescale(uint32_t tmem_o, float keep) {
#pragma unroll 1
  for (int k = 0; k < DP; k += 32) {
    float o[32];
    tmem_ld32(tmem_o + k, o);
    tmem_wait_ld(o);
#pragma unroll
    for (int y = 0; y < 32; ++y) o[y] *= keep;
    tmem_st32(tmem_o + k, o);
  }
}

// The largest of 64 values and x (the least, where the scores' factor is negative).
__device__ __forceinline__ float att_max64(const float* f, bool largest, float x) {
  float top[4] = {x, f[1], f[2], f[3]};
  if (__builtin_expect(largest, 1)) {
    top[0] = fmaxf(top[0], f[0]);
#pragma unroll
    for (int y = 4; y < 60; y += 8)
#pragma unroll
      for (int z = 0; z < 4; ++z) top[z] = max3(top[z], f[y + z], f[y + z + 4]);
#pragma unroll
    for (int z = 0; z < 4; ++z) top[z] = fmaxf(top[z], f[60 + z]);
    return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
  }
  top[0] = fminf(top[0], f[0]);
#pragma unroll
  for (int y = 4; y < 64; ++y) top[y & 3] = fminf(top[y & 3], f[y]);
  return fminf(fminf(top[0], top[1]), fminf(top[2], top[3]));
}

// log2 of what every P and l carries beside 2^-m: fp16 has few exponents below 1.
template <bool BF16>
__device__ constexpr float att_bias() {
  return BF16 ? 0.f : 7.f;
}
template <bool BF16>
__device__ __forceinline__ float att_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l) - att_bias<BF16>()) * 0.69314718055994531f;
}

template <int DP, bool BF16>
__device__ __forceinline__ void att_softmax(AttBase& sh, const AttendParams& p, int warp, int lane) {
  constexpr float kBias = att_bias<BF16>();
  const int s = warp >> 2, row = (warp & 3) * 32 + lane;
  const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
  const uint32_t tmem_s = sh.tmem + lanes + s * 128;
  const uint32_t tmem_o = sh.tmem + lanes + 256;
  const int row_token = row / p.G, row_head = row - row_token * p.G;
  unsigned s_count = 0, joins = 0;
  // The walk's entries, after one round that only brings the code near: its instructions come
  // from L2 the first time, which takes as long as the list's head and the first loads do. It
  // works on whatever TMEM holds, sees no row, and neither waits nor tells anyone.
  for (int e = -1;; ++e) {
    const bool dry = e < 0;
    const int at = e & (kAttSegs - 1);
    AttSeg g = {2, 0, 0, 0, 0, p.tile_tokens, 0, 0, 1, 0x7fffffff, 0, 0, 0, 0, -1};
    if (!dry) {
      if (!att_wait_warp(sh, p, &sh.seg_full[at], e / kAttSegs)) return;
      g = sh.seg[at];
      if (g.n == 0) return;
    }
    // This thread's row: token and position; rows past the unit's tokens see nothing.
    const int tile0 = g.pair ? s * p.tile_tokens : 0;  // the stream's first token
    const int tokens = min(p.tile_tokens, g.tokens - tile0);
    const bool mine = row_token < tokens && !dry;
    const int pos = mine ? g.pos + tile0 + row_token : -1;
    const bool busy = (warp & 3) * 32 < tokens * p.G;  // rows in this warp
    const int first_pos = g.pos + tile0, last_pos = g.pos + tile0 + tokens - 1;
    float m = -INFINITY, l = 0.f;
    const int step = g.pair ? 1 : 2;
    for (int i = g.pair ? 0 : s; i < g.n; i += step) {
      // what can be known before S is there
      const int j0 = att_tile(g, i) * kAttTile;
      const bool all_seen = j0 + kAttTile - 1 <= first_pos &&
                            (!p.window || j0 > last_pos - p.window || j0 + kAttTile <= p.sinks);
      if (!dry && !att_wait_warp(sh, p, &sh.s_full[s], s_count++)) return;
      if (busy) {
        tmem_fence_after();
        if (__builtin_expect(!all_seen, 0)) att_hide(tmem_s, pos, j0, p.window, p.sinks, p.hidden);
        float f[64], top;
        {
          float x[64];
          tmem_ld32(tmem_s + 64, x);
          tmem_ld32(tmem_s + 96, x + 32);
          tmem_wait_ld(x);
          tmem_wait_ld(x + 32);
          tmem_ld32(tmem_s, f);
          tmem_ld32(tmem_s + 32, f + 32);
          top = att_max64(x, p.c > 0.f, p.hidden);
        }
        tmem_wait_ld(f);
        tmem_wait_ld(f + 32);
        top = att_max64(f, p.c > 0.f, top) * p.c;
        const bool grown = mine && top > m + kAttGrow;
        if (__builtin_expect(__any_sync(~0u, grown), 0)) {
          const float keep = grown ? ex2(m - top) : 1.f;
          l *= keep;
          if (grown) m = top;
          if (i >= step) att_rescale<DP>(tmem_o + s * 128, keep);  // O holds earlier tiles
        }
        const float shift = kBias - (m == -INFINITY ? 0.f : m);
        const unsigned long long c2 = f2_pack(p.c, p.c), shift2 = f2_pack(shift, shift);
        unsigned long long sum2[2] = {0, 0};
        // P over S, half a tile at a time in a rolled loop: the warps of a block run through
        // more code than the SM's instruction cache holds, and every line less counts.
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          uint32_t w[32];
#pragma unroll
          for (int y = 0; y < 32; ++y) {
            float a, b;
            f2_unpack(f2_fma(f2_pack(f[2 * y], f[2 * y + 1]), c2, shift2), a, b);
            a = ex2(a);
            b = ex2(b);
            sum2[y & 1] = f2_add(sum2[y & 1], f2_pack(a, b));
            w[y] = pack2<BF16>(a, b);
          }
          tmem_st32(tmem_s + 32 * k, w);
          tmem_wait_st();
          tmem_fence_before();
          __syncwarp();
          if (lane == 0 && !dry) mbar_arrive(k ? &sh.p_full[s] : &sh.p_half[s]);
          if (k == 0) {
            tmem_ld32(tmem_s + 64, f);
            tmem_ld32(tmem_s + 96, f + 32);
            tmem_wait_ld(f);
            tmem_wait_ld(f + 32);
          }
        }
        float a, b;
        f2_unpack(f2_add(sum2[0], sum2[1]), a, b);
        l += a + b;
      } else if (lane == 0 && !dry) {
        mbar_arrive(&sh.p_half[s]);
        mbar_arrive(&sh.p_full[s]);
      }
      __syncwarp();
    }
    // ---- results of the segment
    float w[2] = {1.f, 1.f};  // of the two streams' O
    if (!g.pair) {
      // ml of the segment before has been read by all
      if (!dry && !att_wait_warp(sh, p, &sh.o_free, e + 1)) return;
      sh.ml[s][row] = make_float2(m, l);
      __syncwarp();
      if (lane == 0 && !dry) mbar_arrive(&sh.ml_full);
      if (!dry && !att_wait_warp(sh, p, &sh.ml_full, joins++)) return;
      const float2 x = sh.ml[0][row], y = sh.ml[1][row];
      m = fmaxf(x.x, y.x);
      w[0] = x.x == -INFINITY ? 0.f : ex2(x.x - m);
      w[1] = y.x == -INFINITY ? 0.f : ex2(y.x - m);
      l = x.y * w[0] + y.y * w[1];
    }
    if (!dry && !att_wait_warp(sh, p, &sh.o_full, e)) return;
    if (busy) {
      tmem_fence_after();
      const int half = g.pair ? DP : DP / 2;  // columns of this warp: stream s of a pair, or
      const int col0 = g.pair ? 0 : s * half;  // half the columns of both streams
      const uint32_t first = tmem_o + (g.pair ? s * 128 : 0);
      const bool both = !g.pair && g.n > 1;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const long long token = g.token + tile0 + row_token;
      const int head = g.head * p.G + row_head;
      const int part = ((blockIdx.x * 2 + max(g.slot, 0)) * 2 + (g.pair ? s : 0));
      char* out = p.out + token * p.out_token + head * p.out_head;
      float4* part_o = p.part_o + (size_t)part * (DP / 4) * kAttTile + row;
#pragma unroll 1
      for (int k = 0; k < half; k += 16) {  // short code: it is cold every time it runs
        float o[16];
        tmem_ld16(first + col0 + k, o);
#pragma unroll
        for (int z = 0; z < 16; ++z) o[z] *= w[0];
        if (both) {
          float y[16];
          tmem_ld16(first + 128 + col0 + k, y);
#pragma unroll
          for (int z = 0; z < 16; ++z) o[z] += y[z] * w[1];
        }
        if (mine && g.slot >= 0) {
#pragma unroll
          for (int z = 0; z < 4; ++z)
            part_o[((col0 + k) / 4 + z) * kAttTile] =
                make_float4(o[4 * z], o[4 * z + 1], o[4 * z + 2], o[4 * z + 3]);
        } else if (mine) {
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            if (col0 + k + 8 * z >= p.dim) break;
            uint4 v;
            v.x = pack2<BF16>(o[8 * z] * inv, o[8 * z + 1] * inv);
            v.y = pack2<BF16>(o[8 * z + 2] * inv, o[8 * z + 3] * inv);
            v.z = pack2<BF16>(o[8 * z + 4] * inv, o[8 * z + 5] * inv);
            v.w = pack2<BF16>(o[8 * z + 6] * inv, o[8 * z + 7] * inv);
            *(uint4*)(out + (col0 + k + 8 * z) * 2) = v;
          }
        }
        __syncwarp();
      }
      if (mine && (g.pair || s == 0)) {
        if (g.slot >= 0)
          p.part_ml[part * kAttTile + row] = make_float2(m, l);
        else if (p.lse)
          p.lse[token * p.heads + head] = att_lse<BF16>(m, l);
      }
    }
    tmem_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(dry ? &sh.warm : &sh.o_free);
    if (lane == 0 && !dry) mbar_arrive(&sh.seg_empty[at]);
    if (dry) pdl_wait();
  }
}

// ---- the kernels

template <int DP, bool BF16>
__global__ void __launch_bounds__(kAttThreads, 1)
    k_attend(const __grid_constant__ AttendParams p, const int run) {
  using Cfg = AttCfg<DP>;
  extern __shared__ __align__(1024) char smem[];
  char* q_smem = smem;
  char* kv_smem = smem + 2 * Cfg::kTileBytes;
  AttShared<DP>& sh = *reinterpret_cast<AttShared<DP>*>(
      kv_smem + Cfg::kStages * Cfg::kTileBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 0) {
    for (int i = lane; i < Cfg::kRing; i += 32) {
      mbar_init(&sh.kv_full[i], 1);
      mbar_init(&sh.kv_empty[i], 2);
    }
    if (lane < 4) {
      mbar_init(&sh.q_full[lane], 1);
      mbar_init(&sh.seg_full[lane], 1);
      mbar_init(&sh.seg_empty[lane], 12);
    }
    if (lane < 2) {
      mbar_init(&sh.q_empty[lane], 2);
      mbar_init(&sh.s_full[lane], 1);
      mbar_init(&sh.p_half[lane], 4);
      mbar_init(&sh.p_full[lane], 4);
      mbar_init(&sh.turn[lane], 1);
      mbar_init(&sh.drain[lane], 1);
    }
    if (lane == 0) {
      mbar_init(&sh.warm, 8);
      mbar_init(&sh.o_full, 2);
      mbar_init(&sh.o_free, 8);
      mbar_init(&sh.ml_full, 8);
      mbar_init(&sh.edge_full, 1);
      sh.stop = sh.gaps = 0;
    }
    fence_mbar_init();
  } else if (tid == 32) {
    prefetch_map(&p.q_map);
    prefetch_map(&p.k_map);
    prefetch_map(&p.v_map);
  }
  if (warp == 9) tmem_alloc(&sh.tmem, 512);
  pdl_trigger();
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp < 8) {
    regs_take<kAttRegsMany>();
    att_softmax<DP, BF16>(sh, p, warp, lane);
  } else {
    regs_give<kAttRegsFew>();
    pdl_wait();
    // Key tiles of each thread's run of requests, and of all.
    const int t = tid - (kAttThreads - kAttScan), w0 = t >> 5, step = 2 * p.tile_tokens;
    const int r0 = (int)min((long long)t * run, (long long)p.B), r1 = min(r0 + run, p.B);
    int lo = 0, hi = 0, len = 0;  // of the request read last
    auto tiles_of = [&](int r) {
      len = p.request(r, lo, hi);
      const AttUnits units(len, hi - lo, step, p.window, p.sinks);
      return units.before(units.count) * p.kv_heads;
    };
    long long mine = 0;
    int pad = 0;  // rows from here on belong to no request
    for (int r = r0; r < r1; ++r) {
      mine += tiles_of(r);
      pad = max(pad, hi);
      if (lo < 0 || (r == 0 && lo > 0)) sh.gaps = 1;
    }
    long long upto = mine;
    for (int d = 1; d < 32; d <<= 1) {
      const long long x = __shfl_up_sync(~0u, upto, d);
      if (lane >= d) upto += x;
    }
    pad = __reduce_max_sync(~0u, pad);
    if (lane == 31) sh.scan[w0] = upto;
    if (lane == 0) sh.pad[w0] = pad;
    named_sync(1, kAttScan);
    long long all = 0, before = upto - mine;
    for (int w = 0; w < kAttScan / 32; ++w) {
      if (w < w0) before += sh.scan[w];
      all += sh.scan[w];
      pad = max(pad, sh.pad[w]);
    }
    long long total = all;
    if (total > kAttMostPart * gridDim.x) {  // too much for one call: all rows see nothing
      if (t == 0 && blockIdx.x == 0) atomicOr(p.status, SPEC_CACHE_BAD_LENGTHS);
      total = pad = 0;
    }
    const int blocks = (int)min((long long)gridDim.x, total);
    const bool works = (int)blockIdx.x < blocks;
    const AttPart part(blockIdx.x, total, max(blocks, 1));
    if (t == 0) {
      p.join[blockIdx.x].last = -1;
      sh.pad_all = pad;
      if (!works) {
        sh.seg[0].n = 0;
        mbar_arrive(&sh.seg_full[0]);
      }
    }
    __syncwarp();
    if (works && before <= part.begin && part.begin < before + mine) {
      long long at = before;
      int r = r0;
      if (run > 1) {
        for (;; ++r) {
          const long long n = tiles_of(r);
          if (part.begin < at + n || r + 1 >= r1) break;
          at += n;
        }
      }
      AttWalk walk(p, part, blockIdx.x, r, at, lo, hi, len);
      int entry = 0;
      att_publish(walk, entry, sh, p);
      sh.walk = walk;
      sh.entry = entry;
    }
    named_sync(1, kAttScan);
    if (works && warp == 8) {
      att_load<DP, false>(sh, p, q_smem, kv_smem, lane, nullptr);
    } else if (works && warp == 11) {
      AttWalk walk = sh.walk;
      att_load<DP, true>(sh, p, q_smem, kv_smem, lane, &walk);
    } else if (works) {
      const int s = warp - 9;
      att_products<DP, BF16>(sh, p, q_smem, kv_smem, s);
      mma_commit(&sh.drain[s], elect_one());  // no product outlives the block either
      att_land(&sh.drain[s], 0);
    }
    __syncwarp();
  }
  tmem_fence_before();
  __syncthreads();
  if (warp == 9) {
    tmem_fence_after();
    tmem_free(sh.tmem, 512);
  }
  // Rows of q that belong to no request: zeros. Those past the last one as a rule; where the
  // offsets do not start at 0 or cannot be, a row is looked for in all requests.
  const int pad_all = sh.pad_all;
  const bool gaps = sh.gaps;
#pragma unroll 1
  for (long long t = (gaps ? 0 : pad_all) + blockIdx.x; t < p.T; t += gridDim.x) {
    if (t < pad_all) {
      bool mine = false;
#pragma unroll 1
      for (int b = tid; b < p.B; b += kAttThreads) {
        const int lo = p.cu_q[b], hi = p.cu_q[b + 1];
        mine |= lo >= 0 && lo <= t && t < hi && hi <= p.T;
      }
      if (__syncthreads_or(mine)) continue;
    }
    const int pieces = p.dim / 8;
    for (int i = tid; i < p.heads * pieces; i += kAttThreads)
      *(uint4*)(p.out + t * p.out_token + (i / pieces) * p.out_head + (i % pieces) * 16) =
          make_uint4(0, 0, 0, 0);
    if (p.lse)
      for (int i = tid; i < p.heads; i += kAttThreads) p.lse[t * p.heads + i] = -INFINITY;
  }
}

constexpr int kJoinThreads = 512;

// Join the partial results of the unit that starts in block blockIdx.x's part
// of the list and ends in another's: parts of one row weigh 2^(m - max m). An
// item is four columns of a row; where the items are fewer than the threads,
// up to 32 lanes take an item's parts in turn and add up.
template <int DP, bool BF16>
__global__ void __launch_bounds__(kJoinThreads) k_attend_join(const AttendParams p) {
  pdl_trigger();
  pdl_wait();
  const AttJoin j = p.join[blockIdx.x];
  if (j.last < 0) return;
  const int parts = j.last - blockIdx.x + 1;
  const int cols = DP / 4 / gridDim.y;  // groups of four columns of this block
  const int rows0 = min(p.tile_tokens, j.tokens) * p.G, rows = j.tokens * p.G;
  int lanes = 1;  // of an item
  while (lanes < 32 && lanes < parts && rows * cols * lanes * 2 <= kJoinThreads) lanes *= 2;
  const int mine = threadIdx.x & (lanes - 1);
  // whole warps go round together: the sums below take all their lanes
  for (int x0 = 0; x0 < rows * cols; x0 += kJoinThreads / lanes) {
    const int x = x0 + threadIdx.x / lanes;
    const bool real = x < rows * cols;
    const int col4 = real ? x / rows : 0, any_row = real ? x - col4 * rows : 0;
    const int tile = any_row >= rows0, row = any_row - tile * rows0;
    const int c4 = blockIdx.y * cols + col4;
    auto at = [&](int i) { return ((blockIdx.x + i) * 2 + (i == 0)) * 2 + tile; };
    float m = -INFINITY;
#pragma unroll 4
    for (int i = mine; i < parts; i += lanes) m = fmaxf(m, p.part_ml[at(i) * kAttTile + row].x);
    for (int d = 1; d < lanes; d <<= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = mine; i < parts; i += lanes) {
      const float2 ml = p.part_ml[at(i) * kAttTile + row];
      const float4 y = p.part_o[((size_t)at(i) * (DP / 4) + c4) * kAttTile + row];
      const float w = ml.x == -INFINITY ? 0.f : ex2(ml.x - m);
      l += w * ml.y;
      o.x += w * y.x;
      o.y += w * y.y;
      o.z += w * y.z;
      o.w += w * y.w;
    }
    for (int d = 1; d < lanes; d <<= 1) {
      l += __shfl_xor_sync(~0u, l, d);
      o.x += __shfl_xor_sync(~0u, o.x, d);
      o.y += __shfl_xor_sync(~0u, o.y, d);
      o.z += __shfl_xor_sync(~0u, o.z, d);
      o.w += __shfl_xor_sync(~0u, o.w, d);
    }
    if (!real || mine) continue;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int row_token = any_row / p.G;
    const long long token = j.token + row_token;
    const int head = j.head * p.G + (any_row - row_token * p.G);
    if (4 * c4 < p.dim) {
      uint2 v;
      v.x = pack2<BF16>(o.x * inv, o.y * inv);
      v.y = pack2<BF16>(o.z * inv, o.w * inv);
      *(uint2*)(p.out + token * p.out_token + head * p.out_head + 8 * c4) = v;
    }
    if (c4 == 0 && p.lse) p.lse[token * p.heads + head] = att_lse<BF16>(m, l);
  }
}

}  // namespace sv
