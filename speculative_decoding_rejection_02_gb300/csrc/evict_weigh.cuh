// The softmax weights that the new tokens give the cached ones (spec_cache_weigh).
//
//   w_j = (old ? decay w_j : 0) + sum over columns 2^(c q . k_j - lse log2(e)),  c = scale log2(e)
//
// where a column is a new token and one of its query heads on the kv head. With the keys as rows,
//
//   S^T = K Q^T     tcgen05, 128 keys x up to 128 columns, K and Q in shared memory, S in TMEM
//   w += row sums   one thread per key: it reads its row of S, and its sum never leaves it
//
// so a sum needs no other thread and no other key, and there is nothing to join; sums are fp32.
// A pair of key tiles goes over the request's column tiles together, so that a tile of Q is loaded
// for 256 keys: with 128 the loads alone would take what an SM gets from L2. Each key tile has two
// groups of four warps with a place in TMEM each, which take its column tiles in turns; at the end
// of the pair one passes its sums to the other. (One group with both places: 421 us for two chunks
// of 2048 over 11000-14000 where two groups took 391: two warps for each scheduler do not cover the
// latency of what they do.)
//
// The pairs of all requests and kv heads stand in one list, in which a pair counts by the column
// tiles that see it and three more for its start, cut into equal parts, one for each block (one
// block per SM). Every role of a block walks over the part by itself. (Four prompts of 1000-1500
// tokens 55 us; 82 with all of the request's column tiles counted for every pair and the tiles of
// the diagonal looked at column by column.)
//
// Warps: 0-7 and 8-15 the sums of the pair's two tiles, 16 loads K (TMA, through the block table),
// 17 loads Q and the lse, and where those come once for many pairs half of K (with small pages it
// is the issue of the loads that takes the time: 49 single tokens over 38000 in pages of 8 or 16
// 607 us in place of 668), 18 and 19 issue the products of the one and the other tile. (A
// second issuer took two chunks of 2048 over 11000-14000 from 540 us to 409: it is the issue of a
// product that takes its time, not the product.) The two tiles' chains go ahead of one another, so
// each has its own stages of K.
//
// Bound by HBM (the keys, once) for few columns, by the chain of products for many: 64 requests of
// 2-8 tokens over 1000-30000 186 us (0.93 of a copy's rate), two chunks of 2048 over 11000-14000
// 354 us (0.66 of a large library product's rate; 331 in runs of some milliseconds, of which 296 are
// left with no exponential computed).
#pragma once
#include <cuda.h>

#include "sparse_common.cuh"
#include "tcgen05.cuh"

namespace sv {

constexpr int kWeighSums = 16, kWeighThreads = (kWeighSums + 4) * 32, kWeighScan = 128;
constexpr int kWeighTile = 128;
constexpr int kWeighRing = 12;      // stages at most
constexpr int kWeighSmem = 204 * 1024, kWeighStages = 192 * 1024;
constexpr int kWeighShifts = 8;     // column tiles whose lse are ahead
constexpr int kWeighStart = 3;      // what a pair counts beside its column tiles
constexpr long long kWeighPatience = 2000000000;  // clocks that a wait may take

struct WeighParams {
  CUtensorMap q_map, k_map;
  Requests rq;
  int heads, kv_heads, G, dim;
  const float* lse;
  float* weights;
  long long w_page, w_head;  // elements
  float c, decay;
  int bf16;
  int tile_tokens;          // new tokens of a column tile
  int late_tiles;           // of those, how many fewer see a pair of keys than the one before
  int blocks;               // of 64 channels
  int k_stages, q_stages;   // of blocks * 16 KB; of K for each of a pair's two tiles
  int shared_loads;         // the warp that loads Q loads half of K
};

struct WeighShared {
  uint64_t k_full[kWeighRing], k_empty[kWeighRing], q_full[kWeighRing], q_empty[kWeighRing];
  uint64_t s_full[2][2], s_free[2][2], joined[2], drain[2];
  uint64_t l_full[kWeighShifts], l_empty[kWeighShifts];
  alignas(16) float shift[kWeighShifts][kWeighTile];  // of a column tile: -lse log2(e)
  // Sums on their way from one group of a tile to the other, of two pairs in turn.
  float part[2][2][kWeighTile];
  int pages[kWeighRing][16];  // of a tile of keys; -1: none
  long long sums[kWeighScan / 32];
  long long at, begin, end;  // of the request that the part starts in, and of the part
  int first;
  uint32_t tmem;
  int stop;
};
static_assert(sizeof(WeighShared) <= kWeighSmem - kWeighStages, "shared memory beside the tiles");

// MUTE, test only (SPEC_CACHE_TEST_WAIT_TIMEOUT): no column tile's lse is ever said to be there, and
// waits are short. (A kernel of its own: with both as parameters the others take 0.5 % longer.)
template <bool MUTE>
struct WeighRun : WeighShared {
  static constexpr long long kPatience = MUTE ? 200000 : kWeighPatience;
};

// A bounded wait of a whole warp (about a second), with one answer for all its lanes; once one
// has run out every later one that would wait returns at once.
template <typename S>
__device__ __forceinline__ bool weigh_wait(S& sh, const WeighParams& p, uint64_t* bar,
                                           uint32_t parity) {
  bool there = mbar_poll(bar, parity & 1);
  if (__builtin_expect(!there, 0)) {
    const long long from = clock64();
    do {
      there = mbar_poll(bar, parity & 1);
    } while (!there && !*(volatile int*)&sh.stop && clock64() - from < S::kPatience);
    if (!there) {
      *(volatile int*)&sh.stop = 1;
      atomicOr(p.rq.status, SPEC_STATUS_TIMEOUT);
    }
  }
  return __all_sync(~0u, there);
}

// The wait for what is in flight when a warp ends, 20 ms at most.
__device__ __forceinline__ void weigh_land(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < 1024; ++i)
    if (mbar_try(bar, parity & 1)) break;
}

// Pairs of key tiles of a request and kv head, and what each counts.
struct WeighUnit {
  int lo, tokens, len, pairs, tiles;  // (of column tiles)
  __device__ __forceinline__ WeighUnit() {}
  __device__ __forceinline__ WeighUnit(const WeighParams& p, int b) {
    lo = p.rq.cu_q[b];
    len = p.rq.kv_lens[b];
    const int hi = p.rq.cu_q[b + 1];
    const bool bad = lo < 0 || hi < lo || hi > p.rq.T || len < 0 ||
                     len > ((long long)p.rq.width << p.rq.page_shift) || len > 0x7fff0000;
    tokens = hi - lo;
    if (bad) {
      atomicOr(p.rq.status, SPEC_CACHE_BAD_LENGTHS);
      lo = tokens = len = 0;
    }
    tiles = (tokens + p.tile_tokens - 1) / p.tile_tokens;
    pairs = tiles ? (len + 2 * kWeighTile - 1) / (2 * kWeighTile) : 0;
  }
  __device__ __forceinline__ int old() const { return len - tokens; }
  // Pairs before this one that column tiles do not see in full.
  __device__ __forceinline__ int late(int pair) const {
    return max(pair - max(old(), 0) / (2 * kWeighTile) - 1, 0);
  }
  // What the pairs before this one count: each its start, and the column tiles that see it.
  __device__ __forceinline__ long long place(const WeighParams& p, int pair) const {
    const long long m = late(pair);
    return (long long)(kWeighStart + tiles) * pair - p.late_tiles * (m * (m - 1) / 2);
  }
  // The first pair at that place or after it (or the number of pairs).
  __device__ __forceinline__ int find(const WeighParams& p, long long at) const {
    const long long all = quotient(at + kWeighStart + tiles - 1, kWeighStart + tiles);
    int a = (int)min(all, (long long)pairs), b = late(a) ? pairs : a;
    while (a < b) {
      const int c = (a + b) / 2;
      if (place(p, c) < at)
        a = c + 1;
      else
        b = c;
    }
    return a;
  }
};

// A block's walk over its part of the list: pairs whose place is in [begin, end).
struct WeighWalk {
  WeighUnit u;
  int b, head, pair, stop;  // stop: where the unit's pairs or the part's end
  bool fresh;               // the unit's first pair here
  long long left;           // of the part from the next unit on
  __device__ __forceinline__ bool start(const WeighParams& p, const WeighShared& sh) {
    b = sh.first;
    if (b < 0) return false;
    long long at = sh.at;
    u = WeighUnit(p, b);
    head = p.kv_heads;
    pair = 0;
    if (u.pairs) {
      const long long all = u.place(p, u.pairs);
      head = (int)quotient(sh.begin - at, all);
      at += head * all;
      pair = u.find(p, sh.begin - at);
      if (pair == u.pairs) {
        at += all;
        pair = 0;
        ++head;
      }
    }
    left = sh.end - at;
    return settle(p);
  }
  // To the next unit, and its pair.
  __device__ __forceinline__ bool settle(const WeighParams& p) {
    while (head >= p.kv_heads) {
      if (left <= 0 || ++b >= p.rq.B) return false;
      u = WeighUnit(p, b);
      head = u.pairs ? 0 : p.kv_heads;
    }
    const long long all = u.place(p, u.pairs);
    stop = left >= all ? u.pairs : left > 0 ? u.find(p, left) : 0;
    left -= all;
    fresh = true;
    return pair < stop;
  }
  __device__ __forceinline__ bool next(const WeighParams& p) {
    fresh = false;
    if (++pair < stop) return true;
    if (stop < u.pairs) return false;
    pair = 0;
    ++head;
    return settle(p);
  }
  // Whether the pair after this one, if it is in the part, is another unit's or there is none.
  __device__ __forceinline__ bool ends_unit() const { return pair + 1 == stop; }
  // The first column tile that sees a key of the pair.
  __device__ __forceinline__ int first_tile(const WeighParams& p) const {
    return max(pair * 2 * kWeighTile - u.old(), 0) / p.tile_tokens;
  }
  __device__ __forceinline__ bool has(int g) const {
    return (pair * 2 + g) * kWeighTile < u.len;
  }
};

// One warp's loads of K, page by page, of one tile of each pair or of both: the first 16 lanes load
// the one, the others the other. Pages are looked up a pair ahead.
struct WeighKeys {
  int tiles;  // bits: which of a pair's tiles
  int page, box, g, part;
  bool on;
  unsigned issued[2] = {0, 0};
  int next;
  __device__ __forceinline__ WeighKeys(const WeighParams& p, const WeighWalk& walk, int tiles)
      : tiles(tiles) {
    const int lane = threadIdx.x & 31;
    page = 1 << p.rq.page_shift;
    box = min(page, kWeighTile);  // tokens of one load
    g = lane >> 4;
    part = lane & 15;
    on = part < kWeighTile / box && (tiles >> g & 1);
    next = look(p, walk);
  }
  __device__ __forceinline__ int place(const WeighWalk& walk) const {
    return (walk.pair * 2 + g) * kWeighTile + part * box;
  }
  // The number of the page that the lane loads; -1: none.
  __device__ __forceinline__ int look(const WeighParams& p, const WeighWalk& walk) const {
    const int j = place(walk);
    if (!on || j >= walk.u.len) return -1;
    return p.rq.table[walk.b * p.rq.table_stride + (j >> p.rq.page_shift)];
  }
  // The pair's loads; `ahead` is the next one, if there is `more`.
  template <typename S>
  __device__ __forceinline__ bool load(S& sh, const WeighParams& p, char* smem, int stage_bytes,
                                       const WeighWalk& walk, const WeighWalk& ahead, bool more) {
    int number = next;
    if (more) next = look(p, ahead);
    const int j = place(walk);
    if (on && j < walk.u.len && (number < 0 || number >= p.rq.num_pages)) {
      atomicOr(p.rq.status, SPEC_CACHE_BAD_PAGE);
      number = -1;
    }
    const int now = tiles & (walk.has(1) ? 3 : 1);
    const unsigned at0 = issued[0] % p.k_stages, at1 = p.k_stages + issued[1] % p.k_stages;
    if ((now & 1) && !weigh_wait(sh, p, &sh.k_empty[at0], issued[0] / p.k_stages + 1))
      return false;
    if ((now & 2) && !weigh_wait(sh, p, &sh.k_empty[at1], issued[1] / p.k_stages + 1))
      return false;
    const unsigned at = g ? at1 : at0;
    const uint32_t live = __ballot_sync(~0u, number >= 0) & 0xffffu << 16 * g;
    if (now >> g & 1) sh.pages[at][part] = number;
    __syncwarp();
    if (part == 0 && (now >> g & 1))
      mbar_arrive_expect_tx(&sh.k_full[at], __popc(live) * p.blocks * box * 128);
    __syncwarp();
    if (number >= 0)
      for (int x = 0; x < p.blocks; ++x)
        tma_load_4d(smem + at * stage_bytes + x * kWeighTile * 128 + part * box * 128, &p.k_map,
                    64 * x, j & (page - 1), walk.head, number, &sh.k_full[at]);
    __syncwarp();
    issued[0] += now & 1;
    issued[1] += now >> 1;
    return true;
  }
  // Lets the last loads land.
  __device__ __forceinline__ void land(WeighShared& sh, const WeighParams& p) const {
#pragma unroll
    for (int t = 0; t < 2; ++t)
      for (unsigned r = issued[t] > p.k_stages ? issued[t] - p.k_stages : 0; r < issued[t]; ++r)
        weigh_land(&sh.k_full[t * p.k_stages + r % p.k_stages], r / p.k_stages);
  }
};

template <bool MUTE>
__global__ void __launch_bounds__(kWeighThreads, 1)
    k_cache_weigh(const __grid_constant__ WeighParams p, const int run) {
  extern __shared__ __align__(1024) char weigh_smem[];
  char* smem = weigh_smem;
  auto& sh = *reinterpret_cast<WeighRun<MUTE>*>(smem + kWeighStages);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int stage_bytes = p.blocks * kWeighTile * 128;
  char* q_smem = smem + 2 * p.k_stages * stage_bytes;
  if (warp == kWeighSums) {
    if (lane < kWeighRing) {
      mbar_init(&sh.k_full[lane], 1);
      mbar_init(&sh.k_empty[lane], 4);
      mbar_init(&sh.q_full[lane], 1);
      mbar_init(&sh.q_empty[lane], 2);
    }
    if (lane < kWeighShifts) {
      mbar_init(&sh.l_full[lane], 1);
      mbar_init(&sh.l_empty[lane], kWeighSums);
    }
    if (lane < 4) {
      mbar_init(&sh.s_full[lane >> 1][lane & 1], 1);
      mbar_init(&sh.s_free[lane >> 1][lane & 1], 4);
    }
    if (lane < 2) {
      mbar_init(&sh.joined[lane], 8);
      mbar_init(&sh.drain[lane], 1);
    }
    if (lane == 0) {
      sh.stop = 0;
      sh.first = -1;
      prefetch_map(&p.q_map);
      prefetch_map(&p.k_map);
    }
    fence_mbar_init();
  }
  if (warp == kWeighSums + 2) tmem_alloc(&sh.tmem, 512);
  pdl_trigger();
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  pdl_wait();
  // ---- this block's part of the list
  if (tid < kWeighScan) {
    const int r0 = (int)min((long long)tid * run, (long long)p.rq.B), r1 = min(r0 + run, p.rq.B);
    auto places = [&](int r) {
      const WeighUnit u(p, r);
      return u.place(p, u.pairs) * p.kv_heads;
    };
    long long mine = 0;
    for (int r = r0; r < r1; ++r) mine += places(r);
    long long upto = mine;
    for (int d = 1; d < 32; d <<= 1) {
      const long long x = __shfl_up_sync(~0u, upto, d);
      if (lane >= d) upto += x;
    }
    if (lane == 31) sh.sums[warp] = upto;
    named_sync(1, kWeighScan);
    long long before = upto - mine, total = 0;
    for (int w = 0; w < kWeighScan / 32; ++w) {
      if (w < warp) before += sh.sums[w];
      total += sh.sums[w];
    }
    const long long each = quotient(total, gridDim.x), more = total - each * gridDim.x;
    const long long begin = each * blockIdx.x + min((long long)blockIdx.x, more);
    const long long end = begin + each + ((long long)blockIdx.x < more);
    if (before <= begin && begin < before + mine) {
      int r = r0;
      if (run > 1)
        for (;; ++r) {
          const long long n = places(r);
          if (begin < before + n || r + 1 >= r1) break;
          before += n;
        }
      sh.first = r;
      sh.at = before;
      sh.begin = begin;
      sh.end = end;
    }
  }
  __syncthreads();
  WeighWalk walk;
  if (walk.start(p, sh)) {
    if (warp == kWeighSums) {
      // ---- K, or of it the pairs' first tiles
      WeighKeys keys(p, walk, p.shared_loads ? 1 : 3);
      for (bool more = true; more;) {
        WeighWalk ahead = walk;
        more = ahead.next(p);
        if (!keys.load(sh, p, smem, stage_bytes, walk, ahead, more)) break;
        walk = ahead;
      }
      keys.land(sh, p);
    } else if (warp == kWeighSums + 1) {
      // ---- Q and its columns' -lse log2(e) (loaded two tiles ahead) of every pair's column
      // tiles, or once for a unit that has only one
      int tok[4], from[4];  // of the lane's columns of a tile: token, place of the lse
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        tok[y] = (lane + 32 * y) / p.G;
        from[y] = tok[y] * p.heads + lane + 32 * y - tok[y] * p.G;
      }
      WeighKeys keys(p, walk, p.shared_loads ? 2 : 0);
      unsigned issued = 0;
      bool ok = true;
      for (bool more = true; ok && more;) {
        const WeighWalk now = walk;
        more = walk.next(p);
        if (p.shared_loads && !keys.load(sh, p, smem, stage_bytes, now, walk, more)) break;
        if (now.u.tiles == 1 && !now.fresh) continue;
        const float* lse = p.lse + (long long)now.u.lo * p.heads + now.head * p.G;
        const int tokens = now.u.tokens, t0 = now.first_tile(p);
        float z[2][4];
        auto look = [&](int t, float* z) {
          const int first = t * p.tile_tokens, n = min(p.tile_tokens, tokens - first);
#pragma unroll
          for (int y = 0; y < 4; ++y)
            z[y] = tok[y] < n ? lse[(long long)first * p.heads + from[y]] : -INFINITY;
        };
        auto put = [&](int t, float* z) {
          const unsigned at = issued % p.q_stages, la = issued % kWeighShifts;
          ok = weigh_wait(sh, p, &sh.q_empty[at], issued / p.q_stages + 1);
          if (!ok) return;
          if (lane == 0) {
            mbar_arrive_expect_tx(&sh.q_full[at], p.blocks * p.tile_tokens * p.G * 128);
            for (int x = 0; x < p.blocks; ++x)
              tma_load_4d(q_smem + at * stage_bytes + x * kWeighTile * 128, &p.q_map, 64 * x, 0,
                          now.head, now.u.lo + t * p.tile_tokens, &sh.q_full[at]);
          }
          __syncwarp();
          ++issued;
          ok = weigh_wait(sh, p, &sh.l_empty[la], (issued - 1) / kWeighShifts + 1);
          if (!ok) return;
#pragma unroll
          for (int y = 0; y < 4; ++y)
            sh.shift[la][lane + 32 * y] =
                z[y] == -INFINITY ? -INFINITY : z[y] * -1.4426950408889634f;
          __syncwarp();
          if (lane == 0 && !MUTE) mbar_arrive(&sh.l_full[la]);
          look(t + 2, z);
        };
        look(t0, z[0]);
        look(t0 + 1, z[1]);
        for (int t = t0; ok && t < now.u.tiles; t += 2) {
          put(t, z[0]);
          if (ok && t + 1 < now.u.tiles) put(t + 1, z[1]);
        }
      }
      keys.land(sh, p);
      for (unsigned r = issued > p.q_stages ? issued - p.q_stages : 0; r < issued; ++r)
        weigh_land(&sh.q_full[r % p.q_stages], r / p.q_stages);
    } else if (warp == kWeighSums + 2 || warp == kWeighSums + 3) {
      // ---- products of the pair's one or other tile
      const int g = __shfl_sync(~0u, warp - kWeighSums - 2, 0);
      // (shuffles tell the compiler that a value is the same in all lanes, so that descriptors are
      // made in uniform registers, where the products take them from)
      const bool one = elect_one();
      const uint32_t tmem = __shfl_sync(~0u, sh.tmem, 0) + g * 256;
      const uint64_t k0 = mma_desc(smem_addr(smem), 16), q0 = mma_desc(smem_addr(q_smem), 16);
      const int steps = (p.dim + 15) / 16;
      unsigned k_count = 0, q_count = 0, s_count = 0;
      bool ok = true;
      do {
        const bool mine = walk.has(g), single = walk.u.tiles == 1, last = walk.ends_unit();
        const unsigned ka = __shfl_sync(~0u, g * p.k_stages + k_count % p.k_stages, 0);
        const uint64_t kd = k0 + ka * (stage_bytes / 16);
        if (mine) ok = weigh_wait(sh, p, &sh.k_full[ka], k_count / p.k_stages);
        for (int t = walk.first_tile(p); ok && t < walk.u.tiles; ++t) {
          const unsigned qa = __shfl_sync(~0u, q_count % p.q_stages, 0);
          ok = weigh_wait(sh, p, &sh.q_full[qa], q_count / p.q_stages);
          if (!ok) break;
          if (mine) {
            const int columns =
                __shfl_sync(~0u, min(p.tile_tokens, walk.u.tokens - t * p.tile_tokens), 0) *
                p.G;
            const uint32_t kind =
                mma_kind(p.bf16, false, kWeighTile, (columns + 15) / 16 * 16);
            const uint32_t s = __shfl_sync(~0u, s_count & 1, 0);
            ok = weigh_wait(sh, p, &sh.s_free[g][s], s_count / 2 + 1);
            if (!ok) break;
            tmem_fence_after();
            const uint64_t qd = q0 + qa * (stage_bytes / 16);
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              const unsigned y = ((x / 4) * (kWeighTile * 128) + (x % 4) * 32) / 16;
              if (x < steps) mma_ss(tmem + s * 128, kd + y, qd + y, kind, x > 0, one);
            }
            mma_commit(&sh.s_full[g][s], one);
            ++s_count;
          }
          if (!single || last) {
            mma_commit(&sh.q_empty[qa], one);
            ++q_count;
          }
        }
        k_count += mine;
      } while (ok && walk.next(p));
      mma_commit(&sh.drain[g], one);
      weigh_land(&sh.drain[g], 0);
    } else if (warp < kWeighSums) {
      // ---- sums
      const int g = warp >> 3, turn = warp >> 2 & 1, row = tid & (kWeighTile - 1);
      const uint32_t tmem =
          sh.tmem + ((uint32_t)((warp & 3) * 32) << 16) + g * 256 + turn * 128;
      const int box_shift = min(p.rq.page_shift, 7);
      const unsigned long long c2 = f2_pack(p.c, p.c);
      unsigned l_count = 0, k_count = 0, s_count = 0, joins = 0;
      bool ok = true;
      do {
        const int t0 = walk.first_tile(p);
        const bool several = walk.u.tiles - t0 > 1;
        const bool mine = walk.has(g), single = walk.u.tiles == 1, last = walk.ends_unit();
        const int key = (walk.pair * 2 + g) * kWeighTile + row;
        float* w = nullptr;
        float before = 0.f;
        // From column tile all_from on all columns see all keys, and up to `whole` there are 128
        // columns: with code that looked at each column's place two chunks of 2048 took 387 us, 350
        // without.
        const int over = max((walk.pair * 2 + g + 1) * kWeighTile - 1 - walk.u.old(), 0);
        const int all_from = (over + p.tile_tokens - 1) / p.tile_tokens;
        const int whole =
            p.tile_tokens * p.G == kWeighTile ? walk.u.tokens / p.tile_tokens : 0;
        unsigned long long sum2[4] = {0, 0, 0, 0};
        float rest = 0.f;
        for (int t = t0; ok && t < walk.u.tiles; ++t) {
          const unsigned la = l_count % kWeighShifts;
          ok = weigh_wait(sh, p, &sh.l_full[la], l_count / kWeighShifts);
          if (!ok) break;
          if (mine && (s_count & 1) == turn) {
            ok = weigh_wait(sh, p, &sh.s_full[g][turn], s_count / 2);
            if (!ok) break;
            tmem_fence_after();
            if (t + 1 == walk.u.tiles) {  // the pair's last: this group writes the weights
              const unsigned ka = g * p.k_stages + k_count % p.k_stages;
              ok = weigh_wait(sh, p, &sh.k_full[ka], k_count / p.k_stages);  // (it has landed)
              if (!ok) break;
              const int number = sh.pages[ka][row >> box_shift];
              __syncwarp();
              if (lane == 0) mbar_arrive(&sh.k_empty[ka]);
              __syncwarp();
              if (number >= 0 && key < walk.u.len)
                w = p.weights + number * p.w_page + walk.head * p.w_head +
                    (key & ((1 << p.rq.page_shift) - 1));
              if (w && key < walk.u.old() && p.decay != 0.f) before = *w;
              __syncwarp();
            }
            const float* shift = sh.shift[la];
            // 32 columns from k on, which all keys see
            auto add = [&](int k) {
              float x[32];
              tmem_ld32(tmem + k, x);
              ulonglong2 z[8];
#pragma unroll
              for (int y = 0; y < 8; ++y) z[y] = *(const ulonglong2*)(shift + k + 4 * y);
              tmem_wait_ld(x);
#pragma unroll
              for (int y = 0; y < 8; ++y) {
                float a, b, c, d;
                f2_unpack(f2_fma(f2_pack(x[4 * y], x[4 * y + 1]), c2, z[y].x), a, b);
                f2_unpack(f2_fma(f2_pack(x[4 * y + 2], x[4 * y + 3]), c2, z[y].y), c, d);
                sum2[2 * (y & 1)] = f2_add(sum2[2 * (y & 1)], f2_pack(ex2(a), ex2(b)));
                sum2[2 * (y & 1) + 1] = f2_add(sum2[2 * (y & 1) + 1], f2_pack(ex2(c), ex2(d)));
              }
            };
            // the same, of which only the first n are columns (others may hold anything)
            auto add_some = [&](int k, int n) {
              float x[32];
              tmem_ld32(tmem + k, x);
              tmem_wait_ld(x);
#pragma unroll
              for (int y = 0; y < 32; ++y) {
                const float e = ex2(fmaf(x[y], p.c, shift[k + y]));
                if (y < n) rest += e;
              }
            };
            const int columns = min(p.tile_tokens, walk.u.tokens - t * p.tile_tokens) * p.G;
            if (t >= all_from && t < whole) {
#pragma unroll
              for (int k = 0; k < kWeighTile; k += 32) add(k);
            } else if (t >= all_from) {
              int k = 0;
#pragma unroll 1
              for (; k + 32 <= columns; k += 32) add(k);
              if (k < columns) add_some(k, columns - k);
            } else {
              // columns [from, columns) of the tile see the key
              const long long ahead = (long long)key - walk.u.old() - t * p.tile_tokens;
              const int from = ahead > 0 ? (int)min(ahead * p.G, (long long)kWeighTile) : 0;
#pragma unroll 1
              for (int k = 0; k < columns; k += 32) {
                if (__all_sync(~0u, from >= k + 32)) continue;
                if (__all_sync(~0u, from <= k) && k + 32 <= columns) {
                  add(k);
                  continue;
                }
                float x[32];
                tmem_ld32(tmem + k, x);
                tmem_wait_ld(x);
#pragma unroll
                for (int y = 0; y < 32; ++y) {
                  const float e = ex2(fmaf(x[y], p.c, shift[k + y]));
                  if (k + y >= from && k + y < columns) rest += e;
                }
              }
            }
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.s_free[g][turn]);
          }
          s_count += mine;
          __syncwarp();
          if (!single || last) {
            if (lane == 0) mbar_arrive(&sh.l_empty[la]);
            ++l_count;
          }
        }
        if (!ok) break;
        k_count += mine;
        float a, b;
        f2_unpack(f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3])), a, b);
        a = rest + (a + b);
        if (mine && several) {
          // The other group's part: all eight warps meet, and meet again before `part` is
          // written anew.
          const bool writes = (s_count - 1 & 1) == turn;
          float* part = sh.part[g][joins & 1] + row;
          if (!writes) *part = a;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.joined[g]);
          __syncwarp();
          ok = weigh_wait(sh, p, &sh.joined[g], joins);
          if (!ok) break;
          if (writes) a += *part;
          ++joins;
        }
        if (w) *w = before * p.decay + a;
      } while (walk.next(p));
    }
  }
  tmem_fence_before();
  __syncthreads();
  if (warp == kWeighSums + 2) {
    tmem_fence_after();
    tmem_free(sh.tmem, 512);
  }
}

}  // namespace sv
