// The columns of the highest scores (spec_cache_select).
//
// Scores become whole numbers of the same order; columns that are always selected have one above
// all scores'. The k-th largest is found by histograms of its bits, and of equal ones the lowest
// columns are taken. One block for a row (token, kv head): with 16 columns in each thread's
// registers up to 4096 columns (k_cache_select_short), else with ITEMS (pick_items; with scores
// from a model two of the three histograms decide) up to 16384. Longer rows are picked from by a
// cluster of blocks where there are few, else by a block that reads them again from shared memory,
// and what does not fit there from L2.
//
// Bound by the chain of a row: request, scores, histograms, the places.
#pragma once
#include <type_traits>

#include "sparse_common.cuh"

namespace sv {

struct SelectParams {
  Requests rq;  // width: columns of scores
  int kv_heads, count, first, recent;
  const float* scores;
  long long s_token, s_head;
  int vec;      // rows on 16-byte boundaries
  int* out;
  int ranks;    // blocks of a row
  int held;     // scores that fit the dynamic shared memory (any length)
};

// Visible columns of token t; the same in all lanes of the warp. The request is searched for by
// 32 offsets at a time, which rise (the first block looks whether all do).
__device__ __forceinline__ int select_visible(const SelectParams& p, long long t) {
  const int lane = threadIdx.x & 31;
  int from = 0, to = p.rq.B;  // the last of these requests whose offset is t at most
  while (to - from > 1) {
    const int step = (to - from + 31) / 32, b = from + lane * step;
    const int n = __popc(__ballot_sync(~0u, b < to && p.rq.cu_q[b] <= t));
    from += max(n - 1, 0) * step;
    to = min(to, from + step);
  }
  if (from >= p.rq.B) return 0;
  const int lo = p.rq.cu_q[from], hi = p.rq.cu_q[from + 1], len = p.rq.kv_lens[from];
  if (lo > t || t >= hi || hi > p.rq.T) return 0;
  if (len < 0 || len > ((long long)p.rq.width << p.rq.page_shift) || len > 0x7fff0000) return 0;
  const long long pos = (long long)len - hi + t;
  return len > 0 && pos >= 0 ? (int)(pos >> p.rq.page_shift) + 1 : 0;
}
// Tells of lengths and offsets that cannot be. By one block.
template <int NT>
__device__ __forceinline__ void select_check(const SelectParams& p) {
  if (blockIdx.x > 0) return;
  for (int b = threadIdx.x; b < p.rq.B; b += NT) {
    int lo, hi;
    p.rq.request(b, lo, hi);
  }
}

constexpr int kShortWords = 4;  // of 128 columns for each warp: 16 columns a thread
constexpr int kShortList = 32;  // candidates that are compared with one another

// Rows of up to 16 NT columns: a run of columns in the registers of each warp, and one histogram of
// 256 bins. The bins divide the values between the least and the largest score evenly, so that the
// bin of the k-th largest as a rule holds a few, which are compared with one another; else it is
// divided again, by the bits of the values' keys, which takes four rounds at most. 2560 rows of
// some 500 columns: 13 us, 21 with pick_items (with bins by the first bits most scores of a row
// are in a few bins, whose counts come one after the other), 15 to 21 with a warp for a row at
// other sizes. Instructions are what bounds it, so scores stay floats (NaN as +inf), and only words
// of columns with one that is always selected, or past the last, look at each column's place.
template <int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) k_cache_select_short(const SelectParams p) {
  constexpr int kWarps = NT / 32, kWords = kShortWords, kAllTies = 0x7fffffff;
  __shared__ __align__(16) int hist[2][256];
  __shared__ float list[kShortList], low_of[2][kWarps], high_of[2][kWarps];
  __shared__ int listed, taken_of[kWarps], ties_of[kWarps];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  select_check<NT>(p);
  const long long t = blockIdx.x / p.kv_heads;
  const int head = (int)(blockIdx.x - t * p.kv_heads);
  int* out = p.out + blockIdx.x * (long long)p.count;
  const int n = select_visible(p, t);
  if (n <= p.count) {
    for (int i = tid; i < p.count; i += NT) out[i] = i < n ? i : -1;
    return;
  }
  for (int i = tid; i < 128; i += NT) ((int4*)hist)[i] = make_int4(0, 0, 0, 0);
  if (tid == 0) listed = 0;
  const float* row = p.scores + t * p.s_token + head * p.s_head;
  // ---- the warp's words of 128 columns; a lane has four adjacent ones of each
  const int words = (n + 127) / 128, run = (words + kWarps - 1) / kWarps;
  const int c0 = 128 * run * warp + 4 * lane, busy = max(min(run, words - run * warp), 0);
  float v[kWords][4];
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    const int c = c0 + 128 * w;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (w < busy) {
      if (p.vec && c + 3 < n) {
        x = *(const float4*)(row + c);
      } else {
        if (c < n) x.x = row[c];
        if (c + 1 < n) x.y = row[c + 1];
        if (c + 2 < n) x.z = row[c + 2];
        if (c + 3 < n) x.w = row[c + 3];
      }
    }
    v[w][0] = x.x, v[w][1] = x.y, v[w][2] = x.z, v[w][3] = x.w;
  }
  // bits of the columns that scores decide, and of those that are always selected
  uint32_t free = 0, always = 0;
  float least = INFINITY, most = -INFINITY;
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    if (w >= busy) break;
    const int first = c0 - 4 * lane + 128 * w;
    uint32_t mine = 15;
    if (first < p.first || first + 128 > n - p.recent) {
      mine = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + 128 * w + i;
        const bool decides = c >= p.first && c < n - p.recent;
        mine |= (uint32_t)decides << i;
        always |= (uint32_t)(c < n && !decides) << (4 * w + i);
      }
    }
    free |= mine << (4 * w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (v[w][i] != v[w][i]) v[w][i] = INFINITY;
      if (mine >> i & 1) least = fminf(least, v[w][i]), most = fmaxf(most, v[w][i]);
    }
  }
  auto spread = [&](int turn) {  // least and most of all warps
    for (int d = 1; d < 32; d <<= 1) {
      least = fminf(least, __shfl_xor_sync(~0u, least, d));
      most = fmaxf(most, __shfl_xor_sync(~0u, most, d));
    }
    if (lane == 0) low_of[turn][warp] = least, high_of[turn][warp] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      least = fminf(least, low_of[turn][w]);
      most = fmaxf(most, high_of[turn][w]);
    }
  };
  spread(0);
  // ---- the cut: values above it are taken, and the first `equals` of those equal to it
  float cut = INFINITY;
  int k = p.count - p.first - p.recent, equals = 0;
  const float scale = 254.9f / (most - least);
  bool linear = least > -INFINITY && scale > 0.f && scale < INFINITY;
#pragma unroll 1
  for (int turn = 0; k > 0; turn ^= 1) {
    const float low = least, high = most;
    const uint32_t low_key = order_key(low);
    const int shift = max(24 - __clz(order_key(high) - low_key), 0);
    auto bin_of = [&](float x) {  // from 0 to 255, never falls where x rises
      if (linear) return __float_as_int(fmaf(x - low, scale, 8388608.f)) & 255;
      return (int)((order_key(x) - low_key) >> shift);
    };
    int* bins = hist[turn];
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      if (w >= busy) break;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (free >> (4 * w + i) & 1 && v[w][i] >= low && v[w][i] <= high)
          atomicAdd(&bins[bin_of(v[w][i])], 1);
    }
    __syncthreads();
    // each warp for itself: the lane's bins, the first lane's the highest
    const int first = 256 - 8 * (lane + 1);
    const int4 a = *(const int4*)&bins[first], b = *(const int4*)&bins[first + 4];
    const int h[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    int upto = ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));
    const int mine = upto;
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(~0u, upto, d);
      if (lane >= d) upto += y;
    }
    const int who = __ffs(__ballot_sync(~0u, k <= upto)) - 1;
    int left = k - (upto - mine), bin = 0, rest = 0, there = 0;
#pragma unroll
    for (int i = 7; i >= 0; --i) {
      if (left > 0 && left <= h[i]) bin = first + i, rest = left, there = h[i];
      left -= h[i];
    }
    bin = __shfl_sync(~0u, bin, who);
    k = __shfl_sync(~0u, rest, who);
    there = __shfl_sync(~0u, there, who);
    // the bin's values
    least = INFINITY, most = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      if (w >= busy) break;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (free >> (4 * w + i) & 1 && v[w][i] >= low && v[w][i] <= high &&
            bin_of(v[w][i]) == bin) {
          least = fminf(least, v[w][i]), most = fmaxf(most, v[w][i]);
          if (there <= kShortList) list[atomicAdd(&listed, 1)] = v[w][i];
        }
    }
    spread(turn ^ 1);
    if (there == k || least == most) {  // all of them, or the first of them
      cut = least;
      equals = k;
      if (there == k) equals = kAllTies;
      break;
    }
    if (there <= kShortList) {
      const float y = lane < there ? list[lane] : 0.f;
      int above = 0, same = 0;
      for (int i = 0; i < there; ++i) {
        const float z = list[i];
        above += z > y;
        same += z == y;
      }
      const uint32_t it = __ballot_sync(~0u, lane < there && above < k && k <= above + same);
      const int who = __ffs(it) - 1;
      cut = __shfl_sync(~0u, y, who);
      equals = k - __shfl_sync(~0u, above, who);
      if (equals == __shfl_sync(~0u, same, who)) equals = kAllTies;
      break;
    }
    linear = false;
    for (int i = tid; i < 256; i += NT) bins[i] = 0;  // (the next round has the other one)
  }
  // ---- the places of what is taken
  uint32_t taken = 0, ties = 0;
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    if (w >= busy) break;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      taken |= (uint32_t)(v[w][i] > cut) << (4 * w + i);
      ties |= (uint32_t)(v[w][i] == cut) << (4 * w + i);
    }
  }
  taken = (taken & free) | always;
  ties &= free;
  auto before_in_word = [&](uint32_t bits, int w, int& all) {
    const int mine = __popc(bits >> (4 * w) & 15);
    int upto = mine;
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(~0u, upto, d);
      if (lane >= d) upto += y;
    }
    all = __shfl_sync(~0u, upto, 31);
    return upto - mine;
  };
  if (equals == kAllTies) {
    taken |= ties;
  } else if (equals > 0) {  // (in all threads or none)
    const int mine = __reduce_add_sync(~0u, __popc(ties));
    if (lane == 0) ties_of[warp] = mine;
    __syncthreads();
    int at = 0;
    for (int w = 0; w < warp; ++w) at += ties_of[w];
    for (int w = 0; w < busy; ++w) {
      int all, before = at + before_in_word(ties, w, all);
      at += all;
      for (int i = 4 * w; i < 4 * w + 4; ++i)
        if (ties >> i & 1) taken |= (uint32_t)(before++ < equals) << i;
    }
  }
  const int mine = __reduce_add_sync(~0u, __popc(taken));
  if (lane == 0) taken_of[warp] = mine;
  __syncthreads();
  int at = 0;
  for (int w = 0; w < warp; ++w) at += taken_of[w];
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    if (w >= busy) break;
    int all, before = at + before_in_word(taken, w, all);
    at += all;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (taken >> (4 * w + i) & 1) out[before++] = c0 + 128 * w + i;
  }
}

// ITEMS: columns of a thread, or 0 for rows of any length. CLUSTER: p.ranks blocks for a row.
template <int NT, int ITEMS, bool CLUSTER>
__global__ void __launch_bounds__(NT) k_cache_select(const SelectParams p) {
  __shared__ std::conditional_t<CLUSTER, ClusterPick<NT>, PickShared<NT>> sh;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  const int rank = CLUSTER ? blockIdx.x % p.ranks : 0;
  const long long at_row = CLUSTER ? blockIdx.x / p.ranks : blockIdx.x;
  const long long t = at_row / p.kv_heads;
  const int head = (int)(at_row - t * p.kv_heads);
  int* out = p.out + at_row * p.count;
  select_check<NT>(p);
  const int n = select_visible(p, t);
  if (n <= p.count) {
    for (int i = tid + rank * NT; i < p.count; i += (CLUSTER ? p.ranks : 1) * NT)
      out[i] = i < n ? i : -1;
    return;
  }
  const float* row = p.scores + t * p.s_token + head * p.s_head;
  auto always = [&](int c) { return c < p.first || c >= n - p.recent; };
  if constexpr (ITEMS > 0) {
    uint32_t keys[ITEMS];
    const int c0 = (rank * NT + tid) * ITEMS;
#pragma unroll
    for (int i = 0; i < ITEMS; i += 4) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p.vec && c0 + i + 3 < n) {
        v = *(const float4*)(row + c0 + i);
      } else {
        if (c0 + i < n) v.x = row[c0 + i];
        if (c0 + i + 1 < n) v.y = row[c0 + i + 1];
        if (c0 + i + 2 < n) v.z = row[c0 + i + 2];
        if (c0 + i + 3 < n) v.w = row[c0 + i + 3];
      }
      keys[i] = order_key(v.x), keys[i + 1] = order_key(v.y);
      keys[i + 2] = order_key(v.z), keys[i + 3] = order_key(v.w);
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      keys[i] = c0 + i >= n ? 0u : always(c0 + i) ? kAlways : keys[i];
    int at;
    uint32_t taken;
    if constexpr (CLUSTER)
      taken = pick_items_cluster<NT, ITEMS>(keys, p.count, sh, p.ranks, rank, at);
    else
      taken = pick_items<NT, ITEMS>(keys, p.count, sh, at);
    for (; taken; taken &= taken - 1) out[at++] = c0 + __ffs(taken) - 1;
  } else {
    extern __shared__ __align__(128) char smem[];
    uint32_t* held = (uint32_t*)smem;
    auto look = [&](int c) { return always(c) ? kAlways : order_key(row[c]); };
    const int fits = min(n, p.held);
#pragma unroll 4
    for (int c = tid; c < fits; c += NT) held[c] = look(c);
    __syncthreads();
    auto key = [&](int c) { return c < fits ? held[c] : look(c); };
    pick_any<NT>(key, n, p.count, sh, [&](int w, uint32_t taken, int at) {
      for (; taken; taken &= taken - 1) out[at++] = 32 * w + __ffs(taken) - 1;
    });
  }
}

}  // namespace sv
