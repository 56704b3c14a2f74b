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

// Rows of up to 16 NT columns, which the registers hold (pick_short).
template <int NT>
__global__ void __launch_bounds__(NT, NT == 32 ? 24 : 1024 / NT)
    k_cache_select_short(const SelectParams p) {
  __shared__ ShortPick<NT> sh;
  pdl_trigger();
  pdl_wait();
  select_check<NT>(p);
  const long long t = blockIdx.x / p.kv_heads;
  const int head = (int)(blockIdx.x - t * p.kv_heads);
  int* out = p.out + blockIdx.x * (long long)p.count;
  const int n = select_visible(p, t);
  if (n <= p.count) {
    for (int i = threadIdx.x; i < p.count; i += NT) out[i] = i < n ? i : -1;
    return;
  }
  sh.clear();
  const float* scores = p.scores + t * p.s_token + head * p.s_head;
  const ShortRow<NT> row(n);
  float v[kShortWords][4];
#pragma unroll
  for (int w = 0; w < kShortWords; ++w) {
    const int c = row.c0 + 128 * w;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (w < row.busy) {
      if (p.vec && c + 3 < n) {
        x = *(const float4*)(scores + c);
      } else {
        if (c < n) x.x = scores[c];
        if (c + 1 < n) x.y = scores[c + 1];
        if (c + 2 < n) x.z = scores[c + 2];
        if (c + 3 < n) x.w = scores[c + 3];
      }
    }
    v[w][0] = x.x, v[w][1] = x.y, v[w][2] = x.z, v[w][3] = x.w;
  }
  pick_short<NT>(v, row, n, p.first, p.recent, p.count - p.first - p.recent, sh,
                 [&](int c, int at) { out[at] = c; });
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
