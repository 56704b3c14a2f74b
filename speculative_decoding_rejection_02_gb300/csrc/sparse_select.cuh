// The columns of the highest scores (spec_cache_select).
//
// One block for a row (token, kv head); a thread has a run of ITEMS columns' scores in registers
// as whole numbers of the same order. The k-th largest is found by histograms of its bits
// (pick_cut; with scores from a model two of the three decide), and sums over the threads give
// each selected column its place: of equal scores the lowest columns. Columns that are always
// selected have a key above all scores'.
//
// Bound by the chain of a block: request, scores, two histograms, the sums. Rows that are too long
// for registers (16384 columns) are read again from L2, or from shared memory where they fit.
#pragma once
#include "sparse_common.cuh"

namespace sv {

struct SelectParams {
  Requests rq;  // width: columns of scores
  int kv_heads, count, first, recent;
  const float* scores;
  long long s_token, s_head;
  int vec;      // rows on 16-byte boundaries
  int* out;
  int held;     // scores that fit the dynamic shared memory (any length)
};

// Visible columns of token t. By the whole block; `at` is shared.
template <int NT>
__device__ __forceinline__ int select_visible(const SelectParams& p, long long t, int* at) {
  if (threadIdx.x == 0) *at = 0;
  __syncthreads();
  for (int b = threadIdx.x; b < p.rq.B; b += NT) {
    const int lo = p.rq.cu_q[b], hi = p.rq.cu_q[b + 1], len = p.rq.length(b);
    if (lo < 0 || hi < lo || hi > p.rq.T) {
      atomicOr(p.rq.status, SPEC_CACHE_BAD_LENGTHS);
    } else if (lo <= t && t < hi) {
      const long long pos = (long long)len - hi + t;
      // (of several requests that claim the token, the one that shows most)
      if (len > 0 && pos >= 0) atomicMax(at, (int)(pos >> p.rq.page_shift) + 1);
    }
  }
  __syncthreads();
  return *at;
}

// ITEMS: columns of a thread, or 0 for rows of any length.
template <int NT, int ITEMS>
__global__ void __launch_bounds__(NT) k_cache_select(const SelectParams p) {
  __shared__ PickShared<NT> sh;
  __shared__ int visible;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  const long long t = blockIdx.x / p.kv_heads;
  const int head = (int)(blockIdx.x - t * p.kv_heads);
  int* out = p.out + blockIdx.x * (long long)p.count;
  const int n = select_visible<NT>(p, t, &visible);
  if (n <= p.count) {
    for (int i = tid; i < p.count; i += NT) out[i] = i < n ? i : -1;
    return;
  }
  const float* row = p.scores + t * p.s_token + head * p.s_head;
  auto always = [&](int c) { return c < p.first || c >= n - p.recent; };
  if constexpr (ITEMS > 0) {
    uint32_t keys[ITEMS];
    const int c0 = tid * ITEMS;
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
    for (uint32_t taken = pick_items<NT, ITEMS>(keys, p.count, sh, at); taken; taken &= taken - 1)
      out[at++] = c0 + __ffs(taken) - 1;
  } else {
    extern __shared__ __align__(1024) char smem[];
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
