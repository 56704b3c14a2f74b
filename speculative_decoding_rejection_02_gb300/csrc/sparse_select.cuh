// The columns of the highest scores (spec_cache_select).
//
// One block for a row (token, kv head). The k-th largest of the free columns' scores is found by
// three histograms of its bits (pick_cut), then all columns are gone over once in order, as bits
// of words, which gives each selected column its place (pick_words): of equal scores the lowest
// columns, and no result depends on the order of the threads. Scores are kept in shared memory
// where they fit.
#pragma once
#include "sparse_common.cuh"

namespace sv {

constexpr int kSelectThreads = 256;

struct SelectParams {
  Requests rq;  // width: columns of scores
  int kv_heads, count, first, recent;
  const float* scores;
  long long s_token, s_head;
  int* out;
  int held;  // scores that fit the dynamic shared memory
};

__global__ void __launch_bounds__(kSelectThreads) k_cache_select(const SelectParams p) {
  extern __shared__ uint32_t held[];
  __shared__ PickShared<kSelectThreads> sh;
  __shared__ int sh_b;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  const long long t = blockIdx.x / p.kv_heads;
  const int head = (int)(blockIdx.x - t * p.kv_heads);
  int* out = p.out + blockIdx.x * (long long)p.count;
  // the token's request (of several that claim it, the last), and its position
  if (tid == 0) sh_b = -1;
  __syncthreads();
  for (int b = tid; b < p.rq.B; b += kSelectThreads) {
    const int lo = p.rq.cu_q[b], hi = p.rq.cu_q[b + 1];
    if (lo < 0 || hi < lo || hi > p.rq.T)
      atomicOr(p.rq.status, SPEC_CACHE_BAD_LENGTHS);
    else if (lo <= t && t < hi)
      atomicMax(&sh_b, b);
  }
  __syncthreads();
  const int b = sh_b;
  int n = 0;  // visible columns
  if (b >= 0) {
    const int len = p.rq.length(b);
    const long long pos = (long long)len - p.rq.cu_q[b + 1] + t;
    if (len > 0 && pos >= 0) n = (int)(pos >> p.rq.page_shift) + 1;
  }
  if (n <= p.count) {
    for (int i = tid; i < p.count; i += kSelectThreads) out[i] = i < n ? i : -1;
    return;
  }
  const float* row = p.scores + t * p.s_token + head * p.s_head;
  const int m = n - p.first - p.recent, k = p.count - p.first - p.recent;
  uint32_t cut = 0xffffffffu;
  int equals = 0;
  const bool fits = m <= p.held;
  if (fits)
    for (int j = tid; j < m; j += kSelectThreads) held[j] = order_key(row[p.first + j]);
  __syncthreads();
  auto key = [&](int j) { return fits ? held[j] : order_key(row[p.first + j]); };
  if (k > 0) equals = pick_cut<kSelectThreads>(key, m, k, sh, cut);
  auto kind = [&](int c) {
    if (c < p.first || c >= n - p.recent) return 2;
    if (k == 0) return 0;
    const uint32_t x = key(c - p.first);
    return x > cut ? 2 : x == cut ? 1 : 0;
  };
  pick_words<kSelectThreads>(kind, n, equals, sh, [&](int w, uint32_t taken, int at) {
    for (; taken; taken &= taken - 1) out[at++] = 32 * w + __ffs(taken) - 1;
  });
}

}  // namespace sv
