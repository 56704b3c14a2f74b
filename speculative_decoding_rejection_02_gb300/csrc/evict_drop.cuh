// Eviction: which tokens stay, and the closing of the gaps (spec_cache_evict).
//
// k_evict_pick, one block for a request and kv head: the heaviest free tokens by the largest
// weights' cut (pick_cut) and one pass over all tokens in order (pick_words), which writes for
// each kept token that moves where it comes from. The same blocks do the requests' bookkeeping:
// every block adds up all requests' pages that go, so each finds for itself whether the call can
// be done at all and where its request's pages come on the stack.
//
// k_evict_move: keys, values and weights to their new places. Tokens only move down and keep
// their order, so a warp that takes 64 bytes of the channels may go upwards in batches: it has
// read a batch before it writes one, and what it overwrites is never a later batch's source.
#pragma once
#include "sparse_common.cuh"

namespace sv {

constexpr int kPickThreads = 512;
constexpr int kMoveThreads = 128;

struct EvictParams {
  Requests rq;  // kv_lens: lens; no cu_q
  int kv_heads, dim, first, recent;
  char* k;
  long long k_page, k_token, k_head;  // bytes
  char* v;
  long long v_page, v_token, v_head;
  float* weights;
  long long w_page, w_head;  // elements
  const int* budget;
  int* free_pages;
  const int* free_count;
  int* lens_out;
  int* free_count_out;
  int held;      // weights that fit the dynamic shared memory
  int by_page;   // whether `from` goes by pages of the pool, or by columns of the table
  int* begin;    // [B][kv_heads] the first kept token that moves; none: 0x7fffffff
  int* from;     // where kept tokens come from, in pages [kv_heads][page_size]
  int slices;    // 64-byte pieces of a key

  __device__ __forceinline__ int kept(int len, int budget) const {
    return (int)min((long long)len, max((long long)budget, (long long)first + recent));
  }
  __device__ __forceinline__ int pages(int len) const {
    return (int)(((long long)len + (1 << rq.page_shift) - 1) >> rq.page_shift);
  }
  // The place of kept token i of request b: NULL where its page is none.
  __device__ __forceinline__ int* from_at(int b, int head, int i) const {
    const int c = i >> rq.page_shift;
    long long page = (long long)b * rq.width + c;
    if (by_page) {
      page = rq.table[b * rq.table_stride + c];
      if (page < 0 || page >= rq.num_pages) return nullptr;
    }
    return from + (((page * kv_heads + head) << rq.page_shift) +
                   (i & ((1 << rq.page_shift) - 1)));
  }
};

__global__ void __launch_bounds__(kPickThreads) k_evict_pick(const EvictParams p) {
  extern __shared__ uint32_t held[];
  __shared__ PickShared<kPickThreads> sh;
  __shared__ int begin;
  __shared__ long long sums[kPickThreads / 32], befores[kPickThreads / 32];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / p.kv_heads, head = blockIdx.x - b * p.kv_heads;
  const long long most = (long long)p.rq.width << p.rq.page_shift;
  // ---- all requests' pages that go, and those of the requests before this one
  long long gone = 0, before = 0;
  bool bad = false;
  for (int r = tid; r < p.rq.B; r += kPickThreads) {
    const int len = p.rq.kv_lens[r], budget = p.budget[r];
    bad |= len < 0 || len > most || len > 0x7fff0000 || budget < 0;
    const int n = p.pages(len) - p.pages(p.kept(len, budget));
    gone += n;
    if (r < b) before += n;
  }
  for (int d = 16; d > 0; d >>= 1) {
    gone += __shfl_xor_sync(~0u, gone, d);
    before += __shfl_xor_sync(~0u, before, d);
  }
  if (lane == 0) sums[warp] = gone, befores[warp] = before;
  if (tid == 0) begin = 0x7fffffff;
  bad = __syncthreads_or(bad);
  gone = before = 0;
  for (int w = 0; w < kPickThreads / 32; ++w) gone += sums[w], before += befores[w];
  const int free_now = *p.free_count;
  bad |= free_now < 0 || free_now + gone > p.rq.num_pages;
  if (blockIdx.x == 0 && tid == 0) {
    *p.free_count_out = free_now + (bad ? 0 : (int)gone);
    if (bad) atomicOr(p.rq.status, SPEC_CACHE_BAD_LENGTHS);
  }
  if (b >= p.rq.B) return;  // (a call without requests)
  const int len = p.rq.kv_lens[b], kept = bad ? len : p.kept(len, p.budget[b]);
  if (head == 0) {
    if (tid == 0) p.lens_out[b] = kept;
    if (!bad) {
      const int c0 = p.pages(kept), n = p.pages(len) - c0;
      for (int i = tid; i < n; i += kPickThreads)
        p.free_pages[free_now + before + i] = p.rq.table[b * p.rq.table_stride + c0 + i];
    }
  }
  if (kept == len) {
    if (tid == 0) p.begin[blockIdx.x] = begin;
    return;
  }
  // ---- the kept tokens
  auto weight = [&](int j) {
    const int page = p.rq.page(b, j >> p.rq.page_shift);
    return page < 0 ? 0.f
                    : p.weights[page * p.w_page + head * p.w_head +
                                (j & ((1 << p.rq.page_shift) - 1))];
  };
  const int m = len - p.first - p.recent, k = kept - p.first - p.recent;
  const bool fits = m <= p.held;
  if (fits && k > 0)
    for (int j = tid; j < m; j += kPickThreads) held[j] = order_key(weight(p.first + j));
  __syncthreads();
  auto key = [&](int j) { return fits ? held[j] : order_key(weight(p.first + j)); };
  uint32_t cut = 0xffffffffu;
  int equals = 0;
  if (k > 0) equals = pick_cut<kPickThreads>(key, m, k, sh, cut);
  auto kind = [&](int j) {
    if (j < p.first || j >= len - p.recent) return 2;
    if (k == 0) return 0;
    const uint32_t x = key(j - p.first);
    return x > cut ? 2 : x == cut ? 1 : 0;
  };
  int mine = 0x7fffffff;
  pick_words<kPickThreads>(kind, len, equals, sh, [&](int w, uint32_t taken, int at) {
    for (; taken; taken &= taken - 1, ++at) {
      const int j = 32 * w + __ffs(taken) - 1;
      if (j == at) continue;
      mine = min(mine, at);
      int* to = p.from_at(b, head, at);
      if (to) *to = j;
    }
  });
  mine = __reduce_min_sync(~0u, mine);
  if (lane == 0) atomicMin(&begin, mine);
  __syncthreads();
  if (tid == 0) p.begin[blockIdx.x] = begin;
}

__global__ void __launch_bounds__(kMoveThreads) k_evict_move(const EvictParams p) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long task = blockIdx.x * (kMoveThreads / 32ll) + (threadIdx.x >> 5);
  const int tasks = 2 * p.slices + 1;
  const long long row = task / tasks;
  const int slice = (int)(task - row * tasks);
  if (row >= (long long)p.rq.B * p.kv_heads) return;
  const int b = (int)(row / p.kv_heads), head = (int)(row - (long long)b * p.kv_heads);
  const int begin = p.begin[row], kept = p.lens_out[b];
  if (begin >= kept) return;
  const int len = p.rq.kv_lens[b], mask = (1 << p.rq.page_shift) - 1;
  // where kept token i comes from; -1 where that cannot be
  auto source = [&](int i) {
    const int* at = i < kept ? p.from_at(b, head, i) : nullptr;
    const int j = at ? *at : -1;
    return j > i && j < len ? j : -1;
  };
  if (slice == 2 * p.slices) {
    for (int i0 = begin; i0 < kept; i0 += 128) {
      float got[4];
      float* to[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + 32 * u + lane, j = source(i);
        const int src = j < 0 ? -1 : p.rq.page(b, j >> p.rq.page_shift);
        const int dst = j < 0 ? -1 : p.rq.page(b, i >> p.rq.page_shift);
        to[u] = src < 0 || dst < 0
                    ? nullptr
                    : p.weights + dst * p.w_page + head * p.w_head + (i & mask);
        if (to[u]) got[u] = p.weights[src * p.w_page + head * p.w_head + (j & mask)];
      }
      __syncwarp();
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (to[u]) *to[u] = got[u];
      __syncwarp();
    }
    return;
  }
  const bool is_v = slice >= p.slices;
  const int piece = (is_v ? slice - p.slices : slice) * 4 + (lane & 3);
  const long long s_page = is_v ? p.v_page : p.k_page, s_token = is_v ? p.v_token : p.k_token;
  char* base = (is_v ? p.v + head * p.v_head : p.k + head * p.k_head) + piece * 16;
  const bool there = piece * 8 < p.dim;
  for (int i0 = begin; i0 < kept; i0 += 64) {
    uint4 got[8];
    char* to[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + 8 * u + (lane >> 2), j = there ? source(i) : -1;
      const int src = j < 0 ? -1 : p.rq.page(b, j >> p.rq.page_shift);
      const int dst = j < 0 ? -1 : p.rq.page(b, i >> p.rq.page_shift);
      to[u] = src < 0 || dst < 0 ? nullptr : base + dst * s_page + (i & mask) * s_token;
      if (to[u]) got[u] = *(const uint4*)(base + src * s_page + (j & mask) * s_token);
    }
    __syncwarp();
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (to[u]) *(uint4*)to[u] = got[u];
    __syncwarp();
  }
}

}  // namespace sv
