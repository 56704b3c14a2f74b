// Eviction: which tokens stay, and the closing of the gaps (spec_cache_evict).
//
// k_evict_pick, one block for a request and kv head, or a cluster: the kept tokens are those of
// the largest weights (pick_short, pick_items, pick_any), the ones that always stay among them; for
// each that moves it is written down where it comes from. The same blocks do the bookkeeping:
// every block adds up all requests' pages that go, so each finds for itself whether the call can
// be done at all and where its request's pages come on the stack. Numbers there that are no pages
// are found by the block that puts them on; where there are some the stack is written again
// without them, by one more block of k_evict_move, before anything can take from it.
//
// k_evict_move: keys, values and weights to their new places. Tokens only move down and keep
// their order, so a request and head go upwards in batches: all of a batch is read, in registers,
// before any of it is written, and what is overwritten is never a later batch's source. One block
// for a request and head, or a cluster of up to eight where there are few. Bound by HBM: 64 requests
// of 1990-2500 move 765 MB in 159 us, 0.72 of the rate of a copy.
#pragma once
#include <type_traits>

#include "sparse_common.cuh"

namespace sv {

constexpr int kMoveThreads = 256;

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
  int held;      // weights that fit the dynamic shared memory (any length)
  int vec;       // weights of 8 tokens on 16-byte boundaries
  int by_page;   // whether `from` goes by pages of the pool, or by columns of the table
  int* begin;    // [B][kv_heads] the first kept token that moves; none: 0x7fffffff
  int* broken;   // [B] whether a column that is given back holds no page
  int* from;     // where kept tokens come from, in pages [kv_heads][page_size]
  int ranks;     // blocks of a request and kv head that pick its tokens
  int cluster;   // ... that move its tokens

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

template <int NT>
struct EvictBooks {
  int begin;
  long long sums[NT / 32], befores[NT / 32];
};

// A request's bookkeeping. True: tokens go, of which `kept` of `len` stay. By the whole block.
template <int NT>
__device__ __forceinline__ bool evict_books(const EvictParams& p, int row, int b, int head,
                                            int rank, EvictBooks<NT>& sh, int& len, int& kept) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long most = (long long)p.rq.width << p.rq.page_shift;
  // ---- all requests' pages that go, and those of the requests before this one
  long long gone = 0, before = 0;
  bool bad = false;
  for (int r = tid; r < p.rq.B; r += NT) {
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
  if (lane == 0) sh.sums[warp] = gone, sh.befores[warp] = before;
  if (tid == 0) sh.begin = 0x7fffffff;
  bad = __syncthreads_or(bad);
  gone = before = 0;
  for (int w = 0; w < NT / 32; ++w) gone += sh.sums[w], before += sh.befores[w];
  const int free_now = *p.free_count;
  bad |= free_now < 0 || free_now + gone > p.rq.num_pages;
  if (blockIdx.x == 0 && tid == 0) {
    *p.free_count_out = free_now + (bad ? 0 : (int)gone);
    if (bad) atomicOr(p.rq.status, SPEC_CACHE_BAD_LENGTHS);
  }
  if (b >= p.rq.B) return false;  // (a call without requests)
  len = p.rq.kv_lens[b];
  kept = bad ? len : p.kept(len, p.budget[b]);
  if (head == 0 && rank == 0) {
    bool none = false;
    if (!bad) {
      const int c0 = p.pages(kept), n = p.pages(len) - c0;
      for (int i = tid; i < n; i += NT) {
        const int page = p.rq.table[b * p.rq.table_stride + c0 + i];
        none |= page < 0 || page >= p.rq.num_pages;
        p.free_pages[free_now + before + i] = page;
      }
    }
    none = __syncthreads_or(none);
    if (tid == 0) {
      p.lens_out[b] = kept;
      p.broken[b] = none;
      if (none) atomicOr(p.rq.status, SPEC_CACHE_BAD_PAGE);
    }
  }
  if (kept < len) return true;
  if (tid == 0 && rank == 0) p.begin[row] = 0x7fffffff;
  return false;
}

// Token j of request b becomes token `at`: `least` is the first that moves.
__device__ __forceinline__ void evict_note(const EvictParams& p, int b, int head, int j, int at,
                                           int& least) {
  if (j == at) return;
  least = min(least, at);
  int* to = p.from_at(b, head, at);
  if (to) *to = j;
}

// Requests of up to 16 NT tokens, whose weights the registers hold (pick_short). 108 requests of
// 138-173 tokens with 8 heads: both kernels 17.3 us, 33 with pick_items in as many threads, 76 in the
// 1024 of longer requests; 64 of 1990-2500, on three pools in turn, 187 and with those 1024 207.
template <int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) k_evict_pick_short(const EvictParams p) {
  __shared__ ShortPick<NT> sh;
  __shared__ EvictBooks<NT> books;
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x / p.kv_heads, head = blockIdx.x - b * p.kv_heads;
  sh.clear();
  int len, kept;
  if (!evict_books<NT>(p, blockIdx.x, b, head, 0, books, len, kept)) return;
  const ShortRow<NT> row(len);
  float v[kShortWords][4] = {};
#pragma unroll
  for (int w = 0; w < kShortWords; ++w) {
    const int j = row.c0 + 128 * w;  // (four tokens of one page)
    if (w >= row.busy || j >= len) break;
    const int page = p.rq.page(b, j >> p.rq.page_shift);
    if (page < 0) continue;
    const float* src = p.weights + page * p.w_page + head * p.w_head +
                       (j & ((1 << p.rq.page_shift) - 1));
    if (p.vec) {
      const float4 x = *(const float4*)src;
      v[w][0] = x.x, v[w][1] = x.y, v[w][2] = x.z, v[w][3] = x.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[w][i] = src[i];
    }
  }
  int least = 0x7fffffff;
  pick_short<NT>(v, row, len, p.first, p.recent, kept - p.first - p.recent, sh,
                 [&](int j, int at) { evict_note(p, b, head, j, at, least); });
  least = __reduce_min_sync(~0u, least);
  if ((threadIdx.x & 31) == 0) atomicMin(&books.begin, least);
  __syncthreads();
  if (threadIdx.x == 0) p.begin[blockIdx.x] = books.begin;
}

// ITEMS: tokens of a thread (8 at a time, which one page holds), or 0 for requests of any length.
// CLUSTER: p.ranks blocks for a request and kv head.
template <int NT, int ITEMS, bool CLUSTER>
__global__ void __launch_bounds__(NT) k_evict_pick(const EvictParams p) {
  __shared__ std::conditional_t<CLUSTER, ClusterPick<NT>, PickShared<NT>> sh;
  __shared__ EvictBooks<NT> books;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  const int rank = CLUSTER ? blockIdx.x % p.ranks : 0;
  const int row = CLUSTER ? blockIdx.x / p.ranks : blockIdx.x;
  const int b = row / p.kv_heads, head = row - b * p.kv_heads;
  int len, kept;
  if (!evict_books<NT>(p, row, b, head, rank, books, len, kept)) return;
  const int in_page = (1 << p.rq.page_shift) - 1;
  auto always = [&](int j) { return j < p.first || j >= len - p.recent; };
  int least = 0x7fffffff;
  auto moves = [&](int j, int at) { evict_note(p, b, head, j, at, least); };
  // the keys of tokens j .. j + 7, which are in one page
  auto look8 = [&](int j, uint32_t* keys) {
    float w[8] = {};
    const int page = j < len ? p.rq.page(b, j >> p.rq.page_shift) : -1;
    if (page >= 0) {
      const float* src = p.weights + page * p.w_page + head * p.w_head + (j & in_page);
      if (p.vec) {
        const float4 x = *(const float4*)src, y = *(const float4*)(src + 4);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
      } else {
#pragma unroll
        for (int y = 0; y < 8; ++y) w[y] = src[y];
      }
    }
#pragma unroll
    for (int y = 0; y < 8; ++y)
      keys[y] = j + y >= len ? 0u : always(j + y) ? kAlways : order_key(w[y]);
  };
  if constexpr (ITEMS > 0) {
    uint32_t keys[ITEMS];
    const int j0 = (rank * NT + tid) * ITEMS;
#pragma unroll
    for (int i = 0; i < ITEMS; i += 8) look8(j0 + i, keys + i);
    int at = 0;
    uint32_t taken = 0;
    if (kept > 0) {
      if constexpr (CLUSTER)
        taken = pick_items_cluster<NT, ITEMS>(keys, kept, sh, p.ranks, rank, at);
      else
        taken = pick_items<NT, ITEMS>(keys, kept, sh, at);
    }
    for (; taken; taken &= taken - 1) moves(j0 + __ffs(taken) - 1, at++);
  } else {
    extern __shared__ __align__(128) char smem[];
    uint32_t* held = (uint32_t*)smem;
    auto look = [&](int j) {
      if (always(j)) return kAlways;
      const int page = p.rq.page(b, j >> p.rq.page_shift);
      return order_key(
          page < 0 ? 0.f : p.weights[page * p.w_page + head * p.w_head + (j & in_page)]);
    };
    const int fits = min(len, p.held);
#pragma unroll 4
    for (int j = 8 * tid; j < fits; j += 8 * NT) {  // (room for a multiple of 8)
      uint32_t x[8];
      look8(j, x);
      *(uint4*)(held + j) = make_uint4(x[0], x[1], x[2], x[3]);
      *(uint4*)(held + j + 4) = make_uint4(x[4], x[5], x[6], x[7]);
    }
    __syncthreads();
    auto key = [&](int j) { return j < fits ? held[j] : look(j); };
    if (kept > 0)
      pick_any<NT>(key, len, kept, sh, [&](int w, uint32_t taken, int at) {
        for (; taken; taken &= taken - 1, ++at) moves(32 * w + __ffs(taken) - 1, at);
      });
  }
  least = __reduce_min_sync(~0u, least);
  if ((tid & 31) == 0) atomicMin(&books.begin, least);
  __syncthreads();
  if constexpr (CLUSTER) {  // the least of all blocks
    if (tid == 0) sh.counts[1].y = books.begin;
    cluster_sync();
    if (tid == 0 && rank == 0) {
      for (int r = 1; r < p.ranks; ++r) least = min(least, cluster_load(&sh.counts[1], r).y);
      p.begin[row] = min(least, books.begin);
    }
    cluster_sync();
  } else {
    if (tid == 0) p.begin[row] = books.begin;
  }
}

// The stack without the numbers that are no pages, if there are such. By a whole block; what a
// broken table costs does not matter, so one warp goes through the requests in order.
__device__ __forceinline__ void evict_restack(const EvictParams& p) {
  bool any = false;
  for (int b = threadIdx.x; b < p.rq.B; b += kMoveThreads) any |= p.broken[b] != 0;
  if (!__syncthreads_or(any) || threadIdx.x >= 32) return;
  const int lane = threadIdx.x;
  int top = *p.free_count;
  for (int b = 0; b < p.rq.B; ++b) {
    const int end = p.pages(p.rq.kv_lens[b]);
    for (int c = p.pages(p.lens_out[b]); c < end; c += 32) {
      const int page = c + lane < end ? p.rq.table[b * p.rq.table_stride + c + lane] : -1;
      const bool there = page >= 0 && page < p.rq.num_pages;
      const uint32_t votes = __ballot_sync(~0u, there);
      if (there) p.free_pages[top + __popc(votes & ((1u << lane) - 1))] = page;
      top += __popc(votes);
    }
  }
  if (lane == 0) *p.free_count_out = top;
}

// One row of blocks for each request and kv head, and one for the stack.
__global__ void __launch_bounds__(kMoveThreads) k_evict_move(const EvictParams p) {
  constexpr int kWarps = kMoveThreads / 32;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = p.cluster > 1 ? blockIdx.x % p.cluster : 0;
  const long long row = blockIdx.x / p.cluster;
  const int b = (int)(row / p.kv_heads), head = (int)(row - (long long)b * p.kv_heads);
  if (b == p.rq.B) {
    if (rank == 0) evict_restack(p);
    return;
  }
  const int begin = p.begin[row], kept = p.lens_out[b];
  if (begin >= kept) return;  // (the whole cluster)
  const int len = p.rq.kv_lens[b], mask = (1 << p.rq.page_shift) - 1;
  // A warp's lanes take the 16-byte pieces of a token's keys and values, of up to four tokens at
  // a time; eight times as many are a batch, and a lane keeps what one of those needs.
  const int pieces = p.dim / 8, at_once = min(32 / (2 * pieces), 4);
  const int sub = lane / (2 * pieces), piece = lane - sub * 2 * pieces;
  const bool is_v = piece >= pieces, there = sub < at_once;
  const int per_warp = 8 * at_once, per_batch = p.cluster * kWarps * per_warp;
  const long long s_page = is_v ? p.v_page : p.k_page, s_token = is_v ? p.v_token : p.k_token;
  char* base = is_v ? p.v + head * p.v_head + (piece - pieces) * 16
                    : p.k + head * p.k_head + piece * 16;
  struct Token {
    int src, src_page, dst_page;  // pages < 0: does not move
  };
  const long long first = (long long)begin + (rank * kWarps + warp) * per_warp;
  auto look = [&](long long batch) {
    const long long i = first + batch * per_batch + lane;
    Token t = {0, -1, -1};
    if (lane >= per_warp || i >= kept) return t;
    const int* at = p.from_at(b, head, (int)i);
    t.src = at ? *at : -1;
    if (t.src <= i || t.src >= len) return t;
    t.src_page = p.rq.page(b, t.src >> p.rq.page_shift);
    t.dst_page = t.src_page < 0 ? -1 : p.rq.page(b, (int)i >> p.rq.page_shift);
    return t;
  };
  auto load = [&](const Token& t, uint4* got, float& w) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int from = there ? u * at_once + sub : 0;
      const int src = __shfl_sync(~0u, t.src, from), page = __shfl_sync(~0u, t.src_page, from);
      const bool moves = __shfl_sync(~0u, t.dst_page, from) >= 0 && there;
      if (moves) got[u] = *(const uint4*)(base + page * s_page + (src & mask) * s_token);
    }
    if (t.dst_page >= 0) w = p.weights[t.src_page * p.w_page + head * p.w_head + (t.src & mask)];
  };
  auto store = [&](const Token& t, long long batch, const uint4* got, float w) {
    const long long i0 = first + batch * per_batch;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int from = there ? u * at_once + sub : 0;
      const int page = __shfl_sync(~0u, t.dst_page, from);
      if (page >= 0 && there)
        *(uint4*)(base + page * s_page + ((int)(i0 + from) & mask) * s_token) = got[u];
    }
    if (t.dst_page >= 0)
      p.weights[t.dst_page * p.w_page + head * p.w_head + ((int)(i0 + lane) & mask)] = w;
  };
  auto meet = [&] {
    if (p.cluster > 1)
      cluster_sync();
    else
      __syncthreads();
  };
  // Everything of a batch is read before any of it is written; the next batch's reads, which no
  // write of this one can hit, are under way by then.
  const long long batches = ((long long)kept - begin + per_batch - 1) / per_batch;
  Token now = look(0), then = look(1);
  uint4 got[2][8];
  float w[2];
  load(now, got[0], w[0]);
#pragma unroll 1
  for (long long k = 0; k < batches; k += 2) {
    Token more = look(k + 2);
    load(then, got[1], w[1]);
    meet();
    store(now, k, got[0], w[0]);
    if (k + 1 >= batches) break;
    now = more;
    more = look(k + 3);
    load(now, got[0], w[0]);
    meet();
    store(then, k + 1, got[1], w[1]);
    then = more;
  }
}

}  // namespace sv
