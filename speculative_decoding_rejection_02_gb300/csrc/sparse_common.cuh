// What the kernels of sparse attention and eviction share: requests and groups of new
// tokens, 16-bit products on the warp's tensor cores, the choice of the k largest values.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/spec_sparse.h"
#include "pipe.cuh"

namespace sv {

// a / b of numbers that are not negative; most fit 32 bits, whose division is much shorter.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return (a | b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

struct Requests {
  int B, T, width, page_shift;
  long long table_stride, num_pages;
  const int* table;
  const int* kv_lens;
  const int* cu_q;
  unsigned* status;

  // The length of request b; 0 with a status bit if it cannot be.
  __device__ __forceinline__ int length(int b) const { return checked(kv_lens[b]); }
  __device__ __forceinline__ int checked(int len) const {
    if (len >= 0 && len <= ((long long)width << page_shift) && len <= 0x7fff0000) return len;
    atomicOr(status, SPEC_CACHE_BAD_LENGTHS);
    return 0;
  }
  // The new tokens of request b as rows [lo, hi), and its length. Offsets that cannot be give
  // no rows (lo = hi = -1).
  __device__ __forceinline__ int request(int b, int& lo, int& hi) const {
    lo = cu_q[b];
    hi = cu_q[b + 1];
    if (lo < 0 || hi < lo || hi > T) {
      atomicOr(status, SPEC_CACHE_BAD_LENGTHS);
      lo = hi = -1;
    }
    return length(b);
  }
  // The page number in column c of request b; -1 with a status bit if it is none.
  __device__ __forceinline__ int page(int b, int c) const {
    const int x = table[b * table_stride + c];
    if (x >= 0 && x < num_pages) return x;
    atomicOr(status, SPEC_CACHE_BAD_PAGE);
    return -1;
  }
};

// Up to `per` new tokens of one request, in order: rows token .. token + tokens - 1, the first
// at position pos. b < 0: none. `pad`: rows from there on belong to no request, nor do some
// before it if `gaps`.
struct TokenGroup {
  int b, token, tokens, pos, len;
  int pad, gaps;
};

template <int NT>
struct GroupShared {
  TokenGroup group;
  long long sums[NT / 32];
  int pad[NT / 32], gaps[NT / 32];
};

// Group number `unit` of all requests' groups of `per` tokens. By the whole block.
template <int NT>
__device__ __forceinline__ TokenGroup find_group(const Requests& p, long long unit, int per,
                                                 GroupShared<NT>& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (p.B + NT - 1) / NT, r0 = min((long long)tid * run, (long long)p.B);
  const int r1 = min(r0 + run, p.B);
  long long mine = 0;
  int pad = 0, gaps = 0, lo = 0, hi = 0, len = 0;
  auto groups_of = [&](int r) {
    lo = p.cu_q[r];
    hi = p.cu_q[r + 1];
    len = p.kv_lens[r];
    if (lo < 0 || hi < lo || hi > p.T) {
      atomicOr(p.status, SPEC_CACHE_BAD_LENGTHS);
      lo = hi = -1;
    }
    return (hi - lo + per - 1) / per;
  };
#pragma unroll 1
  for (int r = r0; r < r1; ++r) {
    mine += groups_of(r);
    pad = max(pad, hi);
    gaps |= lo < 0 || (r == 0 && lo > 0);
  }
  long long upto = mine;
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(~0u, upto, d);
    if (lane >= d) upto += x;
  }
  pad = __reduce_max_sync(~0u, pad);
  gaps = __any_sync(~0u, gaps);
  if (lane == 31) sh.sums[warp] = upto;
  if (lane == 0) sh.pad[warp] = pad, sh.gaps[warp] = gaps;
  if (tid == 0) sh.group.b = -1;
  __syncthreads();
  long long before = upto - mine;
  for (int w = 0; w < warp; ++w) before += sh.sums[w];
  if (before <= unit && unit < before + mine) {
    long long at = before;
    int r = r0;
    if (run > 1)
      for (;; ++r) {
        const int n = groups_of(r);
        if (unit < at + n || r + 1 >= r1) break;
        at += n;
      }
    const int skip = (int)(unit - at) * per;
    len = p.checked(len);
    TokenGroup g;
    g.b = r;
    g.token = lo + skip;
    g.tokens = min(per, hi - lo - skip);
    g.pos = len - (hi - lo) + skip;
    g.len = len;
    if (len == 0) g.pos = -(1 << 30);  // sees nothing
    sh.group = g;
  }
  __syncthreads();
  TokenGroup g = sh.group;
  g.pad = 0;
  g.gaps = 0;
  for (int w = 0; w < NT / 32; ++w) g.pad = max(g.pad, sh.pad[w]), g.gaps |= sh.gaps[w];
  __syncthreads();
  return g;
}

// f(t) for every row t that belongs to no request, spread over the blocks. By whole blocks.
template <int NT, typename F>
__device__ __forceinline__ void for_idle_rows(const Requests& p, const TokenGroup& g, F f) {
#pragma unroll 1
  for (long long t = (g.gaps ? 0 : g.pad) + blockIdx.x; t < p.T; t += gridDim.x) {
    if (t < g.pad) {
      bool mine = false;
#pragma unroll 1
      for (int b = threadIdx.x; b < p.B; b += NT) {
        const int lo = p.cu_q[b], hi = p.cu_q[b + 1];
        mine |= lo >= 0 && lo <= t && t < hi && hi <= p.T;
      }
      if (__syncthreads_or(mine)) continue;
    }
    f((int)t);
  }
}

// D += A B on 16 x 8 x 16 of 16-bit values with fp32 sums. Lane 4 x + c of the warp holds rows x
// and x + 8 of A and D and column x of B: of A the columns 2c, 2c + 1 (a0, a1) and 2c + 8, 2c + 9
// (a2, a3), of B those rows (b0 and b1), of D columns 2c and 2c + 1 of row x, then of row x + 8.
// These tensor-core instructions of the warp have a fraction of tcgen05's rate, but need neither
// 64 rows nor TMEM: the calls here have 8 to 32 rows against keys that come once from memory,
// and wait for those.
template <bool BF16>
__device__ __forceinline__ void mma_16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  if (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D = A B.
template <bool BF16>
__device__ __forceinline__ void mma_16816_new(float* d, uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  if (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
  uint32_t r;
  if (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack_pair_down(float lo, float hi) {  // cut off, not rounded
  uint32_t r;
  if (BF16)
    asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool BF16>
__device__ __forceinline__ float2 unpack_pair(uint32_t v) {
  if (BF16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// ---- clusters of blocks

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// The float or integers at the same place of another block's shared memory.
__device__ __forceinline__ float cluster_load(const float* p, uint32_t rank) {
  uint32_t at;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ float2 cluster_load(const float2* p, uint32_t rank) {
  uint32_t at;
  float2 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
               : "=f"(v.x), "=f"(v.y)
               : "r"(at)
               : "memory");
  return v;
}
__device__ __forceinline__ int2 cluster_load(const int2* p, uint32_t rank) {
  uint32_t at;
  int2 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "r"(at)
               : "memory");
  return v;
}

// ---- the k largest of many values, of equal ones the first: no result depends on the order of
// the threads

// Whole numbers in the order of the values: NaN as +inf, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) v = INFINITY;
  const uint32_t u = __float_as_uint(v + 0.f);
  return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}

// Items that are taken whatever the others: their key, which no value has.
constexpr uint32_t kAlways = 0xffffffffu;

template <int NT>
struct PickShared {
  alignas(16) int hist[2048];
  int sums[2][NT / 32];
  int bin, rest, count;
};

// Sum of v over the threads before this one, and over all. By the whole block; `sums` is free
// again after the block's next barrier.
template <int NT>
__device__ __forceinline__ int block_before(int v, int* sums, int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int upto = v;
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(~0u, upto, d);
    if (lane >= d) upto += x;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  int w = lane < NT / 32 ? sums[lane] : 0;
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(~0u, w, d);
    if (lane >= d) w += x;
  }
  all = __shfl_sync(~0u, w, 31);
  const int before = __shfl_sync(~0u, w, max(warp - 1, 0));
  return (warp ? before : 0) + upto - v;
}

// The cut of the k largest of all keys, 0 < k: fewer than k keys are above it, and with the first
// `equals` keys that are equal to it there are k. `count(add)` calls add(key) for each of the
// thread's keys. Histograms of 11, 11 and 10 bits, of which one is left out when all that the one
// before it left open is taken. By the whole block.
template <int NT, typename F>
__device__ __forceinline__ uint32_t pick_cut(F count, int k, PickShared<NT>& sh, int& equals) {
  constexpr int kRun = 2048 / NT;  // bins of a thread, the first thread's the highest
  const int low = 2048 - (threadIdx.x + 1) * kRun;
  uint32_t prefix = 0, mask = 0;
  for (int i = threadIdx.x; i < 2048; i += NT) sh.hist[i] = 0;
  __syncthreads();
#pragma unroll 1
  for (int pass = 0;; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
    count([&](uint32_t x) {
      if ((x & mask) == prefix) atomicAdd(&sh.hist[x >> shift & (bins - 1)], 1);
    });
    __syncthreads();
    int h[kRun], mine = 0, all;
#pragma unroll
    for (int i = 0; i < kRun; i += 2) {
      const int2 v = *(const int2*)&sh.hist[low + i];
      *(int2*)&sh.hist[low + i] = make_int2(0, 0);
      h[i] = v.x, h[i + 1] = v.y;
      mine += v.x + v.y;
    }
    const int before = block_before<NT>(mine, sh.sums[0], all);
    if (before < k && k <= before + mine) {
      int left = k - before;
#pragma unroll
      for (int i = kRun - 1; i >= 0; --i) {
        if (left > 0 && left <= h[i]) sh.bin = low + i, sh.rest = left, sh.count = h[i];
        left -= h[i];
      }
    }
    __syncthreads();
    prefix |= (uint32_t)sh.bin << shift;
    mask |= (uint32_t)(bins - 1) << shift;
    k = sh.rest;
    if (sh.count == k) {  // all of this bin
      equals = 0;
      return prefix - 1;  // (prefix > 0, or all keys there are would be taken)
    }
    if (pass == 2) break;
    __syncthreads();
  }
  equals = k;
  return prefix;
}

// Of the thread's ITEMS keys (items ITEMS * thread .. of the block's) those among the k largest,
// of equal ones the first, as bits; `before`: how many items are taken before the thread's.
// Items that are not there have key 0; k are. By the whole block.
template <int NT, int ITEMS>
__device__ __forceinline__ uint32_t pick_items(const uint32_t* keys, int k, PickShared<NT>& sh,
                                               int& before) {
  int equals, all;
  const uint32_t cut = pick_cut<NT>(
      [&](auto add) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
          if (keys[i]) add(keys[i]);
      },
      k, sh, equals);
  uint32_t taken = 0, ties = 0;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    taken |= (uint32_t)(keys[i] > cut) << i;
    ties |= (uint32_t)(keys[i] == cut) << i;
  }
  if (equals > 0) {
    const int at = block_before<NT>(__popc(ties), sh.sums[1], all);
    for (int x = __popc(ties); x > 0 && at + x > equals; --x) ties &= ~(1u << (31 - __clz(ties)));
    taken |= ties;
    __syncthreads();
  }
  before = block_before<NT>(__popc(taken), sh.sums[0], all);
  return taken;
}

__device__ __forceinline__ int cluster_load(const int* p, uint32_t rank) {
  uint32_t at;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// pick_items by a cluster of `ranks` blocks (a power of two), of which each has the next run of
// items. Other blocks' shared memory is far, so only one warp of each looks at their histograms:
// at the sums of 64 bins, then at the 64 bins that have the cut. By the whole cluster.
template <int NT>
struct ClusterPick {
  static_assert(NT == 1024, "a warp for each 64 bins");
  PickShared<NT> own;
  alignas(16) int hist[2][2048];
  int coarse[2][32];
  int2 counts[2];  // (ties, -) and (taken, the first item that the caller looks for)
};
template <int NT, int ITEMS>
__device__ __forceinline__ uint32_t pick_items_cluster(const uint32_t* keys, int k,
                                                       ClusterPick<NT>& sh, int ranks, int rank,
                                                       int& before) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t prefix = 0, mask = 0, cut = 0;
  int equals = 0, all;
  for (int i = threadIdx.x; i < 4096; i += NT) sh.hist[0][i] = 0;
  __syncthreads();
#pragma unroll 1
  for (int pass = 0;; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
    int* hist = sh.hist[pass & 1];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      if (keys[i] && (keys[i] & mask) == prefix) atomicAdd(&hist[keys[i] >> shift & (bins - 1)], 1);
    __syncthreads();
    const int2 mine = ((const int2*)hist)[32 * warp + lane];
    const int sum = __reduce_add_sync(~0u, mine.x + mine.y);
    if (lane == 0) sh.coarse[pass & 1][warp] = sum;
    cluster_sync();
    // the other one is free for the next pass: all blocks have read it before they came here
    ((int2*)sh.hist[~pass & 1])[threadIdx.x] = make_int2(0, 0);
    if (warp == 0) {
      // lane l has the l-th highest group, then the l-th highest pair of bins
      auto upto = [&](int v) {
        for (int d = 1; d < 32; d <<= 1) {
          const int y = __shfl_up_sync(~0u, v, d);
          if (lane >= d) v += y;
        }
        return v;
      };
      int v[8], n = 0;
#pragma unroll
      for (int r = 0; r < 8; ++r)  // (from ranks on the same ones again)
        v[r] = cluster_load(&sh.coarse[pass & 1][31 - lane], r & (ranks - 1));
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < ranks) n += v[r];
      int sums = upto(n);
      int who = __ffs(__ballot_sync(~0u, k <= sums)) - 1;
      int left = k - __shfl_sync(~0u, sums - n, who);
      const int pair = 32 * (31 - who) + 31 - lane;
      int2 w[8];
      int low = 0, high = 0;
#pragma unroll
      for (int r = 0; r < 8; ++r) w[r] = cluster_load((const int2*)hist + pair, r & (ranks - 1));
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < ranks) low += w[r].x, high += w[r].y;
      sums = upto(low + high);
      who = __ffs(__ballot_sync(~0u, left <= sums)) - 1;
      if (lane == who) {
        left -= sums - low - high;
        const bool upper = left <= high;
        sh.own.bin = 2 * pair + upper;
        sh.own.rest = upper ? left : left - high;
        sh.own.count = upper ? high : low;
      }
    }
    __syncthreads();
    prefix |= (uint32_t)sh.own.bin << shift;
    mask |= (uint32_t)(bins - 1) << shift;
    k = sh.own.rest;
    cut = prefix;
    equals = k;
    if (sh.own.count == k) {
      cut = prefix - 1;
      equals = 0;
      break;
    }
    if (pass == 2) break;
    __syncthreads();
  }
  uint32_t taken = 0, ties = 0;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    taken |= (uint32_t)(keys[i] > cut) << i;
    ties |= (uint32_t)(keys[i] == cut) << i;
  }
  auto other_ranks = [&](int which) {  // the sum of the ranks before this one
    cluster_sync();
    int sum = 0;
    for (int r = 0; r < rank; ++r) sum += cluster_load(&sh.counts[which], r).x;
    return sum;
  };
  if (equals > 0) {
    int at = block_before<NT>(__popc(ties), sh.own.sums[1], all);
    if (threadIdx.x == 0) sh.counts[0].x = all;
    at += other_ranks(0);
    for (int x = __popc(ties); x > 0 && at + x > equals; --x) ties &= ~(1u << (31 - __clz(ties)));
    taken |= ties;
  }
  before = block_before<NT>(__popc(taken), sh.own.sums[0], all);
  if (threadIdx.x == 0) sh.counts[1].x = all;
  before += other_ranks(1);
  cluster_sync();  // (the last reads of others' shared memory)
  return taken;
}

// The same for any number n of items, with key(j) looked at again for every histogram: put(w,
// taken, before) gets the bits of items 32 w .. that are taken and how many are before them.
template <int NT, typename K, typename P>
__device__ __forceinline__ void pick_any(K key, int n, int k, PickShared<NT>& sh, P put) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int equals, all;
  const uint32_t cut = pick_cut<NT>(
      [&](auto add) {
#pragma unroll 4
        for (int j = threadIdx.x; j < n; j += NT) add(key(j));
      },
      k, sh, equals);
  int ties_before = 0, taken_before = 0;
#pragma unroll 1
  for (int base = 0; base < n; base += NT * 32) {
    uint32_t sure = 0, ties = 0;
#pragma unroll 4
    for (int i = 0; i < 32; ++i) {
      const int j0 = base + (warp * 32 + i) * 32;
      if (j0 >= n) break;
      const uint32_t x = j0 + lane < n ? key(j0 + lane) : 0;
      const uint32_t a = __ballot_sync(~0u, j0 + lane < n && x > cut);
      const uint32_t b = __ballot_sync(~0u, j0 + lane < n && x == cut);
      if (lane == i) sure = a, ties = b;
    }
    __syncthreads();
    const int at = ties_before + block_before<NT>(__popc(ties), sh.sums[1], all);
    ties_before += all;
    for (int x = __popc(ties); x > 0 && at + x > equals; --x) ties &= ~(1u << (31 - __clz(ties)));
    const uint32_t taken = sure | ties;
    const int before = taken_before + block_before<NT>(__popc(taken), sh.sums[0], all);
    taken_before += all;
    put(base / 32 + (int)threadIdx.x, taken, before);
  }
}

// ---- the same for 16 values of each thread, of rows of up to 16 NT items

constexpr int kShortWords = 4;  // of 128 items for each warp
constexpr int kShortList = 32;  // candidates that are compared with one another

template <int NT>
struct ShortPick {
  alignas(16) int hist[2][256];
  float list[kShortList], low_of[2][NT / 32], high_of[2][NT / 32];
  int listed, taken_of[NT / 32], ties_of[NT / 32];
  __device__ __forceinline__ void clear() {  // by the whole block, before a barrier
    for (int i = threadIdx.x; i < 128; i += NT) ((int4*)hist)[i] = make_int4(0, 0, 0, 0);
    if (threadIdx.x == 0) listed = 0;
  }
};

// A warp's words of 128 items; a lane has four adjacent ones of each.
template <int NT>
struct ShortRow {
  int c0, busy;  // the lane's first item, and the warp's words
  __device__ __forceinline__ explicit ShortRow(int n) {
    const int warp = threadIdx.x >> 5, words = (n + 127) / 128;
    const int run = (words + NT / 32 - 1) / (NT / 32);
    c0 = 128 * run * warp + 4 * (threadIdx.x & 31);
    busy = max(min(run, words - run * warp), 0);
  }
};

// Of n items the first `first`, the last `recent`, and the k others of the largest values v: put(c,
// before) for each that is taken, with how many are before it. `sh` is clear. By the whole block.
//
// One histogram of 256 bins, which divide the values between the least and the largest evenly, so
// that the bin of the k-th largest as a rule holds a few, which are compared with one another; else
// it is divided again, by the bits of the values' keys, which takes four rounds at most. 2560 rows
// of some 500 items: 13 us, 21 with pick_items (with bins by the first bits most scores of a row
// are in a few bins, whose counts come one after the other), 15 with a warp for a row.
// Instructions are what bounds it, so values stay floats (NaN as +inf), and only words with an item
// that is always taken, or past the last, look at each item's place.
template <int NT, typename F>
__device__ __forceinline__ void pick_short(float (&v)[kShortWords][4], const ShortRow<NT>& row,
                                           int n, int n_first, int n_recent, int k,
                                           ShortPick<NT>& sh, F put) {
  constexpr int kWarps = NT / 32, kWords = kShortWords, kAllTies = 0x7fffffff;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c0 = row.c0, busy = row.busy;
  // bits of the items that values decide, and of those that are always taken
  uint32_t free = 0, always = 0;
  float least = INFINITY, most = -INFINITY;
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    if (w >= busy) break;
    const int first = c0 - 4 * lane + 128 * w;
    uint32_t mine = 15;
    if (first < n_first || first + 128 > n - n_recent) {
      mine = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + 128 * w + i;
        const bool decides = c >= n_first && c < n - n_recent;
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
    if (lane == 0) sh.low_of[turn][warp] = least, sh.high_of[turn][warp] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      least = fminf(least, sh.low_of[turn][w]);
      most = fmaxf(most, sh.high_of[turn][w]);
    }
  };
  spread(0);
  // ---- the cut: values above it are taken, and the first `equals` of those equal to it
  float cut = INFINITY;
  int equals = 0;
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
    int* bins = sh.hist[turn];
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
          if (there <= kShortList) sh.list[atomicAdd(&sh.listed, 1)] = v[w][i];
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
      const float y = lane < there ? sh.list[lane] : 0.f;
      int above = 0, same = 0;
      for (int i = 0; i < there; ++i) {
        const float z = sh.list[i];
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
    if (lane == 0) sh.ties_of[warp] = mine;
    __syncthreads();
    int at = 0;
    for (int w = 0; w < warp; ++w) at += sh.ties_of[w];
    for (int w = 0; w < busy; ++w) {
      int all, before = at + before_in_word(ties, w, all);
      at += all;
      for (int i = 4 * w; i < 4 * w + 4; ++i)
        if (ties >> i & 1) taken |= (uint32_t)(before++ < equals) << i;
    }
  }
  const int mine = __reduce_add_sync(~0u, __popc(taken));
  if (lane == 0) sh.taken_of[warp] = mine;
  __syncthreads();
  int at = 0;
  for (int w = 0; w < warp; ++w) at += sh.taken_of[w];
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    if (w >= busy) break;
    int all, before = at + before_in_word(taken, w, all);
    at += all;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (taken >> (4 * w + i) & 1) put(c0 + 128 * w + i, before++);
  }
}

}  // namespace sv
