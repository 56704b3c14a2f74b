// The channels' extremes of each page's keys (spec_cache_bounds).
//
// lo_d = min over the page's held tokens of k_d, hi_d = max: packed 16-bit comparisons, exact.
// Bound by HBM: a page's keys read once, 4 dim bytes written for each of its heads. A block is
// one warp, which takes 512 bytes of each of a page's tokens at a time, a thread 8 channels of one
// head over all its tokens, sixteen of them loaded before the first is used. 785 pages of 64 tokens
// of 8 heads: 18.8 us, 15.4 at the rate of a copy; 25.5 with larger blocks, of which some SMs have
// one more than the others.
#pragma once
#include "sparse_common.cuh"

namespace sv {

constexpr int kBoundsThreads = 32, kBoundsAtOnce = 16;  // tokens in flight

struct BoundsParams {
  Requests rq;  // cu_q: NULL for all pages
  const char* k;
  long long k_page, k_token, k_head;  // bytes
  char* out;
  long long o_page, o_head, o_side;
  int pieces, row_pieces;  // 16-byte pieces of a head's row, and of a token's
  int chunks;              // of kBoundsThreads pieces of a token's row
  int spread;              // blocks of a request
};

template <bool BF16, bool MAX>
__device__ __forceinline__ uint32_t extreme2(uint32_t a, uint32_t b) {
  uint32_t r;
  if (BF16 && MAX) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  if (BF16 && !MAX) asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  if (!BF16 && MAX) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  if (!BF16 && !MAX) asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <bool BF16, bool MAX>
__device__ __forceinline__ void extreme8(uint4& a, uint4 b) {
  a.x = extreme2<BF16, MAX>(a.x, b.x);
  a.y = extreme2<BF16, MAX>(a.y, b.y);
  a.z = extreme2<BF16, MAX>(a.z, b.z);
  a.w = extreme2<BF16, MAX>(a.w, b.w);
}

template <bool BF16>
__global__ void __launch_bounds__(kBoundsThreads) k_cache_bounds(const BoundsParams p) {
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x / p.spread, x = blockIdx.x - b * p.spread;
  const int page_size = 1 << p.rq.page_shift;
  int from = 0, len;
  if (p.rq.cu_q) {
    int lo, hi;
    len = p.rq.request(b, lo, hi);
    if (hi == lo || len == 0) return;
    from = max(len - (hi - lo), 0) >> p.rq.page_shift;
  } else {
    len = p.rq.length(b);
  }
  const int columns = (int)(((long long)len + page_size - 1) >> p.rq.page_shift);
  const long long works = (long long)(columns - from) * p.chunks;
#pragma unroll 1
  for (long long w = x; w < works; w += p.spread) {
    const int c = from + (int)quotient(w, p.chunks);
    const int i = (int)(w - (long long)(c - from) * p.chunks) * kBoundsThreads + threadIdx.x;
    const int page = p.rq.page(b, c);
    if (page < 0) continue;
    const int n = min(page_size, len - (c << p.rq.page_shift));
    if (i < p.row_pieces) {
      const int head = i / p.pieces, piece = i - head * p.pieces;
      const char* src = p.k + page * p.k_page + head * p.k_head + piece * 16;
      uint4 low = *(const uint4*)src, high = low;
#pragma unroll 1
      for (int t = 0; t < n; t += kBoundsAtOnce) {
        uint4 v[kBoundsAtOnce];
#pragma unroll
        for (int y = 0; y < kBoundsAtOnce; ++y)  // (the last token again past the end)
          v[y] = *(const uint4*)(src + min(t + y, n - 1) * p.k_token);
#pragma unroll
        for (int y = 0; y < kBoundsAtOnce; ++y) {
          extreme8<BF16, false>(low, v[y]);
          extreme8<BF16, true>(high, v[y]);
        }
      }
      char* dst = p.out + page * p.o_page + head * p.o_head + piece * 16;
      *(uint4*)dst = low;
      *(uint4*)(dst + p.o_side) = high;
    }
  }
}

}  // namespace sv
