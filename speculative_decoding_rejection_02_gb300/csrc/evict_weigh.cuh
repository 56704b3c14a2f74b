// The softmax weights that the new tokens give the cached ones (spec_cache_weigh).
//
//   w_j = (old ? decay w_j : 0) + sum over columns 2^(c q . k_j - lse log2(e)),  c = scale log2(e)
//
// where a column is a new token and one of its query heads on the kv head. A key's sum needs no
// other key, so a warp takes 16 keys, has them in registers as operands, and goes over the
// columns, 8 at a time; the 16 sums are fp32, in an order that does not depend on the call's
// other requests. A lane loads 16 bytes, 8 channels, of a row: the order of the channels in the
// products' sums is free, so they are taken as they come.
//
// Bound by HBM (the keys, once) for few columns, by the columns' reloads from L2 for many.
#pragma once
#include "sparse_common.cuh"

namespace sv {

constexpr int kWeighThreads = 128;

struct WeighParams {
  Requests rq;
  int heads, kv_heads, G, dim;
  const char* q;
  long long q_token, q_head;  // bytes
  const char* k;
  long long k_page, k_token, k_head;
  const float* lse;
  float* weights;
  long long w_page, w_head;  // elements
  float c, decay;
  int spread;  // blocks of a request and a kv head
};

template <int DP, bool BF16>
__global__ void __launch_bounds__(kWeighThreads) k_cache_weigh(const WeighParams p) {
  constexpr int kChunks = DP / 32;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, x = lane >> 2, c = lane & 3;
  const int part = blockIdx.x % p.spread, unit = blockIdx.x / p.spread;
  const int b = unit / p.kv_heads, head = unit - b * p.kv_heads;
  int lo, hi;
  const int len = p.rq.request(b, lo, hi);
  if (hi == lo) return;
  const int old = len - (hi - lo);  // position of the first new token
  const int columns = (hi - lo) * p.G;  // (at most T * heads)
  const char* q = p.q + (long long)lo * p.q_token + (long long)head * p.G * p.q_head + 16 * c;
  const float* lse = p.lse + (long long)lo * p.heads + head * p.G;
  const int step = p.spread * (kWeighThreads / 32) * 16;
#pragma unroll 1
  for (long long j0 = (part * (kWeighThreads / 32) + warp) * 16; j0 < len; j0 += step) {
    const int key[2] = {(int)j0 + x, (int)j0 + x + 8};
    uint4 a[2][kChunks];
    float* w[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int page = key[r] < len ? p.rq.page(b, key[r] >> p.rq.page_shift) : -1;
      const int at = key[r] & ((1 << p.rq.page_shift) - 1);
      const char* src = p.k + page * p.k_page + at * p.k_token + head * p.k_head + 16 * c;
      w[r] = page < 0 ? nullptr : p.weights + page * p.w_page + head * p.w_head + at;
#pragma unroll
      for (int i = 0; i < kChunks; ++i)
        a[r][i] = page >= 0 && 32 * i + 8 * c < p.dim ? *(const uint4*)(src + 64 * i)
                                                      : make_uint4(0, 0, 0, 0);
    }
    float sum[2] = {0.f, 0.f};
    // the first column that sees a key here
    const int from = j0 > old ? (int)min((j0 - old) * p.G, (long long)columns) & ~7 : 0;
#pragma unroll 1
    for (int col0 = from; col0 < columns; col0 += 8) {
      const int mine = col0 + x, tok = mine / p.G;
      const char* src = q + (long long)tok * p.q_token + (long long)(mine - tok * p.G) * p.q_head;
      float d[4] = {};
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const uint4 v = mine < columns && 32 * i + 8 * c < p.dim ? *(const uint4*)(src + 64 * i)
                                                                 : make_uint4(0, 0, 0, 0);
        mma_16816<BF16>(d, a[0][i].x, a[1][i].x, a[0][i].y, a[1][i].y, v.x, v.y);
        mma_16816<BF16>(d, a[0][i].z, a[1][i].z, a[0][i].w, a[1][i].w, v.z, v.w);
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int col = col0 + 2 * c + y, tok = col / p.G;
        if (col >= columns) continue;
        const float z = lse[(long long)tok * p.heads + col - tok * p.G];
        const float shift = z == -INFINITY ? INFINITY : z * 1.4426950408889634f;
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (key[r] <= old + tok) sum[r] += ex2(d[2 * r + y] * p.c - shift);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      sum[r] += __shfl_xor_sync(~0u, sum[r], 1);
      sum[r] += __shfl_xor_sync(~0u, sum[r], 2);
      if (c == 0 && w[r])
        *w[r] = sum[r] + (key[r] < old && p.decay != 0.f ? p.decay * *w[r] : 0.f);
    }
  }
}

}  // namespace sv
