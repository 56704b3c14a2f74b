// Upper bounds of the pages' scores for the new tokens (spec_cache_score).
//
// With lo and hi a page's bounds of one kv head,
//   score = sum_g sum_d max(q_gd lo_d, q_gd hi_d) = P . hi + N . lo,
//   P_d = sum_g max(q_gd, 0),  N_d = sum_g min(q_gd, 0),
// so the heads of a group cost no more than one, and the scores are a product of the bounds
// (pages x 2 dim, 16 bits) with [N, P] (2 dim x tokens, fp32). It runs on the warp's tensor
// cores, 16 pages x 8 tokens at a time: P and N are scaled by a power of two, which is taken out
// again at the end, and split into three 16-bit parts that together hold 24 bits or more (33 of
// the largest in fp16), so the products are exact and the sums are fp32.
//
// Bound by HBM: 4 dim bytes of bounds for each page and head, read once for up to 32 tokens, into
// registers (a warp has 16 pages, 8 KB at dim 128, in flight). A lane loads 16 bytes, 8 channels,
// of a row: the order of the channels in the sums is free, so they go into the products as they
// come, and [N, P] lies in shared memory in the same order.
#pragma once
#include "sparse_common.cuh"

namespace sv {

constexpr int kScoreThreads = 128;
constexpr int kScoreGroup = 8;    // tokens of a product
constexpr int kScoreGroups = 4;   // of those in a block, at most

struct ScoreParams {
  Requests rq;
  int heads, kv_heads, G, dim;
  const char* q;
  long long q_token, q_head;  // bytes
  const char* bounds;
  long long b_page, b_head, b_side;
  float* scores;
  long long s_token, s_head;
  int per;     // tokens of a block
  int spread;  // blocks of a group of tokens and a head
};

template <int DP>
struct ScoreCfg {
  static constexpr int kChunks = 2 * DP / 32;          // of 32 channels: lo's, then hi's
  static constexpr int kGroupBytes = kChunks * 3 * 512;  // [chunk][part][lane] 16 bytes
};

// Three 16-bit parts of x whose sum is x, but for 2^-24 of it.
template <bool BF16>
__device__ __forceinline__ void split3(float x, float* part) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const float2 y = unpack_pair<BF16>(pack_pair<BF16>(x, 0.f));
    part[i] = y.x;
    x = isinf(y.x) ? 0.f : x - y.x;
  }
}

template <int DP, bool BF16>
__global__ void __launch_bounds__(kScoreThreads) k_cache_score(const ScoreParams p) {
  using Cfg = ScoreCfg<DP>;
  extern __shared__ __align__(128) char smem[];
  __shared__ GroupShared<kScoreThreads> sh;
  __shared__ float unscale[kScoreGroups * kScoreGroup];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, x = lane >> 2, c = lane & 3;
  const int part = blockIdx.x % p.spread;
  const long long unit = blockIdx.x / p.spread / p.kv_heads;
  const int head = (int)(blockIdx.x / p.spread - unit * p.kv_heads);
  const TokenGroup g = find_group<kScoreThreads>(p.rq, unit, p.per, sh);
  if (g.b >= 0) {
    // [N, P] of 8 tokens: a thread takes 8 channels of a token (DP / 8 <= 16 pieces)
    const int groups = (g.tokens + kScoreGroup - 1) / kScoreGroup;
    for (int i = tid; i < groups * kScoreGroup * 16; i += kScoreThreads) {
      const int tok = i >> 4, piece = i & 15;
      float up[8], down[8], top = 0.f;
#pragma unroll
      for (int y = 0; y < 8; ++y) up[y] = down[y] = 0.f;
      if (tok < g.tokens && piece * 8 < p.dim) {
        const char* src = p.q + (long long)(g.token + tok) * p.q_token +
                          (long long)head * p.G * p.q_head + piece * 16;
        for (int h = 0; h < p.G; ++h) {
          const uint4 v = *(const uint4*)(src + h * p.q_head);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float2 f = unpack_pair<BF16>(w[y]);
            // (not fmaxf, which would take 0 in place of NaN)
            up[2 * y] += f.x < 0.f ? 0.f : f.x;
            up[2 * y + 1] += f.y < 0.f ? 0.f : f.y;
            down[2 * y] += f.x > 0.f ? 0.f : f.x;
            down[2 * y + 1] += f.y > 0.f ? 0.f : f.y;
          }
        }
#pragma unroll
        for (int y = 0; y < 8; ++y) top = fmaxf(top, fmaxf(up[y], -down[y]));
      }
      for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
      // 2^14 <= top * scale < 2^15; the least values need no more than 2^100
      int e = top > 0.f && top < INFINITY ? 14 - ilogbf(top) : 0;
      e = min(max(e, -100), 100);
      const float scale = __uint_as_float((uint32_t)(127 + e) << 23);
      if (piece == 0) unscale[tok] = __uint_as_float((uint32_t)(127 - e) << 23);
      if (piece * 8 < DP) {
        char* dst = smem + (tok >> 3) * Cfg::kGroupBytes + (piece >> 2) * 3 * 512 +
                    ((tok & 7) * 4 + (piece & 3)) * 16;
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          uint32_t w[3][4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            float a[3], b[3];
            split3<BF16>((side ? up : down)[2 * y] * scale, a);
            split3<BF16>((side ? up : down)[2 * y + 1] * scale, b);
#pragma unroll
            for (int z = 0; z < 3; ++z) w[z][y] = pack_pair<BF16>(a[z], b[z]);
          }
#pragma unroll
          for (int z = 0; z < 3; ++z)
            *(uint4*)(dst + side * (Cfg::kChunks / 2) * 3 * 512 + z * 512) =
                make_uint4(w[z][0], w[z][1], w[z][2], w[z][3]);
        }
      }
    }
    __syncthreads();
    const int last = g.pos + g.tokens - 1;  // position of the last token
    const int seen = last < 0 ? 0 : (last >> p.rq.page_shift) + 1;  // columns
    const char* base = p.bounds + head * p.b_head + 16 * c;
    const bool there[4] = {8 * c < p.dim, 32 + 8 * c < p.dim, 64 + 8 * c < p.dim,
                           96 + 8 * c < p.dim};
    float* row = p.scores + (long long)g.token * p.s_token + head * p.s_head;
    const int step = p.spread * (kScoreThreads / 32) * 16;
#pragma unroll 1
    for (long long col0 = ((long long)part * (kScoreThreads / 32) + warp) * 16; col0 < p.rq.width;
         col0 += step) {
      const int col[2] = {(int)col0 + x, (int)col0 + x + 8};
      bool live[2];
      uint4 a[2][Cfg::kChunks];
      if (col0 < seen) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int page = col[r] < seen ? p.rq.page(g.b, col[r]) : -1;
          live[r] = page >= 0;
          const char* src = base + page * p.b_page;
#pragma unroll
          for (int i = 0; i < Cfg::kChunks; ++i) {
            const int k = i % (Cfg::kChunks / 2);
            a[r][i] = live[r] && there[k]
                          ? *(const uint4*)(src + (i >= Cfg::kChunks / 2) * p.b_side + k * 64)
                          : make_uint4(0, 0, 0, 0);
          }
        }
      } else {
        live[0] = live[1] = false;
      }
#pragma unroll 1
      for (int gr = 0; gr < groups; ++gr) {
        float d[3][4] = {};  // sums of the three parts, the first parts' of lo apart
        if (col0 < seen) {
          const char* frag = smem + gr * Cfg::kGroupBytes + lane * 16;
          float d0[4] = {};
#pragma unroll
          for (int i = 0; i < Cfg::kChunks; ++i) {
#pragma unroll
            for (int z = 0; z < 3; ++z) {
              const uint4 b = *(const uint4*)(frag + (i * 3 + z) * 512);
              float* to = z == 0 && i < Cfg::kChunks / 2 ? d0 : d[z];
              mma_16816<BF16>(to, a[0][i].x, a[1][i].x, a[0][i].y, a[1][i].y, b.x, b.y);
              mma_16816<BF16>(to, a[0][i].z, a[1][i].z, a[0][i].w, a[1][i].w, b.z, b.w);
            }
          }
#pragma unroll
          for (int y = 0; y < 4; ++y) d[0][y] = d[0][y] + d0[y] + (d[1][y] + d[2][y]);
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int tok = gr * kScoreGroup + 2 * c + (y & 1), r = y >> 1;
          if (tok >= g.tokens || col[r] >= p.rq.width) continue;
          const bool visible =
              live[r] && ((long long)col[r] << p.rq.page_shift) <= g.pos + tok;
          row[tok * p.s_token + col[r]] = visible ? d[0][y] * unscale[tok] : -INFINITY;
        }
      }
    }
  }
  for_idle_rows<kScoreThreads>(p.rq, g, [&](int t) {
    for (int h = 0; h < p.kv_heads; ++h)
      for (int j = tid; j < p.rq.width; j += kScoreThreads)
        p.scores[t * p.s_token + h * p.s_head + j] = -INFINITY;
  });
}

}  // namespace sv
