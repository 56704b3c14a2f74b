// Upper bounds of the pages' scores for the new tokens (spec_cache_score).
//
// With lo and hi a page's bounds of one kv head,
//   score = sum_g sum_d max(q_gd lo_d, q_gd hi_d) = P . hi + N . lo,
//   P_d = sum_g max(q_gd, 0),  N_d = sum_g min(q_gd, 0),
// so the heads of a group cost no more than one, and the scores are a product of the bounds
// (pages x 2 dim, 16 bits) with [N, P] (2 dim x tokens, fp32). It runs on the warp's tensor
// cores, 16 pages x 8 tokens at a time: P and N are scaled by powers of two for the types' ranges
// (score_shift), which are taken out again at the end, and split into three 16-bit parts that
// together hold 24 bits or more (33 of the largest in fp16), so the products are exact and the sums
// are fp32. The tensor cores cut their sums off, where an addition rounds, so that the error of a
// long chain grows with its length: the first parts' products are summed two instructions at a time
// and added up in registers (off by 4e-8 to 1e-7 in place of 5e-8 to 4e-7, for 2 % of the time).
//
// Bound by HBM: 4 dim bytes of bounds for each page and head, read once for up to 32 tokens, into
// registers (a warp has 16 pages, 8 KB at dim 128, in flight). A lane loads 16 bytes, 8 channels,
// of a row: the order of the channels in the sums is free, so they go into the products as they
// come, and [N, P] lies in shared memory in the same order.
//
// Work is one list of 16 columns for each group of tokens and kv head, with the start of a group
// counted in, cut into equal parts, one for each block: what a block has to do before its first
// product (find its part, split [N, P]) takes longer than some tens of columns. 64 requests of 2-8
// tokens over 1000-30000, 16-bit bounds of 8 heads: 36 us, 22 at the rate of a copy; 55 with a grid
// over groups, heads and thirds of the columns.
#pragma once
#include "sparse_common.cuh"

namespace sv {

constexpr int kScoreThreads = 128;
constexpr int kScoreGroup = 8;    // tokens of a product
constexpr int kScoreGroups = 4;   // of those in a group of tokens, at most
constexpr int kScoreBlocks = 4;   // of an SM
constexpr int kScorePart = 4;     // places of a block at least: one for each warp
constexpr int kScoreStart = 4;    // what the start of a unit counts: splitting [N, P]

struct ScoreParams {
  Requests rq;
  int heads, kv_heads, G, dim;
  const char* q;
  long long q_token, q_head;  // bytes
  const char* bounds;
  long long b_page, b_head, b_side;
  float* scores;
  long long s_token, s_head;
  int per;  // tokens of a group
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

// P and N are sums over up to 128 heads; of values 2^-8 of q's they stay under 2^127 for any q that
// is finite, and lose no bit (2^-149 holds the last one of 16-bit types' least values so).
constexpr int kScoreDown = 8;
constexpr float kScoreDownBy = 1.f / (1 << kScoreDown);

// The power of two that a token's P and N are multiplied by then, the largest of which is in
// [2^top, 2^(top + 1)), so that their parts are what the type holds. fp16 wants the largest in [2^14,
// 2^15): with bounds under 2^16 no sum of theirs is past 2^40. bf16 has fp32's range, and bounds of
// any size, so sums must not grow by it: nothing, but for top values under 2^-10, which go up to
// there (a sum of 2 dim products with bounds under 2^128 stays under 2^128 then), so that the
// parts of others a 2^-90th of them are still held.
template <bool BF16>
__device__ __forceinline__ int score_shift(int top) {
  if (!BF16) return min(max(14 - top, -100), 100);
  return top < -10 ? min(-10 - top, 100) : 0;
}

// What a request is in the list that the blocks divide: for each kv head and group of tokens
// kScoreStart places for the start, `reals` of 16 columns that some token may see, then `fills` of
// 128 that none does.
struct ScoreUnits {
  int lo, hi, len, groups, reals, fills;
  __device__ __forceinline__ ScoreUnits() {}
  __device__ __forceinline__ ScoreUnits(const ScoreParams& p, int b) {
    len = p.rq.request(b, lo, hi);
    groups = (hi - lo + p.per - 1) / p.per;
    const long long held = ((long long)len + (1 << p.rq.page_shift) - 1) >> p.rq.page_shift;
    reals = (int)((held + 15) / 16);
    fills = ((int)(((long long)p.rq.width + 15) / 16) - reals + 7) / 8;
  }
  __device__ __forceinline__ long long places(const ScoreParams& p) const {
    return (long long)groups * (kScoreStart + reals + fills) * p.kv_heads;
  }
};

template <int DP, bool BF16>
__global__ void __launch_bounds__(kScoreThreads, kScoreBlocks)
    k_cache_score(const ScoreParams p, const int run) {
  using Cfg = ScoreCfg<DP>;
  constexpr int kWarps = kScoreThreads / 32;
  extern __shared__ __align__(128) char smem[];
  __shared__ float unscale[kScoreGroups * kScoreGroup];
  __shared__ long long sums[kWarps], sh_at, sh_begin, sh_end;
  __shared__ int pads[kWarps], gap[kWarps], sh_first;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, x = lane >> 2, c = lane & 3;
  // ---- this block's part of the list
  TokenGroup idle = {};
  {
    const int r0 = (int)min((long long)tid * run, (long long)p.rq.B), r1 = min(r0 + run, p.rq.B);
    long long mine = 0;
    int pad = 0, gaps = 0;
    for (int r = r0; r < r1; ++r) {
      const ScoreUnits u(p, r);
      mine += u.places(p);
      pad = max(pad, u.hi);
      gaps |= u.lo < 0 || (r == 0 && u.lo > 0);
    }
    long long upto = mine;
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(~0u, upto, d);
      if (lane >= d) upto += y;
    }
    pad = __reduce_max_sync(~0u, pad);
    gaps = __any_sync(~0u, gaps);
    if (lane == 31) sums[warp] = upto;
    if (lane == 0) pads[warp] = pad, gap[warp] = gaps;
    if (tid == 0) sh_first = -1;
    __syncthreads();
    long long before = upto - mine, total = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sums[w];
      total += sums[w];
      idle.pad = max(idle.pad, pads[w]);
      idle.gaps |= gap[w];
    }
    const long long each = max(quotient(total + gridDim.x - 1, gridDim.x), (long long)kScorePart);
    const long long begin = each * blockIdx.x;
    if (before <= begin && begin < before + mine) {
      int r = r0;
      if (run > 1)
        for (;; ++r) {
          const long long n = ScoreUnits(p, r).places(p);
          if (begin < before + n || r + 1 >= r1) break;
          before += n;
        }
      sh_first = r;
      sh_at = before;
      sh_begin = begin;
      sh_end = min(begin + each, total);
    }
    __syncthreads();
  }
  int b = sh_first;
  if (b >= 0) {
    // walk: place `at` of request b, up to the end of the part
    long long left = sh_end - sh_begin, at = sh_begin - sh_at;
#pragma unroll 1
    while (left > 0) {
      const ScoreUnits u(p, b);
      const long long all = u.places(p);
      if (at >= all) {  // (the next request; the part does not end behind the last)
        at -= all;
        if (++b >= p.rq.B) break;
        continue;
      }
      const int per_unit = kScoreStart + u.reals + u.fills;
      const long long unit = quotient(at, per_unit);
      const int place = (int)(at - unit * per_unit);
      const int end = (int)min((long long)per_unit, place + left);
      left -= end - place;
      at += end - place;
      const int from = max(place - kScoreStart, 0), to = end - kScoreStart;
      if (to <= 0) continue;  // (the next part begins with the unit)
      const int head = (int)quotient(unit, u.groups);
      const int first = (int)(unit - (long long)head * u.groups) * p.per;
      const int tokens = min(p.per, u.hi - u.lo - first), token = u.lo + first;
      const int pos = u.len ? u.len - (u.hi - u.lo) + first : -(1 << 30);
      float* row = p.scores + (long long)token * p.s_token + head * p.s_head;
      // columns that nobody sees
      for (int i = max(from - u.reals, 0) + warp; i < to - u.reals; i += kWarps)
        for (int t = 0; t < tokens; ++t)
          for (int col = u.reals * 16 + i * 128 + lane;
               col < min((long long)p.rq.width, u.reals * 16ll + (i + 1) * 128ll); col += 32)
            row[t * p.s_token + col] = -INFINITY;
      if (from >= u.reals) continue;
      const int columns = (int)(((long long)u.len + (1 << p.rq.page_shift) - 1) >> p.rq.page_shift);
      // the page numbers of the lane's columns x and x + 8 of a place, which are looked up one
      // place ahead; -1: none
      auto look = [&](int i, int* page) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int col = 16 * i + x + 8 * r;
          page[r] = i < u.reals && col < columns ? p.rq.table[b * p.rq.table_stride + col] : -1;
        }
      };
      int next[2];
      look(from + warp, next);
      __syncthreads();  // (the unit before has been done with)
      // [N, P] of 8 tokens: a thread takes 8 channels of a token (DP / 8 <= 16 pieces)
      const int groups = (tokens + kScoreGroup - 1) / kScoreGroup;
      for (int i = tid; i < groups * kScoreGroup * 16; i += kScoreThreads) {
        const int tok = i >> 4, piece = i & 15;
        float up[8], down[8], top = 0.f;
#pragma unroll
        for (int y = 0; y < 8; ++y) up[y] = down[y] = 0.f;
        if (tok < tokens && piece * 8 < p.dim) {
          const char* src = p.q + (long long)(token + tok) * p.q_token +
                            (long long)head * p.G * p.q_head + piece * 16;
          for (int h = 0; h < p.G; ++h) {
            const uint4 v = *(const uint4*)(src + h * p.q_head);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const float2 f = unpack_pair<BF16>(w[y]);
              // (not fmaxf, which would take 0 in place of NaN)
              up[2 * y] = fmaf(f.x < 0.f ? 0.f : f.x, kScoreDownBy, up[2 * y]);
              up[2 * y + 1] = fmaf(f.y < 0.f ? 0.f : f.y, kScoreDownBy, up[2 * y + 1]);
              down[2 * y] = fmaf(f.x > 0.f ? 0.f : f.x, kScoreDownBy, down[2 * y]);
              down[2 * y + 1] = fmaf(f.y > 0.f ? 0.f : f.y, kScoreDownBy, down[2 * y + 1]);
            }
          }
#pragma unroll
          for (int y = 0; y < 8; ++y) top = fmaxf(top, fmaxf(up[y], -down[y]));
        }
        for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
        const int e = top > 0.f && top < INFINITY ? score_shift<BF16>(ilogbf(top)) : 0;
        const float scale = __uint_as_float((uint32_t)(127 + e) << 23);
        if (piece == 0)
          unscale[tok] = __uint_as_float((uint32_t)(127 - e + kScoreDown) << 23);
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
      const char* base = p.bounds + head * p.b_head + 16 * c;
      const bool there[4] = {8 * c < p.dim, 32 + 8 * c < p.dim, 64 + 8 * c < p.dim,
                             96 + 8 * c < p.dim};
#pragma unroll 1
      for (int i = from + warp; i < min(to, u.reals); i += kWarps) {
        const int col[2] = {16 * i + x, 16 * i + x + 8};
        bool live[2];
        uint4 a[2][Cfg::kChunks];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          live[r] = next[r] >= 0 && next[r] < p.rq.num_pages;
          if (col[r] < columns && !live[r]) atomicOr(p.rq.status, SPEC_CACHE_BAD_PAGE);
          const char* src = base + next[r] * p.b_page;
#pragma unroll
          for (int i = 0; i < Cfg::kChunks; ++i) {
            const int k = i % (Cfg::kChunks / 2);
            a[r][i] = live[r] && there[k]
                          ? *(const uint4*)(src + (i >= Cfg::kChunks / 2) * p.b_side + k * 64)
                          : make_uint4(0, 0, 0, 0);
          }
        }
        look(i + kWarps, next);
#pragma unroll 1
        for (int gr = 0; gr < groups; ++gr) {
          float d[4] = {}, low[4] = {};  // sums with the first parts, and with the two others
          const char* frag = smem + gr * Cfg::kGroupBytes + lane * 16;
#pragma unroll
          for (int i = 0; i < Cfg::kChunks; ++i) {
#pragma unroll
            for (int z = 0; z < 3; ++z) {
              const uint4 b = *(const uint4*)(frag + (i * 3 + z) * 512);
              if (z == 0) {
                float now[4];
                mma_16816_new<BF16>(now, a[0][i].x, a[1][i].x, a[0][i].y, a[1][i].y, b.x, b.y);
                mma_16816<BF16>(now, a[0][i].z, a[1][i].z, a[0][i].w, a[1][i].w, b.z, b.w);
#pragma unroll
                for (int y = 0; y < 4; ++y) d[y] += now[y];
              } else {
                mma_16816<BF16>(low, a[0][i].x, a[1][i].x, a[0][i].y, a[1][i].y, b.x, b.y);
                mma_16816<BF16>(low, a[0][i].z, a[1][i].z, a[0][i].w, a[1][i].w, b.z, b.w);
              }
            }
          }
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int tok = gr * kScoreGroup + 2 * c + (y & 1), r = y >> 1;
            if (tok >= tokens || col[r] >= p.rq.width) continue;
            const bool visible = live[r] && ((long long)col[r] << p.rq.page_shift) <= pos + tok;
            row[tok * p.s_token + col[r]] =
                visible ? (d[y] + low[y]) * unscale[tok] : -INFINITY;
          }
        }
      }
    }
  }
  for_idle_rows<kScoreThreads>(p.rq, idle, [&](int t) {
    for (int h = 0; h < p.kv_heads; ++h)
      for (int j = tid; j < p.rq.width; j += kScoreThreads)
        p.scores[t * p.s_token + h * p.s_head + j] = -INFINITY;
  });
}

}  // namespace sv
