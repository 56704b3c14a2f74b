// Attention of new tokens over selected pages (spec_cache_attend_selected).
//
// The columns of a product are up to 8 tokens of one request times the query heads of one kv head
// (16 columns at most, or one token's, up to 32), the keys of the pages that any of the tokens
// selected are gone through once, and a byte for each page says which tokens see it:
//
//   S^T = K Q^T      16 keys x columns, on the warp's tensor cores, fp32
//   P = 2^(c S - m)  running maximum m and sum l of each column in fp32. m follows a higher
//                    maximum only when it has passed m by 2^8, as fp32 and the type allow (fp16's
//                    P starts at 2^7)
//   O^T += V^T P     dim x columns, fp32. The products take 16-bit operands, so P goes in as two
//                    parts of the cache's type, P cut off and what that left over: off by 2^-15
//                    (bf16) or 2^-21 (fp16) of itself. With one part, P rounded, the outputs are
//                    off by 2.0e-3 to 2.3e-3 where 1.7e-3 are their own rounding (bf16), and
//                    calls take 2 to 13 % less (64 requests of 2-8 tokens: 166 us in place of
//                    176). Neither part of a P above 0 is 0 or negative (2^-23 of P is added to the
//                    second), so that an infinite value stays infinite
//
// With c = scale * log2(e). Keys as the rows leave no tensor-core row empty however few columns
// there are; P^T gets from a product's layout of sums to that of an operand by a transposition of
// 8 x 8 values in registers.
//
// Each warp has its own ring of tiles of 16 keys and values, filled by 16-byte asynchronous
// copies, and its own softmax statistics, and waits for no other warp until the end: a block's
// warps, then a cluster's blocks through each other's shared memory, join their parts. Slots that
// no token sees are not loaded; zeros stand in their place. What one token of a unit sees meets the
// others with P = 0, which keeps finite values out of their sums, but not infinities and NaN.
//
// Bound by HBM where the selections of a request's tokens agree, by the latency of the chain
// (requests, list, pages, keys, join) in small calls.
#pragma once
#include "sparse_common.cuh"

namespace sv {

constexpr int kSelList = 640;    // pages that a block lists at a time
constexpr int kSelTokens = 8;    // bits of a page's byte

struct SelectedParams {
  Requests rq;
  int heads, kv_heads, G, dim;
  const char* q;
  long long q_token, q_head;  // bytes
  const char* k;
  long long k_page, k_token, k_head;
  const char* v;
  long long v_page, v_token, v_head;
  const int* selected;
  int count;
  char* out;
  long long out_token, out_head;
  float* lse;
  float c;        // scale * log2(e)
  int per;        // tokens of a unit
  int unit_heads, splits;  // query heads of a unit, and units that share a kv head's
  int cluster;    // blocks of a unit
};

template <int DP, int N8, bool DEEP>
struct SelCfg {
  // Four warps with two tiles each and three blocks on an SM, or three tiles and two blocks where
  // the registers do not allow three: twelve warps hide latency better than eight with more tiles
  // in flight (64 requests of 2-8 tokens over 128 pages of 16: 176 us in place of 193). DEEP: eight
  // warps with three tiles each, for calls that leave most of the SMs idle.
  static constexpr int kWarps = DEEP ? 8 : 4, kThreads = 32 * kWarps;
  static constexpr int kStages = !DEEP && N8 <= 2 ? 2 : 3, kBlocks = DEEP ? 1 : N8 <= 2 ? 3 : 2;
  static constexpr int kTile = 16 * DP * 2;                       // bytes of 16 keys
  static constexpr int kRing = kWarps * kStages * 2 * kTile;
  static constexpr int kQ = N8 * (DP / 16) * 256;                 // [n8][step][lane] 8 bytes
  static constexpr int kCols = 8 * N8;
  static constexpr int kPitch = DP + 4;                           // floats of a column's partial O
  static constexpr int kSmem = kRing + kQ + kSelList * 9;
  static_assert(kBlocks * (kSmem + 2048) <= 228 * 1024, "blocks of an SM");
  static_assert((kWarps + 1) * kCols * (kPitch + 2) * 4 <= kRing, "partial results in the ring");
};

// 16 bytes to shared memory: `bytes` (0 or 16) from src, zeros for the others.
__device__ __forceinline__ void copy16(uint32_t dst, const char* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <bool TRANS>
__device__ __forceinline__ void load_matrix4(uint32_t* r, uint32_t at) {
  if (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// 2^(a - b) for maxima a <= b, of which a may be -inf.
__device__ __forceinline__ float weight_of(float a, float b) {
  return a == -INFINITY ? 0.f : ex2(a - b);
}

template <bool BF16>
__device__ constexpr float sel_bias() {  // log2 of what P and l carry beside 2^-m
  return BF16 ? 0.f : 7.f;
}

struct SelList {
  int* page;
  int* col;
  unsigned char* mask;
};

template <int DP, int N8, bool DEEP, bool BF16>
__global__ void __launch_bounds__(SelCfg<DP, N8, DEEP>::kThreads, SelCfg<DP, N8, DEEP>::kBlocks)
    k_attend_selected(const __grid_constant__ SelectedParams p) {
  using Cfg = SelCfg<DP, N8, DEEP>;
  constexpr int kWarps = Cfg::kWarps, kThreads = Cfg::kThreads;
  constexpr float kBias = sel_bias<BF16>();
  constexpr float kNone = -3e38f;       // the maximum of no score: finite, so that P is 0
  constexpr float kUp = 1.f + 1.f / (1 << 23);  // (the next above 1)
  constexpr int kLanes = DP / 8;        // lanes that copy a row's 16-byte pieces
  constexpr int kRows = 32 / kLanes;    // rows of one copy instruction
  extern __shared__ __align__(128) char smem[];
  __shared__ GroupShared<kThreads> sh;
  __shared__ int sums[kWarps], listed;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, x = lane >> 2, c = lane & 3;
  const int rank = p.cluster > 1 ? blockIdx.x % p.cluster : 0;
  long long unit = blockIdx.x / p.cluster;
  const int split = (int)(unit % p.splits);
  unit /= p.splits;
  const int kv_head = (int)(unit % p.kv_heads);
  unit /= p.kv_heads;
  const TokenGroup g = find_group<kThreads>(p.rq, unit, p.per, sh);
  if (g.b >= 0) {
    char* ring = smem + warp * Cfg::kStages * 2 * Cfg::kTile;
    const uint32_t ring_at = smem_addr(ring);
    uint2* q_frag = (uint2*)(smem + Cfg::kRing);
    SelList list;
    list.page = (int*)(smem + Cfg::kRing + Cfg::kQ);
    list.col = list.page + kSelList;
    list.mask = (unsigned char*)(list.col + kSelList);
    const int shift = p.rq.page_shift, page_size = 1 << shift;
    const int head0 = kv_head * p.G + split * p.unit_heads;
    const int heads = min(p.unit_heads, p.G - split * p.unit_heads);
    const int columns = g.tokens * heads;
    const int steps = (p.dim + 15) / 16, pieces = p.dim / 8;
    const float factor = fabsf(p.c);
    const uint32_t flip = p.c < 0.f ? 0x80008000u : 0u;
    // the tokens of the lane's columns, a byte with one bit for each (none: no such column)
    uint32_t token_of[(2 * N8 + 3) / 4] = {};
#pragma unroll
    for (int y = 0; y < 2 * N8; ++y) {
      const int column = (y >> 1) * 8 + 2 * c + (y & 1);
      if (column < columns) token_of[y / 4] |= 1u << (column / heads + 8 * (y & 3));
    }
    const uint32_t everyone = (1u << g.tokens) - 1;
    const int last = g.pos + g.tokens - 1;                       // the last token's position
    const int visible = last < 0 ? 0 : (last >> shift) + 1;      // columns it sees
    const int* lists = p.selected + ((long long)g.token * p.kv_heads + kv_head) * p.count;
    const long long next_list = (long long)p.kv_heads * p.count;

    float m[N8][2], l[N8][2], o[DP / 16][N8][4];
#pragma unroll
    for (int n = 0; n < N8; ++n) {
      m[n][0] = m[n][1] = kNone;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int y = 0; y < DP / 16; ++y) o[y][n][0] = o[y][n][1] = o[y][n][2] = o[y][n][3] = 0.f;
    }
    // Entry i of token k's list, which follows `before`, as a visible column, or -1. (Broken lists
    // are told of once.)
    auto checked = [&](int k, int i, int col, int before) {
      if (col < 0 || g.len == 0) return -1;
      if ((i > 0 && (before < 0 || before >= col)) ||
          ((long long)col << shift) >= g.len) {
        atomicOr(p.rq.status, SPEC_CACHE_BAD_SELECTION);
        return -1;
      }
      return col < visible && ((long long)col << shift) <= g.pos + k ? col : -1;
    };
    // the lane's place in a copy of rows: 16 bytes of a key
    const int piece = lane & (kLanes - 1), lane_row = lane / kLanes;
    const bool copies = piece < pieces;
    const char* k_lane = p.k + kv_head * p.k_head + lane_row * p.k_token + piece * 16;
    const char* v_lane = p.v + kv_head * p.v_head + lane_row * p.v_token + piece * 16;
    uint32_t lane_dst[8 / kRows];
#pragma unroll
    for (int y = 0; y < 8 / kRows; ++y) {
      const int r = y * kRows + lane_row;
      lane_dst[y] = r * (DP * 2) + ((piece ^ r) & 7) * 16 + (piece & 8) * 16;
    }
    const bool one = g.tokens == 1;
    // The lists (of one token's the start), Q and a first page's number, each on its way while
    // the others are waited for. Q as operands: two channels of one column at a time.
    constexpr int kEntries = (kSelList + kThreads - 1) / kThreads;
    int entries[kEntries], befores[kEntries];
#pragma unroll
    for (int y = 0; y < kEntries; ++y) {
      const int i = tid + y * kThreads;
      const bool there = i < kSelList && i < g.tokens * p.count;
      const int k = one ? 0 : i / p.count, at = i - k * p.count;
      const int* row = lists + k * next_list + at;
      entries[y] = there ? row[0] : -1;
      befores[y] = there && at > 0 ? row[-1] : -1;
    }
    constexpr int kQs = (N8 * (DP / 16) * 32 + kThreads - 1) / kThreads;
    uint2 qs[kQs];
#pragma unroll
    for (int y = 0; y < kQs; ++y) {
      const int i = tid + y * kThreads, n8 = i / ((DP / 16) * 32), step = i / 32 % (DP / 16);
      const int column = n8 * 8 + (i >> 2 & 7), ch = step * 16 + 2 * (i & 3);
      qs[y] = make_uint2(0, 0);
      if (n8 < N8 && column < columns) {
        const int tok = column / heads;
        const char* src = p.q + (long long)(g.token + tok) * p.q_token +
                          (long long)(head0 + column - tok * heads) * p.q_head + ch * 2;
        if (ch < p.dim) qs[y].x = *(const uint32_t*)src;
        if (ch + 8 < p.dim) qs[y].y = *(const uint32_t*)(src + 16);
      }
    }
#pragma unroll
    for (int y = 0; y < kEntries; ++y) {
      const int i = tid + y * kThreads, k = one ? 0 : i / p.count;
      entries[y] = checked(k, i - k * p.count, entries[y], befores[y]);
    }
    const int* table = p.rq.table + g.b * p.rq.table_stride;
    const int page0 = one && entries[0] >= 0 ? table[entries[0]] : -1;
#pragma unroll
    for (int y = 0; y < kQs; ++y)  // (a negative factor of the scores is Q's sign)
      if (tid + y * kThreads < N8 * (DP / 16) * 32)
        q_frag[tid + y * kThreads] = make_uint2(qs[y].x ^ flip, qs[y].y ^ flip);
    // One token's list is taken in parts of what the block lists at a time; of several tokens
    // the host made sure that all their pages fit.
    for (int part = 0; part < (one ? p.count : 1); part += kSelList) {
      __syncthreads();  // (the list before has been used)
      if (tid == 0) listed = 0;
      __syncthreads();
      if (one) {
        int top = 0;
#pragma unroll
        for (int y = 0; y < kEntries; ++y) {
          const int i = tid + y * kThreads;
          if (i >= kSelList || part + i >= p.count) break;
          int col = entries[y];
          if (part > 0)
            col = checked(0, part + i, lists[part + i], lists[part + i - 1]);
          int page = part == 0 && y == 0 ? page0
                     : col >= 0          ? p.rq.table[g.b * p.rq.table_stride + col]
                                         : -1;
          if (col >= 0 && (page < 0 || page >= p.rq.num_pages)) {
            atomicOr(p.rq.status, SPEC_CACHE_BAD_PAGE);
            page = -1;
          }
          list.col[i] = col;
          list.page[i] = page;
          list.mask[i] = col >= 0;
          if (col >= 0) top = i + 1;
        }
        top = __reduce_max_sync(~0u, top);
        if (lane == 0) atomicMax(&listed, top);
      } else {
        // a byte for each visible column, over the ring; then the bytes that are not 0 in order
        uint32_t* bytes = (uint32_t*)smem;
        const int words = (visible + 3) / 4, run = (words + kThreads - 1) / kThreads;
        for (int i = tid; i < words; i += kThreads) bytes[i] = 0;
        __syncthreads();
#pragma unroll
        for (int y = 0; y < kEntries; ++y) {
          const int col = entries[y], k = (tid + y * kThreads) / p.count;
          if (col >= 0) atomicOr(&bytes[col >> 2], 1u << (8 * (col & 3) + k));
        }
        __syncthreads();
        const int w0 = min(tid * run, words), w1 = min(w0 + run, words);
        int n = 0;
        for (int i = w0; i < w1; ++i) n += __popc(__vcmpgtu4(bytes[i], 0)) / 8;
        int all;
        int at = block_before<kThreads>(n, sums, all);
        for (int i = w0; i < w1; ++i)
          for (uint32_t w = bytes[i], y = 0; w; w >>= 8, ++y)
            if (w & 255) {
              list.col[at] = 4 * i + y;
              list.mask[at] = w & 255;
              ++at;
            }
        __syncthreads();
        for (int i = tid; i < all; i += kThreads) list.page[i] = p.rq.page(g.b, list.col[i]);
        if (tid == 0) listed = all;
      }
      __syncthreads();
      const int n = listed;
      if (p.dim % 16) {  // channels that the products take beside those that there are
        for (int i = lane; i < 2 * Cfg::kStages * Cfg::kTile / 16; i += 32)
          *(uint4*)(ring + 16 * i) = make_uint4(0, 0, 0, 0);
        __syncwarp();
      }
      const int tiles = (n * page_size + 15) / 16;
      const int from = rank * kWarps + warp, step = p.cluster * kWarps;
      // of key lane % 16 of the tiles in flight: bits of tokens, the youngest tile's lowest
      unsigned long long seen_by = 0;
      auto issue = [&](int tile, int stage) {
        uint32_t mine = 0;
        if (tile < tiles) {
          // the lane's key (lanes 16 and up have those of 0 to 15 again), and who sees it
          const int key = 16 * tile + (lane & 15), e = key >> shift;
          int page = -1;
          if (e < n) {
            page = list.page[e];
            const int ahead = (int)(((long long)list.col[e] << shift) +
                                    (key & (page_size - 1)) - g.pos);
            if (page >= 0 && ahead < kSelTokens)
              mine = list.mask[e] & (everyone << max(ahead, 0));
          }
          const uint32_t seen = __ballot_sync(~0u, mine != 0) >> (lane / kLanes);
          const uint32_t dst = ring_at + stage * 2 * Cfg::kTile;
#pragma unroll
          for (int half = 0; half < 2; ++half) {  // 8 keys of one page
            const long long at = max(__shfl_sync(~0u, page, 8 * half), 0);
            const int off = (16 * tile + 8 * half) & (page_size - 1);
            const char* ks = k_lane + at * p.k_page + off * p.k_token;
            const char* vs = v_lane + at * p.v_page + off * p.v_token;
            if (copies) {
#pragma unroll
              for (int y = 0; y < 8 / kRows; ++y) {
                const uint32_t bytes = seen >> (8 * half + y * kRows) << 4 & 16;
                copy16(dst + lane_dst[y] + 8 * half * (DP * 2), ks, bytes);
                copy16(dst + lane_dst[y] + 8 * half * (DP * 2) + Cfg::kTile, vs, bytes);
                ks += kRows * p.k_token;
                vs += kRows * p.v_token;
              }
            }
          }
        }
        seen_by = seen_by << 8 | mine;
        copy_commit();
      };
#pragma unroll
      for (int i = 0; i < Cfg::kStages - 1; ++i) issue(from + i * step, i);
      int stage = 0;
#pragma unroll 1
      for (int tile = from; tile < tiles; tile += step) {
        copy_wait<Cfg::kStages - 2>();
        __syncwarp();
        issue(tile + (Cfg::kStages - 1) * step, stage == 0 ? Cfg::kStages - 1 : stage - 1);
        const uint32_t seen = (uint32_t)(seen_by >> (8 * (Cfg::kStages - 1))) & 255;
        const uint32_t k_at = ring_at + stage * 2 * Cfg::kTile, v_at = k_at + Cfg::kTile;
        stage = stage == Cfg::kStages - 1 ? 0 : stage + 1;
        float s[N8][4];
#pragma unroll
        for (int n8 = 0; n8 < N8; ++n8) s[n8][0] = s[n8][1] = s[n8][2] = s[n8][3] = 0.f;
#pragma unroll
        for (int y = 0; y < DP / 16; ++y) {
          if (y >= steps) break;
          uint32_t a[4];
          const int r = lane & 15, piece = 2 * y + (lane >> 4);
          load_matrix4<false>(a, k_at + r * (DP * 2) + ((piece ^ r) & 7) * 16 + (piece & 8) * 16);
#pragma unroll
          for (int n8 = 0; n8 < N8; ++n8) {
            const uint2 b = q_frag[(n8 * (DP / 16) + y) * 32 + lane];
            mma_16816<BF16>(s[n8], a[0], a[1], a[2], a[3], b.x, b.y);
          }
        }
        if (!__all_sync(~0u, seen == everyone)) {
          const uint32_t k0 = __shfl_sync(~0u, seen, x) * 0x01010101u;
          const uint32_t k1 = __shfl_sync(~0u, seen, x + 8) * 0x01010101u;
#pragma unroll
          for (int y = 0; y < 2 * N8; ++y) {
            const uint32_t bits = token_of[y / 4] & 255u << (8 * (y & 3));
            if (!(k0 & bits)) s[y >> 1][y & 1] = -INFINITY;
            if (!(k1 & bits)) s[y >> 1][(y & 1) + 2] = -INFINITY;
          }
        }
        bool grown = false;
#pragma unroll
        for (int n8 = 0; n8 < N8; ++n8)
#pragma unroll
          for (int y = 0; y < 2; ++y)
            grown |= fmaf(fmaxf(s[n8][y], s[n8][y + 2]), factor, -m[n8][y]) > 8.f;
        if (__any_sync(~0u, grown)) {
#pragma unroll
          for (int n8 = 0; n8 < N8; ++n8)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              float top = fmaxf(s[n8][y], s[n8][y + 2]);
              for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
              top = top == -INFINITY ? m[n8][y] : fmaxf(top * factor, m[n8][y]);
              const float keep = m[n8][y] == kNone ? 0.f : ex2(m[n8][y] - top);
              m[n8][y] = top;
              l[n8][y] *= keep;
#pragma unroll
              for (int z = 0; z < DP / 16; ++z) o[z][n8][y] *= keep, o[z][n8][y + 2] *= keep;
            }
        }
        uint32_t b[N8][2], rest[N8][2];
#pragma unroll
        for (int n8 = 0; n8 < N8; ++n8) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            s[n8][y] = ex2(fmaf(s[n8][y], factor, kBias - m[n8][y]));
            s[n8][y + 2] = ex2(fmaf(s[n8][y + 2], factor, kBias - m[n8][y]));
            l[n8][y] += s[n8][y] + s[n8][y + 2];
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float p0 = s[n8][2 * y], p1 = s[n8][2 * y + 1];
            const uint32_t high = pack_pair_down<BF16>(p0, p1);
            const float2 h = unpack_pair<BF16>(high);
            b[n8][y] = transposed(high);
            rest[n8][y] = transposed(pack_pair<BF16>(fmaf(p0, kUp, -h.x), fmaf(p1, kUp, -h.y)));
          }
        }
#pragma unroll
        for (int y = 0; y < DP / 16; ++y) {
          if (y >= steps) break;
          uint32_t a[4];
          const int r = (lane & 7) + (lane >> 4) * 8, piece = 2 * y + (lane >> 3 & 1);
          load_matrix4<true>(a, v_at + r * (DP * 2) + ((piece ^ r) & 7) * 16 + (piece & 8) * 16);
#pragma unroll
          for (int n8 = 0; n8 < N8; ++n8)
            mma_16816<BF16>(o[y][n8], a[0], a[1], a[2], a[3], b[n8][0], b[n8][1]);
#pragma unroll
          for (int n8 = 0; n8 < N8; ++n8)
            mma_16816<BF16>(o[y][n8], a[0], a[1], a[2], a[3], rest[n8][0], rest[n8][1]);
        }
      }
      copy_wait<0>();
    }
    // ---- join: the block's warps
    __syncthreads();
    float* part_o = (float*)smem;                                     // [warp][column][pitch]
    float* all_o = part_o + kWarps * Cfg::kCols * Cfg::kPitch;     // the block's
    float* part_m = all_o + Cfg::kCols * Cfg::kPitch;                 // [warp + 1][column]
    float* part_l = part_m + (kWarps + 1) * Cfg::kCols;
    float* all_m = part_m + kWarps * Cfg::kCols;
    float* all_l = part_l + kWarps * Cfg::kCols;
#pragma unroll
    for (int n8 = 0; n8 < N8; ++n8)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float sum = l[n8][y];
        for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(~0u, sum, d);
        const int column = n8 * 8 + 2 * c + y;
        if (x == 0) {
          part_m[warp * Cfg::kCols + column] = m[n8][y] == kNone ? -INFINITY : m[n8][y];
          part_l[warp * Cfg::kCols + column] = sum;
        }
        float* to = part_o + (warp * Cfg::kCols + column) * Cfg::kPitch + x;
#pragma unroll
        for (int z = 0; z < DP / 16; ++z) {
          to[16 * z] = o[z][n8][y];
          to[16 * z + 8] = o[z][n8][y + 2];
        }
      }
    __syncthreads();
    const int pairs = p.dim / 2;
    auto put = [&](int column, int d, float a, float b, float top, float sum) {
      const int tok = column / heads;
      const long long t = g.token + tok;
      const int head = head0 + column - tok * heads;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      *(uint32_t*)(p.out + t * p.out_token + head * p.out_head + 4 * d) =
          pack_pair<BF16>(a * inv, b * inv);
      if (d == 0 && p.lse)
        p.lse[t * p.heads + head] =
            sum == 0.f ? -INFINITY : (top + log2f(sum) - kBias) * 0.69314718055994531f;
    };
    for (int i = tid; i < columns * pairs; i += kThreads) {
      const int column = i / pairs, d = i - column * pairs;
      float top = -INFINITY, sum = 0.f, a = 0.f, b = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part_m[w * Cfg::kCols + column]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = weight_of(part_m[w * Cfg::kCols + column], top);
        const float2 y =
            *(const float2*)(part_o + (w * Cfg::kCols + column) * Cfg::kPitch + 2 * d);
        sum += f * part_l[w * Cfg::kCols + column];
        a += f * y.x;
        b += f * y.y;
      }
      if (p.cluster == 1) {
        put(column, d, a, b, top, sum);
      } else {
        *(float2*)(all_o + column * Cfg::kPitch + 2 * d) = make_float2(a, b);
        if (d == 0) all_m[column] = top, all_l[column] = sum;
      }
    }
    // ---- the cluster's blocks, each a part of the results
    if (p.cluster > 1) {
      cluster_sync();
      for (int i = tid + rank * kThreads; i < columns * pairs; i += p.cluster * kThreads) {
        const int column = i / pairs, d = i - column * pairs;
        float m[8], l[8], top = -INFINITY, sum = 0.f, a = 0.f, b = 0.f;
        float2 o[8];
#pragma unroll
        for (int w = 0; w < 8; ++w) {  // (the cluster is a power of two: others are read again)
          const int from = w & (p.cluster - 1);
          m[w] = cluster_load(all_m + column, from);
          l[w] = cluster_load(all_l + column, from);
          o[w] = cluster_load((const float2*)(all_o + column * Cfg::kPitch + 2 * d), from);
        }
#pragma unroll
        for (int w = 0; w < 8; ++w) top = fmaxf(top, m[w]);
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          if (w >= p.cluster) break;
          const float f = weight_of(m[w], top);
          sum += f * l[w];
          a += f * o[w].x;
          b += f * o[w].y;
        }
        put(column, d, a, b, top, sum);
      }
      cluster_sync();
    }
  }
  for_idle_rows<kThreads>(p.rq, g, [&](int t) {
    const int pieces = p.dim / 8;
    for (int i = tid; i < p.heads * pieces; i += kThreads)
      *(uint4*)(p.out + t * p.out_token + (i / pieces) * p.out_head + (i % pieces) * 16) =
          make_uint4(0, 0, 0, 0);
    if (p.lse)
      for (int i = tid; i < p.heads; i += kThreads) p.lse[(long long)t * p.heads + i] = -INFINITY;
  });
}

}  // namespace sv
