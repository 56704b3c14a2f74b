// New tokens' keys and values to their cache slots (spec_cache_append).
//
// A copy with a scattered destination, bound by HBM: 4 * kv_heads * dim bytes
// read and as many written per token. A block takes TOKENS tokens; each of its
// threads takes one VEC-byte piece of the keys or the values at the same place
// of every token, so TOKENS loads are in flight per thread before the first
// store: 4 where that still leaves every SM blocks (50001 tokens of 8 heads of
// 128: 65.9 us, 6.2 TB/s, 0.92 of the measured copy rate), 1 in small calls
// (320 tokens: 2.4 us, launch and one round trip).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/spec_cache.h"
#include "pipe.cuh"

namespace sv {

constexpr int kAppendThreads = 256;

struct AppendParams {
  spec_cache_append_args a;  // strides in bytes
  unsigned* status;
  int pieces;       // VEC-byte pieces of a head's row
  int row_pieces;   // of a token's row
};

template <int VEC>
struct AppendPiece;
template <>
struct AppendPiece<16> {
  using type = uint4;
};
template <>
struct AppendPiece<2> {
  using type = unsigned short;
};

template <int VEC, int TOKENS>
__global__ void __launch_bounds__(kAppendThreads) k_cache_append(const AppendParams p) {
  using T = typename AppendPiece<VEC>::type;
  const spec_cache_append_args& a = p.a;
  __shared__ long long dst_k[TOKENS], dst_v[TOKENS];
  pdl_trigger();
  pdl_wait();
  const long long t0 = (long long)blockIdx.x * TOKENS;
  if (threadIdx.x < TOKENS) {
    const long long t = t0 + threadIdx.x;
    long long slot = t < a.num_tokens ? a.slots[t] : -1;
    if (slot >= 0 && slot / a.page_size >= a.num_pages) {
      atomicOr(p.status, SPEC_CACHE_BAD_SLOT);
      slot = -1;
    }
    const long long page = slot / a.page_size, at = slot - page * a.page_size;
    dst_k[threadIdx.x] = slot < 0 ? -1 : page * a.kp_page + at * a.kp_token;
    dst_v[threadIdx.x] = slot < 0 ? -1 : page * a.vp_page + at * a.vp_token;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * p.row_pieces; i += kAppendThreads) {
    const bool is_v = i >= p.row_pieces;
    const int piece = is_v ? i - p.row_pieces : i;
    const int head = piece / p.pieces, x = (piece - head * p.pieces) * VEC;
    const long long token = is_v ? a.v_token : a.k_token;
    const char* src = (const char*)(is_v ? a.v : a.k) + t0 * token +
                      head * (is_v ? a.v_head : a.k_head) + x;
    char* dst = (char*)(is_v ? a.v_pages : a.k_pages) + head * (is_v ? a.vp_head : a.kp_head) + x;
    const long long* at = is_v ? dst_v : dst_k;
    T got[TOKENS];
#pragma unroll
    for (int j = 0; j < TOKENS; ++j)
      if (at[j] >= 0) got[j] = *(const T*)(src + j * token);
#pragma unroll
    for (int j = 0; j < TOKENS; ++j)
      if (at[j] >= 0) *(T*)(dst + at[j]) = got[j];
  }
}

}  // namespace sv
