// Attention of a round's new tokens over the paged cache (spec_cache_attend).
//
// The plainest form: one block per new token and query head, whose warps take
// the visible tokens in turn and keep a running maximum, sum and output each,
// joined at the end.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/spec_cache.h"
#include "pipe.cuh"

namespace sv {

struct AttendParams {
  spec_cache_attend_args a;
  unsigned* status;
  int page_shift;
};

constexpr int kAttendWarps = 4;

__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16& y) { y = __float2bfloat16(x); }
__device__ __forceinline__ void from_f32(float x, __half& y) { y = __float2half(x); }

// The new tokens of request b as rows [lo, hi) of q, and its length; a request
// whose offsets or length cannot be has length 0.
__device__ __forceinline__ int attend_request(const AttendParams& p, int b, int& lo, int& hi) {
  const spec_cache_attend_args& a = p.a;
  lo = a.cu_q[b];
  hi = a.cu_q[b + 1];
  int len = a.kv_lens[b];
  const bool bad = lo < 0 || hi < lo || hi > a.num_tokens || len < 0 ||
                   len > ((long long)a.width << p.page_shift);
  if (bad) {
    if (p.status) atomicOr(p.status, SPEC_CACHE_BAD_LENGTHS);
    lo = min(max(lo, 0), a.num_tokens);
    hi = min(max(hi, lo), a.num_tokens);
    len = 0;
  }
  return len;
}

template <typename T>
__global__ void __launch_bounds__(kAttendWarps * 32) k_cache_attend(const AttendParams p) {
  const spec_cache_attend_args& a = p.a;
  __shared__ float sm[kAttendWarps], sl[kAttendWarps], so[kAttendWarps][128];
  pdl_trigger();
  pdl_wait();
  const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ int owner;
  if (threadIdx.x == 0) owner = -1;
  __syncthreads();
  int lo = 0, hi = 0, len = 0;
  for (int r = threadIdx.x; r < a.B; r += kAttendWarps * 32) {
    attend_request(p, r, lo, hi);
    if (lo <= t && t < hi) owner = r;
  }
  __syncthreads();
  const int b = owner;
  if (b >= 0) len = attend_request(p, b, lo, hi);
  const int pos = len - (hi - lo) + (t - lo);
  const int kvh = h / (a.heads / a.kv_heads);
  const T* q = (const T*)a.q + t * a.q_token + h * a.q_head;
  float qx[4], o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) qx[i] = lane + 32 * i < a.dim ? to_f32(q[lane + 32 * i]) : 0.f;
  float m = -INFINITY, l = 0.f;
  if (b >= 0) {
    const int from = a.window && pos >= a.window ? pos - a.window + 1 : 0;
    const int first = min(min(a.sinks, from), pos + 1);
    const int n = first + max(0, pos + 1 - from);
    for (int i = warp; i < n; i += kAttendWarps) {
      const int j = i < first ? i : from + (i - first);
      const long long page = a.block_table[b * a.table_stride + (j >> p.page_shift)];
      if (page < 0 || page >= a.num_pages) {
        if (p.status) atomicOr(p.status, SPEC_CACHE_BAD_PAGE);
        continue;
      }
      const int at = j & (a.page_size - 1);
      const T* k = (const T*)a.k_pages + page * a.kp_page + at * a.kp_token + kvh * a.kp_head;
      const T* v = (const T*)a.v_pages + page * a.vp_page + at * a.vp_token + kvh * a.vp_head;
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (lane + 32 * e < a.dim) s += qx[e] * to_f32(k[lane + 32 * e]);
      for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
      s *= a.scale;
      const float top = fmaxf(m, s);
      if (top == -INFINITY) continue;  // only scores of -inf so far
      const float keep = __expf(m - top), w = __expf(s - top);
      l = l * keep + w;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (lane + 32 * e < a.dim) o[e] = o[e] * keep + w * to_f32(v[lane + 32 * e]);
      m = top;
    }
  }
  sm[warp] = m;
  sl[warp] = l;
#pragma unroll
  for (int e = 0; e < 4; ++e) so[warp][lane + 32 * e] = o[e];
  __syncthreads();
  if (warp) return;
  float top = -INFINITY;
  for (int w = 0; w < kAttendWarps; ++w) top = fmaxf(top, sm[w]);
  float total = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int w = 0; w < kAttendWarps && top > -INFINITY; ++w) {
    const float keep = __expf(sm[w] - top);
    total += sl[w] * keep;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] += so[w][lane + 32 * e] * keep;
  }
  T* out = (T*)a.out + t * a.out_token + h * a.out_head;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (lane + 32 * e < a.dim) from_f32(total > 0.f ? acc[e] / total : 0.f, out[lane + 32 * e]);
  if (a.lse && lane == 0) a.lse[(long long)t * a.heads + h] = top + logf(total);
}

}  // namespace sv
