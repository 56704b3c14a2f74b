// The paged cache's bookkeeping between two verification rounds
// (spec_cache_step): request lengths after the verdict, pages given back and
// taken, block table, positions and slots of the next round's tokens.
//
// Everything follows from three prefix sums over the requests (new tokens,
// pages given up, pages taken): page i of those taken is entry
// count + freed - 1 - i of the stack, and where that entry is itself one
// given up in this call, its owner is found by a search in the prefix sums
// instead of waiting for it to be written. So every output entry is computed
// on its own, no block waits for another, and one launch does the whole step.
//
// Each block reads all lengths (16 bytes per request, from L2) and scans
// them: a run of consecutive requests per thread, one block-wide scan of the
// run totals. That is work repeated by every block, against a second launch
// or a chain through global memory between blocks. The sums saturate at
// 2^32 - 1, which no valid call reaches.
//
// Latency bounds it: 3.2 us for 8 requests (one block), 6.8 us for 1024 with
// 8192 token slots, 15 us for 6000 with 240000 (the search for each token's
// request, in the scan's prefix sums and then along a run of six).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/spec_cache.h"
#include "pipe.cuh"

namespace sv {

struct StepParams {
  spec_cache_step_args a;
  unsigned* status;
  int run;  // requests per thread of the scan
  // n / page_size = n * page_mul >> page_shift for 0 <= n < 2^31
  unsigned long long page_mul;
  int page_shift;
};

__device__ __forceinline__ int step_pages(const StepParams& p, int n) {  // page of token n
  return (int)((unsigned long long)n * p.page_mul >> p.page_shift);
}

// Lengths and pages of one request.
struct StepRequest {
  int kept, lens, fresh;
  int have, need;  // pages before and after
  bool ok;
};

__device__ __forceinline__ StepRequest step_request(const StepParams& p, int r) {
  const spec_cache_step_args& a = p.a;
  StepRequest q;
  const int held = a.held_lens[r];
  q.fresh = a.new_lens[r];
  int gone = 0;
  q.ok = held >= 0 && q.fresh >= 0;
  if (a.cu_num_draft) {
    const int drafts = a.cu_num_draft[r + 1] - a.cu_num_draft[r];
    const int accepted = a.num_accepted[r];
    gone = drafts - accepted;
    q.ok = q.ok && accepted >= 0 && gone >= 0 && gone <= held && drafts >= 0;
  }
  q.kept = held - gone;
  const long long lens = (long long)q.kept + q.fresh;
  q.ok = q.ok && lens <= 0x7fffffffll;
  q.lens = q.ok ? (int)lens : 0;
  q.have = q.ok && held > 0 ? step_pages(p, held - 1) + 1 : 0;
  q.need = q.lens > 0 ? step_pages(p, q.lens - 1) + 1 : 0;
  q.ok = q.ok && q.have <= a.width && q.need <= a.width;
  return q;
}

struct StepSums {
  unsigned fresh, gone, more;
};

__device__ __forceinline__ unsigned sat_add(unsigned x, unsigned y) {
  const unsigned z = x + y;
  return z < x ? ~0u : z;
}
__device__ __forceinline__ StepSums step_add(StepSums x, StepSums y) {
  return {sat_add(x.fresh, y.fresh), sat_add(x.gone, y.gone), sat_add(x.more, y.more)};
}
__device__ __forceinline__ StepSums step_of(const StepRequest& q) {
  return {(unsigned)max(q.fresh, 0), (unsigned)max(q.have - q.need, 0),
          (unsigned)max(q.need - q.have, 0)};
}
__device__ __forceinline__ StepSums step_up(StepSums x, int d) {
  return {__shfl_up_sync(~0u, x.fresh, d), __shfl_up_sync(~0u, x.gone, d),
          __shfl_up_sync(~0u, x.more, d)};
}

template <int THREADS>
struct StepShared {
  unsigned fresh[THREADS], gone[THREADS], more[THREADS];  // before each thread's run
  StepSums warp_sum[THREADS / 32];
};

// The request that item x of prefix sum WHICH (0 new tokens, 1 pages given
// up, 2 pages taken) belongs to, and the sums before that request.
template <int WHICH, int THREADS>
__device__ __forceinline__ int step_find(const StepParams& p, const StepShared<THREADS>& sh,
                                         unsigned x, StepRequest& q, StepSums& at) {
  const unsigned* before = WHICH == 0 ? sh.fresh : WHICH == 1 ? sh.gone : sh.more;
  auto part = [](const StepSums& s) { return WHICH == 0 ? s.fresh : WHICH == 1 ? s.gone : s.more; };
  int lo = 0;  // the last run that starts at or before x
#pragma unroll
  for (int d = THREADS / 2; d; d >>= 1)
    if (before[lo + d] <= x) lo += d;
  at = {sh.fresh[lo], sh.gone[lo], sh.more[lo]};
  int r = lo * p.run;
  for (;; ++r) {  // x is below the total, so a request of this run holds it
    q = step_request(p, r);
    const StepSums next = step_add(at, step_of(q));
    if (x < part(next) || r + 1 >= p.a.B) return r;
    at = next;
  }
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) k_cache_step(const StepParams p) {
  __shared__ StepShared<THREADS> sh;
  const spec_cache_step_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  pdl_wait();
  const int count = *a.free_count;
  // Totals of this thread's run of requests, then the scan over the block.
  StepSums sum = {0, 0, 0};
  int bad = 0;
  const int r0 = min(tid * p.run, a.B), r1 = min(r0 + p.run, a.B);
#pragma unroll 4
  for (int r = r0; r < r1; ++r) {
    const StepRequest q = step_request(p, r);
    bad |= !q.ok;
    sum = step_add(sum, step_of(q));
  }
  StepSums scan = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const StepSums y = step_up(scan, d);
    if (lane >= d) scan = step_add(scan, y);
  }
  if (lane == 31) sh.warp_sum[warp] = scan;
  bad = __syncthreads_or(bad);
  StepSums base = {0, 0, 0}, total = {0, 0, 0};
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w == warp) base = total;
    total = step_add(total, sh.warp_sum[w]);
  }
  base = step_add(base, {scan.fresh - sum.fresh, scan.gone - sum.gone, scan.more - sum.more});
  sh.fresh[tid] = base.fresh;
  sh.gone[tid] = base.gone;
  sh.more[tid] = base.more;
  __syncthreads();

  bad = bad || total.fresh > (unsigned)a.num_tokens || count < 0 ||
        total.gone > (unsigned)a.num_pages ||
        (unsigned)count + total.gone > (unsigned)a.num_pages;
  const bool dry = !bad && total.more > (unsigned)count + total.gone;
  const bool go = !bad && !dry;
  const unsigned first = blockIdx.x * THREADS + tid, step = gridDim.x * THREADS;
  if (first == 0) {
    if (!go) atomicOr(p.status, bad ? SPEC_CACHE_BAD_LENGTHS : SPEC_CACHE_NO_PAGES);
    *a.free_count_out = go ? (int)(count + total.gone - total.more) : count;
    a.cu_new[0] = 0;
  }
  // Lengths and offsets: the runs are dealt to the blocks in turn.
  if (tid % gridDim.x == blockIdx.x) {
    StepSums at = base;
    for (int r = r0; r < r1; ++r) {
      const StepRequest q = step_request(p, r);
      at = step_add(at, step_of(q));
      a.lens[r] = go ? q.lens : a.held_lens[r];
      a.cu_new[r + 1] = go ? (int)at.fresh : 0;
    }
  }
  if (!go) {
    for (unsigned t = first; t < (unsigned)a.num_tokens; t += step) {
      a.slots[t] = -1;
      if (a.positions) a.positions[t] = -1;
    }
    return;
  }
  // Entry i of the stack once the pages given up are on it.
  auto entry = [&](unsigned i) -> int {
    if (i < (unsigned)count) return a.free_pages[i];
    StepRequest q;
    StepSums at;
    const int r = step_find<1, THREADS>(p, sh, i - count, q, at);
    return a.block_table[r * a.table_stride + q.need + (i - count - at.gone)];
  };
  const unsigned top = count + total.gone - 1;
  for (unsigned i = first; i < total.gone; i += step) a.free_pages[count + i] = entry(count + i);
  for (unsigned i = first; i < total.more; i += step) {
    StepRequest q;
    StepSums at;
    const int r = step_find<2, THREADS>(p, sh, i, q, at);
    a.block_table[r * a.table_stride + q.have + (i - at.more)] = entry(top - i);
  }
  for (unsigned t = first; t < (unsigned)a.num_tokens; t += step) {
    long long slot = -1;
    int pos = -1;
    if (t < total.fresh) {
      StepRequest q;
      StepSums at;
      const int r = step_find<0, THREADS>(p, sh, t, q, at);
      pos = q.kept + (int)(t - at.fresh);
      const int col = step_pages(p, pos);
      // a page taken in this call is looked up where it came from: another
      // block may not have written it to the table yet
      const int page = col < q.have ? a.block_table[r * a.table_stride + col]
                                    : entry(top - (at.more + (col - q.have)));
      slot = (long long)page * a.page_size + (pos - col * a.page_size);
    }
    a.slots[t] = slot;
    if (a.positions) a.positions[t] = pos;
  }
}

}  // namespace sv
