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
// them: a run of E consecutive requests per thread, one block-wide scan of
// the run totals. That is work repeated by every block, against a second
// launch or a chain through global memory between blocks.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/spec_cache.h"
#include "pipe.cuh"

namespace sv {

constexpr int kStepThreads = 512;

struct StepParams {
  spec_cache_step_args a;
  unsigned* status;
  int run;  // requests per thread of the scan
};

// Lengths and pages of one request.
struct StepRequest {
  long long kept, lens;
  long long have, need;  // pages before and after
  int fresh;             // new tokens
  bool ok;
};

__device__ __forceinline__ StepRequest step_request(const spec_cache_step_args& a, int r) {
  StepRequest q;
  const int held = a.held_lens[r];
  q.fresh = a.new_lens[r];
  int gone = 0;
  q.ok = held >= 0 && q.fresh >= 0;
  if (a.cu_num_draft) {
    const int drafts = a.cu_num_draft[r + 1] - a.cu_num_draft[r];
    const int accepted = a.num_accepted[r];
    q.ok = q.ok && drafts >= 0 && accepted >= 0 && accepted <= drafts;
    gone = drafts - accepted;
  }
  q.kept = (long long)held - gone;
  q.lens = q.kept + q.fresh;
  const unsigned page = (unsigned)a.page_size;
  // lengths are below 2^31, so the rounded-up sums fit 32 unsigned bits
  q.have = ((unsigned)max(held, 0) + (page - 1u)) / page;
  q.ok = q.ok && q.kept >= 0 && q.have <= a.width && q.lens <= (long long)a.width * page &&
         q.lens <= 0x7fffffffll;
  q.need = q.ok ? ((unsigned)q.lens + (page - 1u)) / page : 0;
  return q;
}

struct StepSums {
  long long fresh, gone, more;
};

__device__ __forceinline__ StepSums step_add(StepSums x, StepSums y) {
  return {x.fresh + y.fresh, x.gone + y.gone, x.more + y.more};
}
__device__ __forceinline__ StepSums step_of(const StepRequest& q) {
  return {q.fresh, q.have > q.need ? q.have - q.need : 0, q.need > q.have ? q.need - q.have : 0};
}
__device__ __forceinline__ StepSums step_up(StepSums x, int d) {
  return {__shfl_up_sync(~0u, x.fresh, d), __shfl_up_sync(~0u, x.gone, d),
          __shfl_up_sync(~0u, x.more, d)};
}

// The request that item x of prefix sum WHICH (0 new tokens, 1 pages given
// up, 2 pages taken) belongs to, and the sums before that request.
template <int WHICH>
__device__ __forceinline__ int step_find(const StepParams& p, const StepSums* before, long long x,
                                         StepRequest& q, StepSums& at) {
  auto part = [](const StepSums& s) { return WHICH == 0 ? s.fresh : WHICH == 1 ? s.gone : s.more; };
  int lo = 0, hi = kStepThreads - 1;  // the last run that starts at or before x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (part(before[mid]) <= x) lo = mid; else hi = mid - 1;
  }
  at = before[lo];
  int r = lo * p.run;
  for (;; ++r) {  // x is below the total, so a request of this run holds it
    q = step_request(p.a, r);
    const StepSums next = step_add(at, step_of(q));
    if (x < part(next) || r + 1 >= p.a.B) return r;
    at = next;
  }
}

__global__ void __launch_bounds__(kStepThreads) k_cache_step(const StepParams p) {
  __shared__ StepSums before[kStepThreads];
  __shared__ StepSums warp_sum[kStepThreads / 32];
  const spec_cache_step_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  pdl_wait();
  // Totals of this thread's run of requests, then the scan over the block.
  StepSums sum = {0, 0, 0};
  int bad = 0;
  const int r0 = min((long long)tid * p.run, (long long)a.B), r1 = min(r0 + p.run, a.B);
  for (int r = r0; r < r1; ++r) {
    const StepRequest q = step_request(a, r);
    bad |= !q.ok;
    sum = step_add(sum, step_of(q));
  }
  StepSums scan = sum;
  for (int d = 1; d < 32; d <<= 1) {
    const StepSums y = step_up(scan, d);
    if (lane >= d) scan = step_add(scan, y);
  }
  if (lane == 31) warp_sum[warp] = scan;
  bad = __syncthreads_or(bad);
  StepSums base = {0, 0, 0}, total = {0, 0, 0};
  for (int w = 0; w < kStepThreads / 32; ++w) {
    if (w == warp) base = total;
    total = step_add(total, warp_sum[w]);
  }
  base = step_add(base, {scan.fresh - sum.fresh, scan.gone - sum.gone, scan.more - sum.more});
  before[tid] = base;
  __syncthreads();

  const long long count = *a.free_count;
  bad = bad || total.fresh > a.num_tokens || count < 0 || count + total.gone > a.num_pages;
  const bool dry = !bad && total.more > count + total.gone;
  const bool go = !bad && !dry;
  const int first = blockIdx.x * kStepThreads + tid, step = gridDim.x * kStepThreads;
  if (first == 0) {
    if (!go && p.status) atomicOr(p.status, bad ? SPEC_CACHE_BAD_LENGTHS : SPEC_CACHE_NO_PAGES);
    *a.free_count_out = (int)(go ? count + total.gone - total.more : count);
    a.cu_new[0] = 0;
  }
  // Lengths and offsets: the runs are dealt to the blocks in turn.
  if (tid % gridDim.x == blockIdx.x) {
    StepSums at = base;
    for (int r = r0; r < r1; ++r) {
      const StepRequest q = step_request(a, r);
      at = step_add(at, step_of(q));
      a.lens[r] = go ? (int)q.lens : a.held_lens[r];
      a.cu_new[r + 1] = go ? (int)at.fresh : 0;
    }
  }
  if (!go) {
    for (long long t = first; t < a.num_tokens; t += step) {
      a.slots[t] = -1;
      if (a.positions) a.positions[t] = -1;
    }
    return;
  }
  // Entry i of the stack once the pages given up are on it.
  auto entry = [&](long long i) -> int {
    if (i < count) return a.free_pages[i];
    StepRequest q;
    StepSums at;
    const int r = step_find<1>(p, before, i - count, q, at);
    return a.block_table[r * a.table_stride + q.need + (i - count - at.gone)];
  };
  const long long top = count + total.gone - 1;
  for (long long i = first; i < total.gone; i += step) a.free_pages[count + i] = entry(count + i);
  for (long long i = first; i < total.more; i += step) {
    StepRequest q;
    StepSums at;
    const int r = step_find<2>(p, before, i, q, at);
    a.block_table[r * a.table_stride + q.have + (i - at.more)] = entry(top - i);
  }
  for (long long t = first; t < a.num_tokens; t += step) {
    long long slot = -1;
    int pos = -1;
    if (t < total.fresh) {
      StepRequest q;
      StepSums at;
      const int r = step_find<0>(p, before, t, q, at);
      pos = (int)(q.kept + (t - at.fresh));
      const int col = (int)((unsigned)pos / (unsigned)a.page_size);
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
