// C ABI of sparse attention and eviction on the paged cache (declared in
// include/spec_sparse.h): host-side argument checks and launches.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/spec_sparse.h"
#include "cache_host.cuh"
#include "evict_drop.cuh"
#include "evict_weigh.cuh"
#include "sparse_attend.cuh"
#include "sparse_bounds.cuh"
#include "sparse_score.cuh"
#include "sparse_select.cuh"

namespace {

using sv::aligned;
using sv::launch;
using sv::launch_cluster;
using sv::sm_count;
using sv::status_word;
using sv::tensor_map;

struct Axis {
  long long extent, stride;  // elements
};

// What an array of `element` bytes takes up; stride 1 inside.
struct Span {
  const void* at;
  long long bytes;
};
template <int N>
Span span(const void* at, int element, long long inner, const Axis (&axes)[N]) {
  long long last = inner - 1;
  for (auto& x : axes) {
    if (x.extent < 1) return {at, 0};
    last += (x.extent - 1) * x.stride;
  }
  return {at, (last + 1) * element};
}
Span span(const void* at, long long bytes) { return {at, bytes}; }
bool meet(const Span& a, const Span& b) {
  const unsigned long long p = (uintptr_t)a.at, q = (uintptr_t)b.at;
  return p && q && a.bytes > 0 && b.bytes > 0 && p < q + b.bytes && q < p + a.bytes;
}
// Whether one of the first `written` spans overlaps another one.
template <int N>
bool overlap(const Span (&x)[N], int written) {
  for (int i = 0; i < written; ++i)
    for (int j = i + 1; j < N; ++j)
      if (meet(x[i], x[j])) return true;
  return false;
}

// Strides that 16-byte accesses of 16-bit elements can take, where they are used at all.
template <int N>
bool wide(const void* base, const Axis (&axes)[N]) {
  if (!base || !aligned(base, 16)) return false;
  for (auto& x : axes)
    if (x.extent > 1 && (x.stride <= 0 || x.stride % 8 || x.stride >= 1ll << 38)) return false;
  return true;
}
template <int N>
bool words(const void* base, const Axis (&axes)[N]) {
  if (!base || !aligned(base, 4)) return false;
  for (auto& x : axes)
    if (x.extent > 1 && (x.stride <= 0 || x.stride >= 1ll << 38)) return false;
  return true;
}

// The sizes that all calls on pages have.
int check_sizes(int B, int width, int kv_heads, int dim, int page_size, long long num_pages,
                int dtype) {
  if (B < 0 || width < 1 || kv_heads < 1 || dim < 1 || page_size < 1 || num_pages < 1)
    return SPEC_ERR_INVALID_ARG;
  if (dtype != SPEC_CACHE_BF16 && dtype != SPEC_CACHE_F16) return SPEC_ERR_INVALID_ARG;
  if (dim % 8 || dim > 128 || page_size < 8 || (page_size & (page_size - 1)) ||
      page_size > 1 << 20 || num_pages > 0x7fffffffll || kv_heads > 1 << 16)
    return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}
int check_heads(int heads, int kv_heads, int T, int max_q) {
  if (heads < 1 || kv_heads < 1 || heads % kv_heads || T < 0 || max_q < 1)
    return SPEC_ERR_INVALID_ARG;
  return heads / kv_heads > 128 ? SPEC_ERR_UNSUPPORTED : SPEC_OK;
}

int page_shift(int page_size) {
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

sv::Requests requests(int B, int T, int width, int page_size, long long table_stride,
                      long long num_pages, const int* table, const int* lens, const int* cu_q,
                      unsigned* status) {
  sv::Requests r;
  r.B = B;
  r.T = T;
  r.width = width;
  r.page_shift = page_shift(page_size);
  r.table_stride = table_stride;
  r.num_pages = num_pages;
  r.table = table;
  r.kv_lens = lens;
  r.cu_q = cu_q;
  r.status = status;
  return r;
}

// The blocks of a grid as the launch takes them, or 0.
unsigned blocks(long long n) { return n > 0 && n <= 0x7fffffffll ? (unsigned)n : 0; }

// Groups of `per` tokens that the requests may have.
long long groups(int T, int B, int per) {
  const long long n = (long long)T / per + B;
  return n < T ? n : T;
}

// Lets a kernel have more than 48 KB of shared memory, once for each device.
template <typename K>
int allow(K kernel, int smem, std::atomic<unsigned long long>& ready) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return SPEC_ERR_CUDA;
  if (ready.load() >> dev & 1) return SPEC_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
      cudaSuccess) {
    cudaGetLastError();
    return SPEC_ERR_CUDA;
  }
  ready.fetch_or(1ull << dev);
  return SPEC_OK;
}

constexpr int kMostHeld = 48 * 1024;  // keys of a row that is looked at from shared memory
// Blocks of a cluster that pick from a row of n items together, up to 8; 1: a block alone. A row
// that fits one block's registers (16384 items) is as fast there (40 rows of 12500: 12.7 us alone,
// 13.0 with two blocks each), longer ones are faster in a cluster as long as that has an SM for
// each block (12 rows of 20000-33000: 30.6 us alone, 19.3 with eight).
int pick_ranks(long long rows, long long n, int sms) {
  int ranks = 1;
  while (ranks < 8 && rows * ranks * 2 <= sms) ranks *= 2;
  return n > 16384 && n <= 16384ll * ranks ? ranks : 1;
}

constexpr float kLog2e = 1.4426950408889634f;

int check_bounds(const spec_cache_bounds_args* a) {
  if (!a || a->max_q < 1) return SPEC_ERR_INVALID_ARG;
  const int rc = check_sizes(a->B, a->width, a->kv_heads, a->dim, a->page_size, a->num_pages,
                             a->dtype);
  if (rc != SPEC_OK || a->B == 0) return rc;
  if (!a->block_table || !a->kv_lens || a->table_stride < a->width) return SPEC_ERR_INVALID_ARG;
  const Axis k[] = {{a->num_pages, a->kp_page}, {a->page_size, a->kp_token},
                    {a->kv_heads, a->kp_head}};
  const Axis b[] = {{a->num_pages, a->b_page}, {a->kv_heads, a->b_head}, {2, a->b_side}};
  if (!wide(a->k_pages, k) || !wide(a->bounds, b)) return SPEC_ERR_INVALID_ARG;
  const Span x[] = {span(a->bounds, 2, a->dim, b), span(a->k_pages, 2, a->dim, k),
                    span(a->block_table, 4 * ((a->B - 1) * a->table_stride + a->width)),
                    span(a->kv_lens, 4ll * a->B), span(a->cu_q, 4ll * (a->B + 1))};
  return overlap(x, 1) ? SPEC_ERR_INVALID_ARG : SPEC_OK;
}

int check_score(const spec_cache_score_args* a) {
  if (!a) return SPEC_ERR_INVALID_ARG;
  int rc = check_sizes(a->B, a->width, a->kv_heads, a->dim, a->page_size, a->num_pages, a->dtype);
  if (rc == SPEC_OK) rc = check_heads(a->heads, a->kv_heads, a->num_tokens, a->max_q);
  if (rc != SPEC_OK || a->num_tokens == 0) return rc;
  const Axis q[] = {{a->num_tokens, a->q_token}, {a->heads, a->q_head}};
  const Axis b[] = {{a->num_pages, a->b_page}, {a->kv_heads, a->b_head}, {2, a->b_side}};
  const Axis s[] = {{a->num_tokens, a->s_token}, {a->kv_heads, a->s_head}};
  if (!wide(a->q, q) || !words(a->scores, s) || !a->cu_q) return SPEC_ERR_INVALID_ARG;
  if (a->B > 0 && (!wide(a->bounds, b) || !a->block_table || !a->kv_lens ||
                   a->table_stride < a->width))
    return SPEC_ERR_INVALID_ARG;
  const Span x[] = {span(a->scores, 4, a->width, s), span(a->q, 2, a->dim, q),
                    span(a->bounds, 2, a->dim, b),
                    span(a->block_table, 4 * ((a->B - 1) * a->table_stride + a->width)),
                    span(a->kv_lens, 4ll * a->B), span(a->cu_q, 4ll * (a->B + 1))};
  return overlap(x, 1) ? SPEC_ERR_INVALID_ARG : SPEC_OK;
}

int check_select(const spec_cache_select_args* a) {
  if (!a || a->count < 1 || a->first < 0 || a->recent < 0 ||
      (long long)a->first + a->recent > a->count)
    return SPEC_ERR_INVALID_ARG;
  int rc = check_sizes(a->B, a->width, a->kv_heads, 8, a->page_size, 1, SPEC_CACHE_BF16);
  if (rc == SPEC_OK) rc = check_heads(a->kv_heads, a->kv_heads, a->num_tokens, 1);
  if (rc != SPEC_OK || a->num_tokens == 0) return rc;
  const Axis s[] = {{a->num_tokens, a->s_token}, {a->kv_heads, a->s_head}};
  if (!words(a->scores, s) || !a->selected || !a->cu_q || (a->B > 0 && !a->kv_lens))
    return SPEC_ERR_INVALID_ARG;
  const Span x[] = {span(a->selected, 4ll * a->num_tokens * a->kv_heads * a->count),
                    span(a->scores, 4, a->width, s), span(a->kv_lens, 4ll * a->B),
                    span(a->cu_q, 4ll * (a->B + 1))};
  return overlap(x, 1) ? SPEC_ERR_INVALID_ARG : SPEC_OK;
}

int check_selected(const spec_cache_attend_selected_args* a) {
  if (!a || a->count < 1) return SPEC_ERR_INVALID_ARG;
  int rc = check_sizes(a->B, a->width, a->kv_heads, a->dim, a->page_size, a->num_pages, a->dtype);
  if (rc == SPEC_OK) rc = check_heads(a->heads, a->kv_heads, a->num_tokens, 1);
  if (rc != SPEC_OK || a->num_tokens == 0) return rc;
  if (!std::isfinite(a->scale * kLog2e)) return SPEC_ERR_INVALID_ARG;
  const Axis q[] = {{a->num_tokens, a->q_token}, {a->heads, a->q_head}};
  const Axis o[] = {{a->num_tokens, a->out_token}, {a->heads, a->out_head}};
  const Axis k[] = {{a->num_pages, a->kp_page}, {a->page_size, a->kp_token},
                    {a->kv_heads, a->kp_head}};
  const Axis v[] = {{a->num_pages, a->vp_page}, {a->page_size, a->vp_token},
                    {a->kv_heads, a->vp_head}};
  if (!wide(a->q, q) || !wide(a->out, o) || !a->cu_q) return SPEC_ERR_INVALID_ARG;
  if (a->B > 0 && (!wide(a->k_pages, k) || !wide(a->v_pages, v) || !a->block_table ||
                   !a->kv_lens || !a->selected || a->table_stride < a->width))
    return SPEC_ERR_INVALID_ARG;
  const Span x[] = {span(a->out, 2, a->dim, o),
                    span(a->lse, 4ll * a->num_tokens * a->heads),
                    span(a->q, 2, a->dim, q),
                    span(a->k_pages, 2, a->dim, k),
                    span(a->v_pages, 2, a->dim, v),
                    span(a->block_table, 4 * ((a->B - 1) * a->table_stride + a->width)),
                    span(a->selected, 4ll * a->num_tokens * a->kv_heads * a->count),
                    span(a->kv_lens, 4ll * a->B),
                    span(a->cu_q, 4ll * (a->B + 1))};
  return overlap(x, 2) ? SPEC_ERR_INVALID_ARG : SPEC_OK;
}

int check_weigh(const spec_cache_weigh_args* a) {
  if (!a || a->flags & ~SPEC_CACHE_TEST_WAIT_TIMEOUT) return SPEC_ERR_INVALID_ARG;
  int rc = check_sizes(a->B, a->width, a->kv_heads, a->dim, a->page_size, a->num_pages, a->dtype);
  if (rc == SPEC_OK) rc = check_heads(a->heads, a->kv_heads, a->num_tokens, a->max_q);
  if (rc != SPEC_OK || a->num_tokens == 0 || a->B == 0) return rc;
  if (!std::isfinite(a->scale * kLog2e) || !std::isfinite(a->decay)) return SPEC_ERR_INVALID_ARG;
  if ((long long)a->num_tokens * a->heads > 0x7fffffffll) return SPEC_ERR_UNSUPPORTED;
  const Axis q[] = {{a->num_tokens, a->q_token}, {a->heads, a->q_head}};
  const Axis k[] = {{a->num_pages, a->kp_page}, {a->page_size, a->kp_token},
                    {a->kv_heads, a->kp_head}};
  const Axis w[] = {{a->num_pages, a->w_page}, {a->kv_heads, a->w_head}};
  if (!wide(a->q, q) || !wide(a->k_pages, k) || !words(a->weights, w) || !a->lse ||
      !aligned(a->lse, 4) || !a->block_table || !a->kv_lens || !a->cu_q ||
      a->table_stride < a->width)
    return SPEC_ERR_INVALID_ARG;
  const Span x[] = {span(a->weights, 4, a->page_size, w),
                    span(a->q, 2, a->dim, q),
                    span(a->k_pages, 2, a->dim, k),
                    span(a->lse, 4ll * a->num_tokens * a->heads),
                    span(a->block_table, 4 * ((a->B - 1) * a->table_stride + a->width)),
                    span(a->kv_lens, 4ll * a->B),
                    span(a->cu_q, 4ll * (a->B + 1))};
  return overlap(x, 1) ? SPEC_ERR_INVALID_ARG : SPEC_OK;
}

int check_evict(const spec_cache_evict_args* a, bool pointers) {
  if (!a || a->first < 0 || a->recent < 0) return SPEC_ERR_INVALID_ARG;
  const int rc = check_sizes(a->B, a->width, a->kv_heads, a->dim, a->page_size, a->num_pages,
                             a->dtype);
  if (rc != SPEC_OK || !pointers) return rc;
  if (!a->free_count || !a->free_count_out) return SPEC_ERR_INVALID_ARG;
  if (a->B == 0)
    return a->free_count == a->free_count_out ? SPEC_ERR_INVALID_ARG : SPEC_OK;
  const Axis k[] = {{a->num_pages, a->kp_page}, {a->page_size, a->kp_token},
                    {a->kv_heads, a->kp_head}};
  const Axis v[] = {{a->num_pages, a->vp_page}, {a->page_size, a->vp_token},
                    {a->kv_heads, a->vp_head}};
  const Axis w[] = {{a->num_pages, a->w_page}, {a->kv_heads, a->w_head}};
  if (!wide(a->k_pages, k) || !wide(a->v_pages, v) || !words(a->weights, w) || !a->block_table ||
      !a->lens || !a->budget || !a->free_pages || !a->lens_out || a->table_stride < a->width)
    return SPEC_ERR_INVALID_ARG;
  if (a->k_pages == a->v_pages) return SPEC_ERR_INVALID_ARG;
  // (keys and values may be laid out between one another, so only the others are held apart)
  const Span ks = span(a->k_pages, 2, a->dim, k), vs = span(a->v_pages, 2, a->dim, v);
  const Span x[] = {span(a->weights, 4, a->page_size, w),
                    span(a->free_pages, 4ll * a->num_pages),
                    span(a->lens_out, 4ll * a->B),
                    span(a->free_count_out, 4),
                    span(a->workspace, (long long)a->workspace_bytes),
                    span(a->block_table, 4 * ((a->B - 1) * a->table_stride + a->width)),
                    span(a->lens, 4ll * a->B),
                    span(a->budget, 4ll * a->B),
                    span(a->free_count, 4)};
  if (overlap(x, 5)) return SPEC_ERR_INVALID_ARG;
  for (auto& y : x)
    if (meet(y, ks) || meet(y, vs)) return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}

// Workspace of spec_cache_evict: where each request's and head's moves begin, whether a request
// gives back what is no page, then where the moved tokens come from, for all pages of the pool or
// all columns of the table.
struct EvictSpace {
  bool by_page;
  size_t broken, from, bytes;
};
EvictSpace evict_space(const spec_cache_evict_args* a) {
  EvictSpace s;
  const long long columns = (long long)a->B * a->width;
  // (by columns it takes no look at the table to find a place; a table much wider than what the
  // requests can hold is not worth that)
  s.by_page = columns > 4ll * a->num_pages;
  s.broken = (size_t)a->B * a->kv_heads * 4;
  s.from = (s.broken + (size_t)a->B * 4 + 255) / 256 * 256;
  s.bytes = s.from + (size_t)(s.by_page ? a->num_pages : columns) * a->kv_heads * a->page_size * 4;
  return s;
}

template <int DP, bool BF16>
int score(const sv::ScoreParams& p, int sms, void* stream) {
  static std::atomic<unsigned long long> ready;
  using Cfg = sv::ScoreCfg<DP>;
  const int rc = allow(sv::k_cache_score<DP, BF16>, sv::kScoreGroups * Cfg::kGroupBytes, ready);
  if (rc != SPEC_OK) return rc;
  const int groups = (p.per + sv::kScoreGroup - 1) / sv::kScoreGroup;
  const int run = (p.rq.B + sv::kScoreThreads - 1) / sv::kScoreThreads;
  return launch(sv::k_cache_score<DP, BF16>, dim3(sms * sv::kScoreBlocks), sv::kScoreThreads,
                groups * Cfg::kGroupBytes, stream, p, run);
}

template <int DP, int N8, bool DEEP, bool BF16>
int selected(const sv::SelectedParams& p, unsigned grid, void* stream) {
  static std::atomic<unsigned long long> ready;
  constexpr int smem = sv::SelCfg<DP, N8, DEEP>::kSmem;
  const int rc = allow(sv::k_attend_selected<DP, N8, DEEP, BF16>, smem, ready);
  if (rc != SPEC_OK) return rc;
  return launch_cluster(sv::k_attend_selected<DP, N8, DEEP, BF16>, p.cluster, dim3(grid),
                        sv::SelCfg<DP, N8, DEEP>::kThreads, smem, stream, p);
}
template <int DP, bool BF16>
int selected(const sv::SelectedParams& p, int columns, int sms, unsigned grid, void* stream) {
  // more tiles in flight where there is a block for each SM at most (one token over 64 pages of
  // 32: 9.6 us in place of 11.5)
  if (columns <= 8)
    return (int)grid <= sms ? selected<DP, 1, true, BF16>(p, grid, stream)
                            : selected<DP, 1, false, BF16>(p, grid, stream);
  if (columns <= 16) return selected<DP, 2, false, BF16>(p, grid, stream);
  return selected<DP, 4, false, BF16>(p, grid, stream);
}

template <bool MUTE>
int weigh(const sv::WeighParams& p, int sms, int run, void* stream) {
  static std::atomic<unsigned long long> ready;
  const int rc = allow(sv::k_cache_weigh<MUTE>, sv::kWeighSmem, ready);
  if (rc != SPEC_OK) return rc;
  return launch(sv::k_cache_weigh<MUTE>, dim3(sms), sv::kWeighThreads, sv::kWeighSmem, stream, p,
                run);
}

}  // namespace

extern "C" {

int spec_cache_bounds(const spec_cache_bounds_args* a, void* stream, unsigned* device_status) {
  const int rc = check_bounds(a);
  if (rc != SPEC_OK) return rc;
  const int sms = sm_count();
  if (!sms) return SPEC_ERR_UNSUPPORTED;
  if (a->B == 0) return SPEC_OK;
  unsigned* status = status_word(device_status);
  if (!status) return SPEC_ERR_CUDA;
  sv::BoundsParams p;
  p.rq = requests(a->B, 0x7fffffff, a->width, a->page_size, a->table_stride, a->num_pages,
                  a->block_table, a->kv_lens, a->cu_q, status);
  p.k = (const char*)a->k_pages;
  p.k_page = a->kp_page * 2, p.k_token = a->kp_token * 2, p.k_head = a->kp_head * 2;
  p.out = (char*)a->bounds;
  p.o_page = a->b_page * 2, p.o_head = a->b_head * 2, p.o_side = a->b_side * 2;
  p.pieces = a->dim / 8;
  p.row_pieces = p.pieces * a->kv_heads;
  p.chunks = (p.row_pieces + sv::kBoundsThreads - 1) / sv::kBoundsThreads;
  // a block for each piece of work that there may be, up to some waves of blocks
  long long spread = a->cu_q ? ((long long)a->max_q + a->page_size - 2) / a->page_size + 1
                             : a->width;
  if (spread > a->width) spread = a->width;
  spread *= p.chunks;
  const long long most = 128ll * sms / a->B + 1;
  p.spread = (int)(spread < most ? spread : most);
  const unsigned grid = blocks((long long)a->B * p.spread);
  if (!grid) return SPEC_ERR_UNSUPPORTED;
  return launch(a->dtype == SPEC_CACHE_BF16 ? sv::k_cache_bounds<true> : sv::k_cache_bounds<false>,
                dim3(grid), sv::kBoundsThreads, 0, stream, p);
}

int spec_cache_score(const spec_cache_score_args* a, void* stream, unsigned* device_status) {
  const int rc = check_score(a);
  if (rc != SPEC_OK) return rc;
  const int sms = sm_count();
  if (!sms) return SPEC_ERR_UNSUPPORTED;
  if (a->num_tokens == 0) return SPEC_OK;
  unsigned* status = status_word(device_status);
  if (!status) return SPEC_ERR_CUDA;
  sv::ScoreParams p;
  p.rq = requests(a->B, a->num_tokens, a->width, a->page_size, a->table_stride, a->num_pages,
                  a->block_table, a->kv_lens, a->cu_q, status);
  p.heads = a->heads, p.kv_heads = a->kv_heads, p.G = a->heads / a->kv_heads, p.dim = a->dim;
  p.q = (const char*)a->q;
  p.q_token = a->q_token * 2, p.q_head = a->q_head * 2;
  p.bounds = (const char*)a->bounds;
  p.b_page = a->b_page * 2, p.b_head = a->b_head * 2, p.b_side = a->b_side * 2;
  p.scores = a->scores;
  p.s_token = a->s_token, p.s_head = a->s_head;
  const int most = sv::kScoreGroup * sv::kScoreGroups;
  p.per = a->max_q < most ? a->max_q : most;
  const bool bf16 = a->dtype == SPEC_CACHE_BF16;
  if (a->dim > 64)
    return bf16 ? score<128, true>(p, sms, stream) : score<128, false>(p, sms, stream);
  return bf16 ? score<64, true>(p, sms, stream) : score<64, false>(p, sms, stream);
}

int spec_cache_select(const spec_cache_select_args* a, void* stream, unsigned* device_status) {
  const int rc = check_select(a);
  if (rc != SPEC_OK) return rc;
  const int sms = sm_count();
  if (!sms) return SPEC_ERR_UNSUPPORTED;
  if (a->num_tokens == 0) return SPEC_OK;
  unsigned* status = status_word(device_status);
  if (!status) return SPEC_ERR_CUDA;
  sv::SelectParams p;
  p.rq = requests(a->B, a->num_tokens, a->width, a->page_size, 0, 1, nullptr, a->kv_lens, a->cu_q,
                  status);
  p.kv_heads = a->kv_heads, p.count = a->count, p.first = a->first, p.recent = a->recent;
  p.scores = a->scores;
  p.s_token = a->s_token, p.s_head = a->s_head;
  p.out = a->selected;
  p.vec = aligned(a->scores, 16) && a->s_token % 4 == 0 && a->s_head % 4 == 0;
  const unsigned grid = blocks((long long)a->num_tokens * a->kv_heads);
  if (!grid) return SPEC_ERR_UNSUPPORTED;
  // Rows of up to 4096 columns in as few threads as 16 columns each take (12000 rows of some 500
  // columns 44 us, with 128 threads for each 59), longer ones with pick_items, up to 16384 columns
  // in registers (4000 rows of 5000-6250 columns 96 us, 109 with pick_short, which has twice as
  // many counts for each thread between its barriers), and beyond that looked at again for each
  // histogram.
  p.held = 0;
  if (a->width <= 512)
    return launch(sv::k_cache_select_short<32>, dim3(grid), 32, 0, stream, p);
  if (a->width <= 1024)
    return launch(sv::k_cache_select_short<64>, dim3(grid), 64, 0, stream, p);
  if (a->width <= 2048)
    return launch(sv::k_cache_select_short<128>, dim3(grid), 128, 0, stream, p);
  if (a->width <= 4096)
    return launch(sv::k_cache_select_short<256>, dim3(grid), 256, 0, stream, p);
  const long long rows = (long long)a->num_tokens * a->kv_heads;
  p.ranks = pick_ranks(rows, a->width, sms);
  if (p.ranks > 1) {
    const unsigned wide = blocks(rows * p.ranks);
    return a->width <= p.ranks * 8192
               ? launch_cluster(sv::k_cache_select<1024, 8, true>, p.ranks, dim3(wide), 1024, 0,
                                stream, p)
               : launch_cluster(sv::k_cache_select<1024, 16, true>, p.ranks, dim3(wide), 1024, 0,
                                stream, p);
  }
  if (a->width <= 8192)
    return launch(sv::k_cache_select<1024, 8, false>, dim3(grid), 1024, 0, stream, p);
  if (a->width <= 16384)
    return launch(sv::k_cache_select<1024, 16, false>, dim3(grid), 1024, 0, stream, p);
  p.held = a->width < kMostHeld ? a->width : kMostHeld;
  static std::atomic<unsigned long long> ready;
  const int ok = allow(sv::k_cache_select<1024, 0, false>, kMostHeld * 4, ready);
  if (ok != SPEC_OK) return ok;
  return launch(sv::k_cache_select<1024, 0, false>, dim3(grid), 1024, p.held * 4, stream, p);
}

int spec_cache_attend_selected(const spec_cache_attend_selected_args* a, void* stream,
                               unsigned* device_status) {
  const int rc = check_selected(a);
  if (rc != SPEC_OK) return rc;
  const int sms = sm_count();
  if (!sms) return SPEC_ERR_UNSUPPORTED;
  if (a->num_tokens == 0) return SPEC_OK;
  unsigned* status = status_word(device_status);
  if (!status) return SPEC_ERR_CUDA;
  sv::SelectedParams p;
  std::memset(&p, 0, sizeof p);
  p.rq = requests(a->B, a->num_tokens, a->width, a->page_size, a->table_stride, a->num_pages,
                  a->block_table, a->kv_lens, a->cu_q, status);
  p.heads = a->heads, p.kv_heads = a->kv_heads, p.G = a->heads / a->kv_heads, p.dim = a->dim;
  p.q = (const char*)a->q;
  p.q_token = a->q_token * 2, p.q_head = a->q_head * 2;
  p.k = (const char*)a->k_pages;
  p.k_page = a->kp_page * 2, p.k_token = a->kp_token * 2, p.k_head = a->kp_head * 2;
  p.v = (const char*)a->v_pages;
  p.v_page = a->vp_page * 2, p.v_token = a->vp_token * 2, p.v_head = a->vp_head * 2;
  p.selected = a->selected;
  p.count = a->count;
  p.out = (char*)a->out;
  p.out_token = a->out_token * 2, p.out_head = a->out_head * 2;
  p.lse = a->lse;
  // a factor of 0 still leaves masked scores at -inf
  p.c = a->scale * kLog2e;
  if (std::fabs(p.c) < 1.1754944e-38f) p.c = 1.1754944e-38f;
  // A kv head's query heads in units of 32 at most, and as many tokens of a request (if there may
  // be several) as 16 columns, the block's list and the bytes over its ring take. With 8 columns 64
  // requests of 2-8 tokens over 128 pages of 16, four heads on a kv head, take the same 176 us, 28
  // of 11-18 over 43 of 64 182 in place of 177, 40 of 4-6 over 64 of 32, eight heads, 162 in place
  // of 150. 32 columns load a page for more tokens, but leave the SM two thirds of the warps, and
  // columns empty where a request's tokens do not fill them: the same three 256, 160 and 208 us. Of
  // 45 calls of 8 tokens a request or more the best gained 14 % with 32 (18 of 8 over 60 of 16: 59
  // us in place of 69), a third lost 20 to 100 % (20 of 9-10 over 64 of 32, eight heads: 122 in
  // place of 80); the lengths that decide it are not known here.
  p.unit_heads = p.G < 32 ? p.G : 32;
  p.splits = (p.G + p.unit_heads - 1) / p.unit_heads;
  p.per = 1;
  const int ring = a->dim > 64 ? sv::SelCfg<128, 1, false>::kRing : sv::SelCfg<64, 1, false>::kRing;
  if (a->num_tokens > a->B && a->width <= ring) {
    p.per = 16 / p.unit_heads;
    if (p.per > sv::kSelTokens) p.per = sv::kSelTokens;
    if (p.per > sv::kSelList / a->count) p.per = sv::kSelList / a->count;
    if (p.per < 1) p.per = 1;
  }
  long long units = groups(a->num_tokens, a->B, p.per) * a->kv_heads * p.splits;
  if (units < 1) units = 1;
  // clusters of blocks where the units leave SMs idle, as long as each warp keeps two tiles
  const int listed = a->count < a->width ? a->count : a->width;
  const long long tiles = (long long)listed * a->page_size / 16;
  p.cluster = 1;
  while (p.cluster < 8 && units * p.cluster < 3ll * sms && tiles >= 16ll * p.cluster)
    p.cluster *= 2;
  const unsigned grid = blocks(units * p.cluster);
  if (!grid) return SPEC_ERR_UNSUPPORTED;
  const int columns = p.per * p.unit_heads;
  const bool bf16 = a->dtype == SPEC_CACHE_BF16;
  if (a->dim > 64)
    return bf16 ? selected<128, true>(p, columns, sms, grid, stream)
                : selected<128, false>(p, columns, sms, grid, stream);
  return bf16 ? selected<64, true>(p, columns, sms, grid, stream)
              : selected<64, false>(p, columns, sms, grid, stream);
}

int spec_cache_weigh(const spec_cache_weigh_args* a, void* stream, unsigned* device_status) {
  const int rc = check_weigh(a);
  if (rc != SPEC_OK) return rc;
  const int sms = sm_count();
  if (!sms) return SPEC_ERR_UNSUPPORTED;
  if (a->num_tokens == 0 || a->B == 0) return SPEC_OK;
  unsigned* status = status_word(device_status);
  if (!status) return SPEC_ERR_CUDA;
  sv::WeighParams p;
  std::memset(&p, 0, sizeof p);
  p.rq = requests(a->B, a->num_tokens, a->width, a->page_size, a->table_stride, a->num_pages,
                  a->block_table, a->kv_lens, a->cu_q, status);
  p.heads = a->heads, p.kv_heads = a->kv_heads, p.G = a->heads / a->kv_heads, p.dim = a->dim;
  p.lse = a->lse;
  p.weights = a->weights;
  p.w_page = a->w_page, p.w_head = a->w_head;
  p.c = a->scale * kLog2e;
  p.decay = a->decay;
  p.bf16 = a->dtype == SPEC_CACHE_BF16;
  p.tile_tokens = sv::kWeighTile / p.G < a->max_q ? sv::kWeighTile / p.G : a->max_q;
  p.late_tiles = 2 * sv::kWeighTile / p.tile_tokens;
  p.blocks = a->dim > 64 ? 2 : 1;
  // Q of one column tile stays for a unit, and most stages hold keys; of several, they come again
  // for every pair of key tiles. (A wait for keys is rare then: a pair goes over all columns.)
  const int stages = sv::kWeighStages / (p.blocks * sv::kWeighTile * 128);
  p.shared_loads = a->max_q <= p.tile_tokens;
  p.q_stages = p.shared_loads ? 2 : 4;
  p.k_stages = (stages - p.q_stages) / 2;
  const int box = a->page_size < sv::kWeighTile ? a->page_size : sv::kWeighTile;
  if (!tensor_map(&p.q_map, a->dtype, a->q, a->dim, p.G, a->q_head, a->kv_heads, a->q_head * p.G,
                  a->num_tokens, a->q_token, p.G, p.tile_tokens) ||
      !tensor_map(&p.k_map, a->dtype, a->k_pages, a->dim, a->page_size, a->kp_token, a->kv_heads,
                  a->kp_head, a->num_pages, a->kp_page, box, 1))
    return SPEC_ERR_CUDA;
  const int run = a->B > sv::kWeighScan ? (a->B + sv::kWeighScan - 1) / sv::kWeighScan : 1;
  return a->flags & SPEC_CACHE_TEST_WAIT_TIMEOUT ? weigh<true>(p, sms, run, stream)
                                                 : weigh<false>(p, sms, run, stream);
}

long long spec_cache_evict_workspace(const spec_cache_evict_args* a) {
  const int rc = check_evict(a, false);
  if (rc != SPEC_OK) return rc;
  return (long long)evict_space(a).bytes;
}

int spec_cache_evict(const spec_cache_evict_args* a, void* stream, unsigned* device_status) {
  int rc = check_evict(a, true);
  if (rc != SPEC_OK) return rc;
  const int sms = sm_count();
  if (!sms) return SPEC_ERR_UNSUPPORTED;
  const EvictSpace ws = evict_space(a);
  if (a->B > 0 && (!a->workspace || a->workspace_bytes < ws.bytes)) return SPEC_ERR_CAPACITY;
  if (!aligned(a->workspace, 256)) return SPEC_ERR_INVALID_ARG;
  unsigned* status = status_word(device_status);
  if (!status) return SPEC_ERR_CUDA;
  sv::EvictParams p;
  std::memset(&p, 0, sizeof p);
  p.rq = requests(a->B, 0, a->width, a->page_size, a->table_stride, a->num_pages, a->block_table,
                  a->lens, nullptr, status);
  p.kv_heads = a->kv_heads, p.dim = a->dim, p.first = a->first, p.recent = a->recent;
  p.k = (char*)a->k_pages;
  p.k_page = a->kp_page * 2, p.k_token = a->kp_token * 2, p.k_head = a->kp_head * 2;
  p.v = (char*)a->v_pages;
  p.v_page = a->vp_page * 2, p.v_token = a->vp_token * 2, p.v_head = a->vp_head * 2;
  p.weights = a->weights;
  p.w_page = a->w_page, p.w_head = a->w_head;
  p.budget = a->budget;
  p.free_pages = a->free_pages;
  p.free_count = a->free_count;
  p.lens_out = a->lens_out;
  p.free_count_out = a->free_count_out;
  p.begin = (int*)a->workspace;
  p.broken = (int*)((char*)a->workspace + ws.broken);
  p.from = (int*)((char*)a->workspace + ws.from);
  p.by_page = ws.by_page;
  p.vec = aligned(a->weights, 16) && a->w_page % 4 == 0 && a->w_head % 4 == 0;
  const long long rows = (long long)a->B * a->kv_heads;
  // clusters where one block for each request and head leaves SMs idle
  p.cluster = 1;
  while (p.cluster < 8 && rows * p.cluster < sms) p.cluster *= 2;
  const unsigned grid = blocks(rows > 0 ? rows : 1), moves = blocks((rows + 1) * p.cluster);
  if (!grid || !moves) return SPEC_ERR_UNSUPPORTED;
  // Weights in registers up to 16384 tokens, with pick_short up to 4096 as in spec_cache_select
  // (16 requests of 12000-16000 with 8 heads 82 us, 96 with pick_short); longer requests' in
  // clusters' registers where there are few, else in shared memory as far as they fit, and looked
  // at again for each histogram.
  const long long most = (long long)a->width * a->page_size;
  p.ranks = rows > 0 ? pick_ranks(rows, most, sms) : 1;
  if (p.ranks > 1) {
    const unsigned wide = blocks(rows * p.ranks);
    rc = most <= p.ranks * 8192
             ? launch_cluster(sv::k_evict_pick<1024, 8, true>, p.ranks, dim3(wide), 1024, 0,
                              stream, p)
             : launch_cluster(sv::k_evict_pick<1024, 16, true>, p.ranks, dim3(wide), 1024, 0,
                              stream, p);
  } else if (most <= 2048) {
    rc = launch(sv::k_evict_pick_short<128>, dim3(grid), 128, 0, stream, p);
  } else if (most <= 4096) {
    rc = launch(sv::k_evict_pick_short<256>, dim3(grid), 256, 0, stream, p);
  } else if (most <= 16384) {
    rc = launch(sv::k_evict_pick<1024, 16, false>, dim3(grid), 1024, 0, stream, p);
  } else {
    p.held = most < kMostHeld ? (int)most : kMostHeld;
    static std::atomic<unsigned long long> ready;
    rc = allow(sv::k_evict_pick<1024, 0, false>, kMostHeld * 4, ready);
    if (rc != SPEC_OK) return rc;
    rc = launch(sv::k_evict_pick<1024, 0, false>, dim3(grid), 1024, p.held * 4, stream, p);
  }
  if (rc != SPEC_OK || rows == 0) return rc;
  return launch_cluster(sv::k_evict_move, p.cluster, dim3(moves), sv::kMoveThreads, 0, stream, p);
}

}  // extern "C"
