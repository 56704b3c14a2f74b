// C ABI of the paged cache (declared in include/spec_cache.h): host-side
// argument checks and launches.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/spec_cache.h"
#include "cache_append.cuh"
#include "cache_attend.cuh"
#include "cache_host.cuh"
#include "cache_step.cuh"

namespace sv {
namespace {

// Status bits of calls that come without a word for them.
__device__ unsigned g_status;

__global__ void k_clear_status(unsigned bits) { atomicAnd(&g_status, ~bits); }

}  // namespace

// Where a call's status bits go on the current device; NULL: no such place.
unsigned* status_word(unsigned* given) {
  if (given) return given;
  static std::atomic<unsigned*> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  unsigned* word = known[dev].load();
  if (!word) {
    if (cudaGetSymbolAddress((void**)&word, g_status) != cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    known[dev].store(word);
  }
  return word;
}

}  // namespace sv

namespace {

using sv::aligned;
using sv::k_clear_status;
using sv::launch;
using sv::sm_count;
using sv::status_word;
using sv::tensor_map;

// Whether what the call writes overlaps anything else of its arguments.
bool step_overlaps(const spec_cache_step_args* a) {
  const long long B = a->B, T = a->num_tokens;
  const struct {
    const void* at;
    long long bytes;
  } x[] = {{a->lens, 4 * B},
           {a->cu_new, 4 * (B + 1)},
           {a->positions, 4 * T},
           {a->slots, 8 * T},
           {a->free_count_out, 4},
           {a->block_table, B > 0 ? 4 * ((B - 1) * a->table_stride + a->width) : 0},
           {a->free_pages, 4ll * a->num_pages},
           {a->held_lens, 4 * B},  // from here on read only
           {a->new_lens, 4 * B},
           {a->cu_num_draft, 4 * (B + 1)},
           {a->num_accepted, 4 * B},
           {a->free_count, 4}};
  const int written = 7, all = sizeof x / sizeof *x;
  for (int i = 0; i < written; ++i)
    for (int j = i + 1; j < all; ++j) {
      const unsigned long long p = (uintptr_t)x[i].at, q = (uintptr_t)x[j].at;
      if (p && q && x[i].bytes > 0 && x[j].bytes > 0 && p < q + x[j].bytes && q < p + x[i].bytes)
        return true;
    }
  return false;
}

int check_step(const spec_cache_step_args* a) {
  if (!a || a->B < 0 || a->width < 1 || a->table_stride < a->width || a->page_size < 1 ||
      a->num_pages < 1 || a->num_tokens < 0)
    return SPEC_ERR_INVALID_ARG;
  if (!a->free_count || !a->cu_new || !a->free_count_out) return SPEC_ERR_INVALID_ARG;
  if (a->B > 0 && (a->cu_num_draft == nullptr) != (a->num_accepted == nullptr))
    return SPEC_ERR_INVALID_ARG;
  if (a->num_tokens > 0 && !a->slots) return SPEC_ERR_INVALID_ARG;
  if (a->B > 0 && (!a->held_lens || !a->new_lens || !a->block_table || !a->free_pages ||
                   !a->lens))
    return SPEC_ERR_INVALID_ARG;
  return step_overlaps(a) ? SPEC_ERR_INVALID_ARG : SPEC_OK;
}

int check_append(const spec_cache_append_args* a) {
  if (!a || a->num_tokens < 0 || a->kv_heads < 1 || a->dim < 1 || a->page_size < 1 ||
      a->num_pages < 1)
    return SPEC_ERR_INVALID_ARG;
  if (a->dtype != SPEC_CACHE_BF16 && a->dtype != SPEC_CACHE_F16) return SPEC_ERR_INVALID_ARG;
  if ((long long)a->kv_heads * a->dim > (1 << 24)) return SPEC_ERR_UNSUPPORTED;
  if (a->num_tokens == 0) return SPEC_OK;
  if (!a->k || !a->v || !a->slots || !a->k_pages || !a->v_pages) return SPEC_ERR_INVALID_ARG;
  const long long strides[] = {a->k_token, a->k_head,  a->v_token, a->v_head,   a->kp_page,
                               a->kp_token, a->kp_head, a->vp_page, a->vp_token, a->vp_head};
  for (long long s : strides)
    if (s < 0) return SPEC_ERR_INVALID_ARG;
  const void* ptrs[] = {a->k, a->v, a->k_pages, a->v_pages};
  for (const void* p : ptrs)
    if (!aligned(p, 2)) return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}

// The scores' factor: 2^x in place of e^x.
float exponent_scale(const spec_cache_attend_args* a) { return a->scale * 1.4426950408889634f; }

int check_attend(const spec_cache_attend_args* a, bool pointers) {
  if (!a || a->B < 0 || a->num_tokens < 0 || a->max_q < 1 || a->heads < 1 || a->kv_heads < 1 ||
      a->dim < 1 || a->page_size < 1 || a->width < 1 || a->num_pages < 1 || a->window < 0 ||
      a->sinks < 0 || a->heads % a->kv_heads)
    return SPEC_ERR_INVALID_ARG;
  if (a->dtype != SPEC_CACHE_BF16 && a->dtype != SPEC_CACHE_F16) return SPEC_ERR_INVALID_ARG;
  if (a->dim % 8 || a->dim > 128 || a->heads / a->kv_heads > 128 || a->page_size < 8 ||
      (a->page_size & (a->page_size - 1)) || a->num_pages > 0x7fffffffll)
    return SPEC_ERR_UNSUPPORTED;
  if (!pointers || a->num_tokens == 0) return SPEC_OK;
  if (!a->q || !a->out || !a->cu_q) return SPEC_ERR_INVALID_ARG;
  if (a->B > 0 && (!a->k_pages || !a->v_pages || !a->block_table || !a->kv_lens ||
                   a->table_stride < a->width))
    return SPEC_ERR_INVALID_ARG;
  if (!std::isfinite(exponent_scale(a))) return SPEC_ERR_INVALID_ARG;
  const void* ptrs[] = {a->q, a->k_pages, a->v_pages, a->out};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return SPEC_ERR_INVALID_ARG;
  const struct {
    long long extent, stride;
  } axes[] = {{a->num_tokens, a->q_token},   {a->heads, a->q_head},
              {a->num_pages, a->kp_page},    {a->page_size, a->kp_token},
              {a->kv_heads, a->kp_head},     {a->num_pages, a->vp_page},
              {a->page_size, a->vp_token},   {a->kv_heads, a->vp_head},
              {a->num_tokens, a->out_token}, {a->heads, a->out_head}};
  for (auto& x : axes)
    if (x.extent > 1 && (x.stride <= 0 || x.stride % 8 || x.stride >= 1ll << 38))
      return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}

// Partial results of spec_cache_attend: offsets of their parts.
struct Workspace {
  size_t ml, join, bytes;
};
Workspace attend_workspace(int sms, int dim) {
  const size_t tiles = (size_t)sms * 2 * 2;  // two partial units of two tiles for each block
  Workspace w;
  w.ml = tiles * (dim > 64 ? 128 : 64) * sv::kAttTile * sizeof(float);
  w.join = w.ml + tiles * sv::kAttTile * sizeof(float2);
  w.bytes = w.join + sms * sizeof(sv::AttJoin);
  return w;
}

template <int DP, bool BF16>
int attend(const sv::AttendParams& p, int sms, void* stream) {
  constexpr int smem = sv::AttCfg<DP>::kSmem;
  static std::atomic<unsigned long long> ready;  // devices whose kernel may use the memory
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SPEC_ERR_CUDA;
  if (!(ready.load() >> dev & 1)) {
    if (cudaFuncSetAttribute(sv::k_attend<DP, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem) != cudaSuccess) {
      cudaGetLastError();
      return SPEC_ERR_CUDA;
    }
    ready.fetch_or(1ull << dev);
  }
  const int run = p.B > sv::kAttScan ? (p.B + sv::kAttScan - 1) / sv::kAttScan : 1;
  const int rc = launch(sv::k_attend<DP, BF16>, dim3(sms), sv::kAttThreads, smem, stream, p, run);
  if (rc != SPEC_OK) return rc;
  // join's columns over 8 blocks a unit, over 4 where units have up to 32 rows. Microseconds a
  // call with 8 and with 4: 64 requests of 1-6 tokens in a window 68.2 and 66.5, 128 of one
  // token 86.4 and 84.4, one of one token over 4097 15.3 and 15.6; and above 32 rows, 2 of 5
  // tokens (35 rows) over 200000 76.8 and 79.0, 4 of 32 tokens (128 rows) 21.7 and 26.2.
  const int split = p.tile_tokens * p.G <= 32 ? 4 : 8;
  return launch(sv::k_attend_join<DP, BF16>, dim3(sms, split), sv::kJoinThreads, 0,
                stream, p);
}

}  // namespace

extern "C" {

int spec_cache_step(const spec_cache_step_args* a, void* stream, unsigned* device_status) {
  const int rc = check_step(a);
  if (rc != SPEC_OK) return rc;
  const int sms = sm_count();
  if (!sms) return SPEC_ERR_UNSUPPORTED;
  sv::StepParams p;
  p.a = *a;
  p.status = status_word(device_status);
  if (!p.status) return SPEC_ERR_CUDA;
  // for n < 2^31 and d < 2^31: floor(n / d) = n * (floor(2^(31 + s) / d) + 1) >> (31 + s),
  // s the bits of d - 1
  int bits = 0;
  while ((1ll << bits) < a->page_size) ++bits;
  p.page_shift = 31 + bits;
  p.page_mul = (1ull << p.page_shift) / a->page_size + 1;
  // Up to 1792 requests 256 threads scan them, in runs of seven at most, and start sooner than
  // 1024; with more the runs, which every search walks, get long. Microseconds with 256 and
  // with 1024, eight tokens a request: 8 requests 3.2 and 5.9, 1024 6.8 and 8.0, 1536 8.9 and
  // 9.6, 2000 11.2 and 10.3, 6000 25.9 and 17.5.
  const int items = a->num_tokens > a->B ? a->num_tokens : a->B;
  const bool small = a->B <= 1792;
  const int threads = small ? 256 : 1024;
  p.run = a->B > threads ? (a->B + threads - 1) / threads : 1;
  long long blocks = ((long long)items + threads - 1) / threads;
  if (blocks < 1) blocks = 1;
  if (blocks > sms) blocks = sms;
  return launch(small ? sv::k_cache_step<256> : sv::k_cache_step<1024>, dim3((unsigned)blocks),
                threads, 0, stream, p);
}

int spec_cache_append(const spec_cache_append_args* a, void* stream, unsigned* device_status) {
  const int rc = check_append(a);
  if (rc != SPEC_OK) return rc;
  const int sms = sm_count();
  if (!sms) return SPEC_ERR_UNSUPPORTED;
  if (a->num_tokens == 0) return SPEC_OK;
  sv::AppendParams p;
  p.a = *a;
  p.status = status_word(device_status);
  if (!p.status) return SPEC_ERR_CUDA;
  long long* strides[] = {&p.a.k_token,  &p.a.k_head,  &p.a.v_token, &p.a.v_head,   &p.a.kp_page,
                          &p.a.kp_token, &p.a.kp_head, &p.a.vp_page, &p.a.vp_token, &p.a.vp_head};
  bool wide = a->dim % 8 == 0 && aligned(a->k, 16) && aligned(a->v, 16) &&
              aligned(a->k_pages, 16) && aligned(a->v_pages, 16);
  for (long long* s : strides) {
    *s *= 2;
    wide = wide && *s % 16 == 0;
  }
  const int vec = wide ? 16 : 2;
  p.pieces = a->dim * 2 / vec;
  p.row_pieces = p.pieces * a->kv_heads;
  // four tokens a block leave each SM two blocks from there on (5000 tokens: 5.6 us against 7.6
  // with one, 50001: 65 against 90); below, a token a block spreads the call over more SMs
  // (640 tokens: 2.5 us against 2.9)
  const bool many = a->num_tokens > 8ll * sms;
  const int tokens = many ? 4 : 1;
  const long long blocks = (a->num_tokens + tokens - 1) / tokens;
  if (blocks > 0x7fffffffll) return SPEC_ERR_UNSUPPORTED;
  auto kernel = wide ? (many ? sv::k_cache_append<16, 4> : sv::k_cache_append<16, 1>)
                     : (many ? sv::k_cache_append<2, 4> : sv::k_cache_append<2, 1>);
  return launch(kernel, dim3((unsigned)blocks), sv::kAppendThreads, 0, stream, p);
}

long long spec_cache_attend_workspace(const spec_cache_attend_args* a) {
  const int rc = check_attend(a, false);
  if (rc != SPEC_OK) return rc;
  const int sms = sm_count();
  if (!sms) return SPEC_ERR_UNSUPPORTED;
  return (long long)attend_workspace(sms, a->dim).bytes;
}

int spec_cache_attend(const spec_cache_attend_args* a, void* stream, unsigned* device_status) {
  const int rc = check_attend(a, true);
  if (rc != SPEC_OK) return rc;
  const int sms = sm_count();
  if (!sms) return SPEC_ERR_UNSUPPORTED;
  if (a->num_tokens == 0) return SPEC_OK;
  const Workspace ws = attend_workspace(sms, a->dim);
  if (!a->workspace || a->workspace_bytes < ws.bytes) return SPEC_ERR_CAPACITY;
  if (!aligned(a->workspace, 256)) return SPEC_ERR_INVALID_ARG;
  sv::AttendParams p;
  std::memset(&p, 0, sizeof p);
  p.B = a->B;
  p.T = a->num_tokens;
  p.heads = a->heads;
  p.kv_heads = a->kv_heads;
  p.G = a->heads / a->kv_heads;
  p.dim = a->dim;
  while ((1 << p.page_shift) < a->page_size) ++p.page_shift;
  p.width = a->width;
  p.num_pages = a->num_pages;
  p.table_stride = a->table_stride;
  p.table = a->block_table;
  p.kv_lens = a->kv_lens;
  p.cu_q = a->cu_q;
  p.out = (char*)a->out;
  p.out_token = a->out_token * 2;
  p.out_head = a->out_head * 2;
  p.lse = a->lse;
  // a scale of 0 still leaves masked scores at -inf
  p.c = exponent_scale(a);
  if (std::fabs(p.c) < 1.1754944e-38f) p.c = 1.1754944e-38f;
  p.hidden = p.c > 0.f ? -INFINITY : INFINITY;
  p.window = a->window < (long long)a->width * a->page_size ? a->window : 0;
  p.sinks = a->sinks;
  p.tile_tokens = sv::kAttTile / p.G < a->max_q ? sv::kAttTile / p.G : a->max_q;
  p.status = status_word(device_status);
  if (!p.status) return SPEC_ERR_CUDA;
  char* w = (char*)a->workspace;
  p.part_o = (float4*)w;
  p.part_ml = (float2*)(w + ws.ml);
  p.join = (sv::AttJoin*)(w + ws.join);
  const unsigned box_page = a->page_size < sv::kAttTile ? a->page_size : sv::kAttTile;
  const int dim = a->dim, kv = a->kv_heads;
  if (!tensor_map(&p.q_map, a->dtype, a->q, dim, p.G, a->q_head, kv, a->q_head * p.G, p.T,
                  a->q_token, p.G, p.tile_tokens))
    return SPEC_ERR_CUDA;
  if (a->B > 0 &&
      (!tensor_map(&p.k_map, a->dtype, a->k_pages, dim, a->page_size, a->kp_token, kv,
                   a->kp_head, a->num_pages, a->kp_page, box_page, 1) ||
       !tensor_map(&p.v_map, a->dtype, a->v_pages, dim, a->page_size, a->vp_token, kv,
                   a->vp_head, a->num_pages, a->vp_page, box_page, 1)))
    return SPEC_ERR_CUDA;
  if (a->B == 0) p.k_map = p.v_map = p.q_map;  // prefetched all the same, so they have to be maps
  const bool bf16 = a->dtype == SPEC_CACHE_BF16;
  if (dim > 64)
    return bf16 ? attend<128, true>(p, sms, stream) : attend<128, false>(p, sms, stream);
  return bf16 ? attend<64, true>(p, sms, stream) : attend<64, false>(p, sms, stream);
}

int spec_cache_status(unsigned* bits) {
  if (!bits) return SPEC_ERR_INVALID_ARG;
  if (!sm_count()) return SPEC_ERR_UNSUPPORTED;
  const unsigned* word = status_word(nullptr);
  unsigned v = 0;
  if (!word || cudaDeviceSynchronize() != cudaSuccess ||
      cudaMemcpy(&v, word, sizeof v, cudaMemcpyDeviceToHost) != cudaSuccess)
    return SPEC_ERR_CUDA;
  if (v) {  // (bits that another thread's call sets meanwhile stay)
    k_clear_status<<<1, 1>>>(v);
    if (cudaDeviceSynchronize() != cudaSuccess) return SPEC_ERR_CUDA;
  }
  *bits = v;
  return v ? SPEC_ERR_DEVICE_STATUS : SPEC_OK;
}

}  // extern "C"
