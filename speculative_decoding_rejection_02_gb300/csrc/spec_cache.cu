// C ABI of the paged cache (declared in include/spec_cache.h): host-side
// argument checks and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/spec_cache.h"
#include "cache_append.cuh"
#include "cache_attend.cuh"
#include "cache_step.cuh"

namespace {

// The multiprocessors of the current device; 0 if it is not an sm_103.
int sm_count() {
  static int known[64];  // 0: not asked yet, -1: not an sm_103
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (known[dev] == 0) {
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return 0;
    known[dev] = major == 10 && minor == 3 ? sms : -1;
  }
  return known[dev] > 0 ? known[dev] : 0;
}

// Launch after the stream's earlier work, but with the launch itself prepared
// while that work still runs (the kernels begin with pdl_wait).
template <typename P>
int launch(void (*kernel)(P), dim3 grid, int threads, size_t smem, void* stream, const P& p) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess) return SPEC_OK;
  cudaGetLastError();
  return SPEC_ERR_CUDA;
}

bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

int check_step(const spec_cache_step_args* a) {
  if (!a || a->B < 0 || a->width < 1 || a->table_stride < a->width || a->page_size < 1 ||
      a->num_pages < 1 || a->num_tokens < 0)
    return SPEC_ERR_INVALID_ARG;
  if (!a->free_count || !a->cu_new || !a->free_count_out || a->free_count == a->free_count_out)
    return SPEC_ERR_INVALID_ARG;
  if (a->B > 0 && (a->cu_num_draft == nullptr) != (a->num_accepted == nullptr))
    return SPEC_ERR_INVALID_ARG;
  if (a->num_tokens > 0 && !a->slots) return SPEC_ERR_INVALID_ARG;
  if (a->B > 0 && (!a->held_lens || !a->new_lens || !a->block_table || !a->free_pages ||
                   !a->lens || a->lens == a->held_lens || a->lens == a->new_lens))
    return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
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
  if (!std::isfinite(a->scale)) return SPEC_ERR_INVALID_ARG;
  const void* ptrs[] = {a->q, a->k_pages, a->v_pages, a->out};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return SPEC_ERR_INVALID_ARG;
  const long long strides[] = {a->q_token,  a->q_head,  a->kp_page,   a->kp_token, a->kp_head,
                               a->vp_page, a->vp_token, a->vp_head, a->out_token, a->out_head};
  for (long long s : strides)
    if (s < 0 || s % 8) return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
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
  p.status = device_status;
  p.run = a->B > sv::kStepThreads ? (a->B + sv::kStepThreads - 1) / sv::kStepThreads : 1;
  const long long items = a->num_tokens > a->B ? a->num_tokens : a->B;
  long long blocks = (items + 2 * sv::kStepThreads - 1) / (2 * sv::kStepThreads);
  if (blocks < 1) blocks = 1;
  if (blocks > sms) blocks = sms;
  return launch(sv::k_cache_step, dim3((unsigned)blocks), sv::kStepThreads, 0, stream, p);
}

int spec_cache_append(const spec_cache_append_args* a, void* stream, unsigned* device_status) {
  const int rc = check_append(a);
  if (rc != SPEC_OK) return rc;
  const int sms = sm_count();
  if (!sms) return SPEC_ERR_UNSUPPORTED;
  if (a->num_tokens == 0) return SPEC_OK;
  sv::AppendParams p;
  p.a = *a;
  p.status = device_status;
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
  return rc != SPEC_OK ? rc : 0;
}

int spec_cache_attend(const spec_cache_attend_args* a, void* stream, unsigned* device_status) {
  const int rc = check_attend(a, true);
  if (rc != SPEC_OK) return rc;
  const int sms = sm_count();
  if (!sms) return SPEC_ERR_UNSUPPORTED;
  if (a->num_tokens == 0) return SPEC_OK;
  sv::AttendParams p;
  p.a = *a;
  p.status = device_status;
  p.page_shift = 0;
  while ((1 << p.page_shift) < a->page_size) ++p.page_shift;
  auto kernel = a->dtype == SPEC_CACHE_BF16 ? sv::k_cache_attend<__nv_bfloat16>
                                            : sv::k_cache_attend<__half>;
  return launch(kernel, dim3(a->num_tokens, a->heads), sv::kAttendWarps * 32, 0, stream, p);
}

}  // extern "C"
