// Python's way into the paged cache's C ABI: checks torch tensors, allocates
// outputs and workspace on the current stream, and makes the call. In C++
// because a call's kernels take a few microseconds and the same checks in
// Python take twenty. Every function returns its outputs, or the (negative)
// code of a call that was refused.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <stdexcept>

#include "../../include/spec_sparse.h"

namespace {

int (*g_step)(const spec_cache_step_args*, void*, unsigned*);
int (*g_append)(const spec_cache_append_args*, void*, unsigned*);
int (*g_attend)(const spec_cache_attend_args*, void*, unsigned*);
long long (*g_workspace)(const spec_cache_attend_args*);
int (*g_bounds)(const spec_cache_bounds_args*, void*, unsigned*);
int (*g_score)(const spec_cache_score_args*, void*, unsigned*);
int (*g_select)(const spec_cache_select_args*, void*, unsigned*);
int (*g_selected)(const spec_cache_attend_selected_args*, void*, unsigned*);
int (*g_weigh)(const spec_cache_weigh_args*, void*, unsigned*);
int (*g_evict)(const spec_cache_evict_args*, void*, unsigned*);
long long (*g_evict_workspace)(const spec_cache_evict_args*);

using at::Tensor;

// Arguments of one call, taken in order.
struct Args {
  PyObject* const* x;
  int dev = -1;

  bool none() const { return *x == Py_None; }
  // The next tensor; the first one's device is the call's.
  const Tensor& tensor(const char* name) {
    PyObject* o = *x++;
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    const Tensor& t = THPVariable_Unpack(o);
    TORCH_CHECK_VALUE(!t.requires_grad() || !c10::GradMode::is_enabled(), name,
                      " requires a gradient, and the call has no backward pass: detach it, or "
                      "call under torch.no_grad()");
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must be on a CUDA device, not ", t.device());
    if (dev < 0) dev = t.get_device();
    TORCH_CHECK_VALUE(t.get_device() == dev, name, " is on ", t.device(),
                      ", other tensors on cuda:", dev);
    return t;
  }
  // A contiguous int32 tensor of n elements (any number: n < 0).
  const Tensor& ints(const char* name, int64_t n) {
    const Tensor& t = tensor(name);
    TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && t.is_contiguous() && (n < 0 || t.numel() == n),
                      name, " must be contiguous int32", n < 0 ? "" : " of ",
                      n < 0 ? std::string() : std::to_string(n) + " elements", ", not ",
                      t.scalar_type(), " ", t.sizes());
    return t;
  }
  const Tensor& table(int64_t B, long long& stride) {
    const Tensor& t = tensor("block_table");
    TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && t.dim() == 2 && t.size(0) == B &&
                          t.size(1) >= 1 && (t.stride(1) == 1 || t.size(1) == 1),
                      "block_table must be int32 [", B, ", width] with adjacent columns, not ",
                      t.scalar_type(), " ", t.sizes());
    stride = B > 1 ? t.stride(0) : std::max(t.stride(0), t.size(1));
    return t;
  }
  long long integer() {
    const long long v = PyLong_AsLongLong(*x++);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
  }
  int small(const char* name) {
    const long long v = integer();
    TORCH_CHECK_VALUE(v >= INT_MIN && v <= INT_MAX, name, " = ", v);
    return (int)v;
  }
  float number() {
    const double v = PyFloat_AsDouble(*x++);
    if (v == -1. && PyErr_Occurred()) throw python_error();
    return (float)v;
  }
  unsigned* status() {
    if (none()) return ++x, nullptr;
    const Tensor& t = tensor("status");
    TORCH_CHECK_VALUE(t.numel() == 1 && (t.scalar_type() == at::kInt ||
                                         t.scalar_type() == at::ScalarType::UInt32),
                      "status must be one 32-bit integer, not ", t.scalar_type(), " ", t.sizes());
    return (unsigned*)t.data_ptr();
  }
};

int dtype_of(const Tensor& t) {
  const auto d = t.scalar_type();
  TORCH_CHECK_TYPE(d == at::kBFloat16 || d == at::kHalf,
                   "the cache holds bfloat16 or float16, not ", d);
  return d == at::kBFloat16 ? SPEC_CACHE_BF16 : SPEC_CACHE_F16;
}

void check_pages(const Tensor& k, const Tensor& v) {
  TORCH_CHECK_VALUE(k.dim() == 4 && v.sizes() == k.sizes() && v.scalar_type() == k.scalar_type() &&
                        ((k.stride(3) == 1 && v.stride(3) == 1) || k.size(3) == 1),
                    "k_pages and v_pages must be alike, [pages, page_size, kv_heads, dim] with "
                    "adjacent elements, not ", k.scalar_type(), " ", k.sizes(), " and ",
                    v.scalar_type(), " ", v.sizes());
}

void check_rows(const char* name, const Tensor& t, int64_t tokens, int64_t heads, int64_t dim,
                at::ScalarType dtype) {
  TORCH_CHECK_VALUE(t.dim() == 3 && t.scalar_type() == dtype && (tokens < 0 || t.size(0) == tokens) &&
                        t.size(1) == heads && t.size(2) == dim && (t.stride(2) == 1 || dim == 1),
                    name, " must be ", dtype, " [", tokens < 0 ? std::string("tokens")
                    : std::to_string(tokens), ", ", heads, ", ", dim,
                    "] with adjacent elements, not ", t.scalar_type(), " ", t.sizes());
}

Tensor empty(at::IntArrayRef sizes, at::ScalarType dtype, int dev) {
  return Tensor(at::detail::empty_cuda(sizes, dtype, c10::Device(c10::kCUDA, dev), std::nullopt));
}

// n elements of a byte buffer from `at` on, as a tensor that shares its storage.
Tensor part(const Tensor& bytes, int64_t at, int64_t n, at::ScalarType dtype) {
  Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      c10::Storage(bytes.storage()), c10::DispatchKeySet(c10::DispatchKey::CUDA),
      c10::scalarTypeToTypeMeta(dtype));
  t.unsafeGetTensorImpl()->set_storage_offset(at / (int64_t)c10::elementSize(dtype));
  t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
  return t;
}

template <typename F, typename A>
int call(F fn, const A& a, int dev, unsigned* status) {
  return fn(&a, c10::cuda::getCurrentCUDAStream(dev).stream(), status);
}

// held_lens, new_lens, block_table, free_pages, free_count, page_size, num_tokens, cu_num_draft,
// num_accepted, status -> (lens, cu_new, positions, slots, free_count)
PyObject* step(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_TYPE(n == 10, "10 arguments");
  Args x{args};
  spec_cache_step_args a = {};
  const Tensor& held = x.ints("held_lens", -1);
  const int64_t B = held.numel();
  TORCH_CHECK_VALUE(B < INT_MAX, "requests: ", B);
  a.B = (int)B;
  a.held_lens = (const int*)held.data_ptr();
  a.new_lens = (const int*)x.ints("new_lens", B).data_ptr();
  const Tensor& table = x.table(B, a.table_stride);
  a.width = (int)table.size(1);
  a.block_table = (int*)table.data_ptr();
  const Tensor& free_pages = x.ints("free_pages", -1);
  TORCH_CHECK_VALUE(free_pages.numel() <= INT_MAX, "pages: ", free_pages.numel());
  a.num_pages = (int)free_pages.numel();
  a.free_pages = (int*)free_pages.data_ptr();
  a.free_count = (const int*)x.ints("free_count", 1).data_ptr();
  a.page_size = x.small("page_size");
  a.num_tokens = x.small("num_tokens");
  TORCH_CHECK_VALUE(a.num_tokens >= 0, "num_tokens = ", a.num_tokens);
  TORCH_CHECK_VALUE((x.x[0] == Py_None) == (x.x[1] == Py_None),
                    "cu_num_draft and num_accepted go together");
  if (x.none()) {
    x.x += 2;
  } else {
    a.cu_num_draft = (const int*)x.ints("cu_num_draft", B + 1).data_ptr();
    a.num_accepted = (const int*)x.ints("num_accepted", B).data_ptr();
  }
  unsigned* status = x.status();
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)x.dev);
  // Two allocations for the five outputs: the lists of tokens, which a round uses up, and the
  // few numbers that it keeps. (Five take 1.8 us more of host time than one.)
  const int64_t T = a.num_tokens;
  const Tensor few = empty({4 * (2 * B + 2)}, at::kByte, x.dev);
  const Tensor lists = empty({12 * T}, at::kByte, x.dev);
  const Tensor out[5] = {part(few, 0, B, at::kInt), part(few, 4 * B, B + 1, at::kInt),
                         part(lists, 8 * T, T, at::kInt), part(lists, 0, T, at::kLong),
                         part(few, 4 * (2 * B + 1), 1, at::kInt)};
  a.lens = (int*)out[0].data_ptr();
  a.cu_new = (int*)out[1].data_ptr();
  a.positions = (int*)out[2].data_ptr();
  a.slots = (long long*)out[3].data_ptr();
  a.free_count_out = (int*)out[4].data_ptr();
  const int rc = call(g_step, a, x.dev, status);
  if (rc != 0) return PyLong_FromLong(rc);
  PyObject* r = PyTuple_New(5);
  if (!r) throw python_error();
  for (int i = 0; i < 5; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(out[i]));
  return r;
  END_HANDLE_TH_ERRORS
}

// k, v, slots, k_pages, v_pages, status -> None
PyObject* append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_TYPE(n == 6, "6 arguments");
  Args x{args};
  spec_cache_append_args a = {};
  const Tensor& k = x.tensor("k");
  const Tensor& v = x.tensor("v");
  const Tensor& slots = x.tensor("slots");
  const Tensor& kp = x.tensor("k_pages");
  const Tensor& vp = x.tensor("v_pages");
  unsigned* status = x.status();
  a.dtype = dtype_of(kp);
  check_pages(kp, vp);
  check_rows("k", k, -1, kp.size(2), kp.size(3), kp.scalar_type());
  check_rows("v", v, k.size(0), kp.size(2), kp.size(3), kp.scalar_type());
  TORCH_CHECK_VALUE(slots.scalar_type() == at::kLong && slots.is_contiguous() &&
                        slots.numel() == k.size(0),
                    "slots must be contiguous int64 of ", k.size(0), " elements, not ",
                    slots.scalar_type(), " ", slots.sizes());
  TORCH_CHECK_VALUE(kp.size(1) <= INT_MAX && kp.size(2) <= INT_MAX && kp.size(3) <= INT_MAX,
                    "k_pages: ", kp.sizes());
  a.num_tokens = k.size(0);
  a.kv_heads = (int)kp.size(2);
  a.dim = (int)kp.size(3);
  a.page_size = (int)kp.size(1);
  a.num_pages = kp.size(0);
  a.k = k.data_ptr(), a.k_token = k.stride(0), a.k_head = k.stride(1);
  a.v = v.data_ptr(), a.v_token = v.stride(0), a.v_head = v.stride(1);
  a.slots = (const long long*)slots.data_ptr();
  a.k_pages = kp.data_ptr();
  a.kp_page = kp.stride(0), a.kp_token = kp.stride(1), a.kp_head = kp.stride(2);
  a.v_pages = vp.data_ptr();
  a.vp_page = vp.stride(0), a.vp_token = vp.stride(1), a.vp_head = vp.stride(2);
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)x.dev);
  const int rc = call(g_append, a, x.dev, status);
  if (rc != 0) return PyLong_FromLong(rc);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// q, k_pages, v_pages, block_table, kv_lens, cu_q, max_q, scale, window, sinks, out, return_lse,
// status -> out, or (out, lse)
PyObject* attend(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_TYPE(n == 13, "13 arguments");
  Args x{args};
  spec_cache_attend_args a = {};
  const Tensor& q = x.tensor("q");
  const Tensor& kp = x.tensor("k_pages");
  const Tensor& vp = x.tensor("v_pages");
  a.dtype = dtype_of(q);
  check_pages(kp, vp);
  const int64_t kv_heads = kp.size(2), dim = kp.size(3);
  TORCH_CHECK_VALUE(q.dim() == 3, "q must be [tokens, heads, dim], not ", q.sizes());
  const int64_t T = q.size(0), heads = q.size(1);
  check_rows("q", q, T, heads, dim, kp.scalar_type());
  TORCH_CHECK_VALUE(kv_heads > 0 && heads % kv_heads == 0, "q's ", heads,
                    " heads must be a multiple of the pages' ", kv_heads);
  TORCH_CHECK_VALUE(T <= INT_MAX && heads <= INT_MAX && dim <= INT_MAX && kp.size(1) <= INT_MAX,
                    "q ", q.sizes(), ", k_pages ", kp.sizes());
  PyObject* const* at_table = x.x++;  // its rows are known once the lengths are
  const Tensor& lens = x.ints("kv_lens", -1);
  const int64_t B = lens.numel();
  TORCH_CHECK_VALUE(B < INT_MAX, "requests: ", B);
  const Tensor& cu_q = x.ints("cu_q", B + 1);
  Args table_arg{at_table, x.dev};
  const Tensor& table = table_arg.table(B, a.table_stride);
  a.B = (int)B;
  a.num_tokens = (int)T;
  a.max_q = T > 0 ? (int)T : 1;
  if (x.none()) ++x.x; else a.max_q = x.small("max_q");
  a.scale = dim > 0 ? 1.0f / std::sqrt((float)dim) : 1.f;
  if (!x.none()) {
    a.scale = (float)PyFloat_AsDouble(*x.x);
    if (a.scale == -1.f && PyErr_Occurred()) throw python_error();
  }
  ++x.x;
  a.window = x.small("window");
  a.sinks = x.small("sinks");
  a.heads = (int)heads, a.kv_heads = (int)kv_heads, a.dim = (int)dim;
  a.page_size = (int)kp.size(1);
  a.width = (int)table.size(1);
  a.num_pages = kp.size(0);
  a.q = q.data_ptr(), a.q_token = q.stride(0), a.q_head = q.stride(1);
  a.k_pages = kp.data_ptr();
  a.kp_page = kp.stride(0), a.kp_token = kp.stride(1), a.kp_head = kp.stride(2);
  a.v_pages = vp.data_ptr();
  a.vp_page = vp.stride(0), a.vp_token = vp.stride(1), a.vp_head = vp.stride(2);
  a.block_table = (const int*)table.data_ptr();
  a.kv_lens = (const int*)lens.data_ptr();
  a.cu_q = (const int*)cu_q.data_ptr();
  Tensor out, lse, workspace;
  if (x.none()) {
    ++x.x;
  } else {
    out = x.tensor("out");
    check_rows("out", out, T, heads, dim, q.scalar_type());
  }
  const int return_lse = PyObject_IsTrue(*x.x++);
  if (return_lse < 0) throw python_error();
  unsigned* status = x.status();
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)x.dev);
  const long long need = g_workspace(&a);  // of the current device, now the tensors'
  if (need < 0) return PyLong_FromLongLong(need);
  if (!out.defined()) out = empty({T, heads, dim}, q.scalar_type(), x.dev);
  if (return_lse) lse = empty({T, heads}, at::kFloat, x.dev);
  workspace = empty({need}, at::kByte, x.dev);
  a.out = out.data_ptr(), a.out_token = out.stride(0), a.out_head = out.stride(1);
  a.lse = return_lse ? (float*)lse.data_ptr() : nullptr;
  a.workspace = workspace.data_ptr();
  a.workspace_bytes = (size_t)need;
  const int rc = call(g_attend, a, x.dev, status);
  if (rc != 0) return PyLong_FromLong(rc);
  if (!return_lse) return THPVariable_Wrap(out);
  PyObject* r = PyTuple_New(2);
  if (!r) throw python_error();
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(out));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(lse));
  return r;
  END_HANDLE_TH_ERRORS
}

// ---- sparse attention and eviction

// Keys alone, or another array of [pages, ., ., .] with adjacent elements.
void check_pool(const char* name, const Tensor& t) {
  TORCH_CHECK_VALUE(t.dim() == 4 && (t.stride(3) == 1 || t.size(3) == 1) && t.size(1) <= INT_MAX &&
                        t.size(2) <= INT_MAX && t.size(3) <= INT_MAX,
                    name, " must be [pages, ., ., .] with adjacent elements, not ", t.sizes());
}

void check_bounds(const Tensor& t, int64_t pages, int64_t kv_heads, int64_t dim,
                  at::ScalarType dtype) {
  check_pool("bounds", t);
  TORCH_CHECK_VALUE((pages < 0 || t.size(0) == pages) && (kv_heads < 0 || t.size(1) == kv_heads) &&
                        t.size(2) == 2 && t.size(3) == dim && t.scalar_type() == dtype,
                    "bounds must be ", dtype, " [pages, kv_heads, 2, ", dim, "], not ",
                    t.scalar_type(), " ", t.sizes());
}

void check_weights(const Tensor& t, const Tensor& pages) {
  TORCH_CHECK_VALUE(t.scalar_type() == at::kFloat && t.dim() == 3 && t.size(0) == pages.size(0) &&
                        t.size(1) == pages.size(2) && t.size(2) == pages.size(1) &&
                        (t.stride(2) == 1 || t.size(2) == 1),
                    "weights must be float32 [", pages.size(0), ", ", pages.size(2), ", ",
                    pages.size(1), "] with adjacent tokens, not ", t.scalar_type(), " ", t.sizes());
}

// The table, whose rows are known once the lengths are, the lengths and (where there are any)
// the offsets of the new tokens: block_table, kv_lens, cu_q in the arguments' order.
template <typename A>
void take_requests(Args& x, A& a, bool optional_offsets) {
  PyObject* const* at_table = x.x++;
  const Tensor& lens = x.ints("kv_lens", -1);
  const int64_t B = lens.numel();
  TORCH_CHECK_VALUE(B < INT_MAX, "requests: ", B);
  Args table_arg{at_table, x.dev};
  const Tensor& table = table_arg.table(B, a.table_stride);
  TORCH_CHECK_VALUE(table.size(1) <= INT_MAX, "block_table ", table.sizes());
  a.B = (int)B;
  a.width = (int)table.size(1);
  a.block_table = (const int*)table.data_ptr();
  a.kv_lens = (const int*)lens.data_ptr();
  if (optional_offsets && x.none())
    ++x.x;
  else
    a.cu_q = (const int*)x.ints("cu_q", B + 1).data_ptr();
}

// q's rows and, with the pages' heads and sizes, the groups.
template <typename A>
void take_heads(A& a, const Tensor& q, int64_t kv_heads, int64_t dim, at::ScalarType dtype) {
  TORCH_CHECK_VALUE(q.dim() == 3, "q must be [tokens, heads, dim], not ", q.sizes());
  check_rows("q", q, -1, q.size(1), dim, dtype);
  TORCH_CHECK_VALUE(kv_heads > 0 && q.size(1) % kv_heads == 0, "q's ", q.size(1),
                    " heads must be a multiple of the pages' ", kv_heads);
  TORCH_CHECK_VALUE(q.size(0) <= INT_MAX && q.size(1) <= INT_MAX, "q ", q.sizes());
  a.num_tokens = (int)q.size(0);
  a.heads = (int)q.size(1), a.kv_heads = (int)kv_heads, a.dim = (int)dim;
  a.q = q.data_ptr(), a.q_token = q.stride(0), a.q_head = q.stride(1);
}

template <typename A>
void take_keys(A& a, const Tensor& kp) {
  a.page_size = (int)kp.size(1);
  a.num_pages = kp.size(0);
  a.k_pages = kp.data_ptr();
  a.kp_page = kp.stride(0), a.kp_token = kp.stride(1), a.kp_head = kp.stride(2);
}
template <typename A>
void take_values(A& a, const Tensor& vp) {
  a.v_pages = vp.data_ptr();
  a.vp_page = vp.stride(0), a.vp_token = vp.stride(1), a.vp_head = vp.stride(2);
}

template <typename A>
void take_max_q(Args& x, A& a, int64_t tokens) {
  a.max_q = tokens > 0 ? (int)std::min<int64_t>(tokens, INT_MAX) : 1;
  if (x.none()) ++x.x; else a.max_q = x.small("max_q");
}

// k_pages, block_table, kv_lens, cu_q, bounds, max_q, status -> None
PyObject* bounds(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_TYPE(n == 7, "7 arguments");
  Args x{args};
  spec_cache_bounds_args a = {};
  const Tensor& kp = x.tensor("k_pages");
  a.dtype = dtype_of(kp);
  check_pool("k_pages", kp);
  take_keys(a, kp);
  a.kv_heads = (int)kp.size(2), a.dim = (int)kp.size(3);
  take_requests(x, a, true);
  const Tensor& out = x.tensor("bounds");
  check_bounds(out, kp.size(0), kp.size(2), kp.size(3), kp.scalar_type());
  a.bounds = out.data_ptr();
  a.b_page = out.stride(0), a.b_head = out.stride(1), a.b_side = out.stride(2);
  take_max_q(x, a, a.page_size * (int64_t)a.width);
  unsigned* status = x.status();
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)x.dev);
  const int rc = call(g_bounds, a, x.dev, status);
  if (rc != 0) return PyLong_FromLong(rc);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// q, bounds, block_table, kv_lens, cu_q, page_size, max_q, out, status -> scores
PyObject* score(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_TYPE(n == 9, "9 arguments");
  Args x{args};
  spec_cache_score_args a = {};
  const Tensor& q = x.tensor("q");
  const Tensor& b = x.tensor("bounds");
  a.dtype = dtype_of(q);
  check_pool("bounds", b);
  take_heads(a, q, b.size(1), b.size(3), b.scalar_type());
  check_bounds(b, -1, -1, b.size(3), q.scalar_type());
  a.num_pages = b.size(0);
  a.bounds = b.data_ptr();
  a.b_page = b.stride(0), a.b_head = b.stride(1), a.b_side = b.stride(2);
  take_requests(x, a, false);
  a.page_size = x.small("page_size");
  take_max_q(x, a, a.num_tokens);
  Tensor out;
  if (x.none()) {
    ++x.x;
  } else {
    out = x.tensor("out");
    check_rows("out", out, a.num_tokens, a.kv_heads, a.width, at::kFloat);
  }
  unsigned* status = x.status();
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)x.dev);
  if (!out.defined()) out = empty({a.num_tokens, a.kv_heads, a.width}, at::kFloat, x.dev);
  a.scores = (float*)out.data_ptr();
  a.s_token = out.stride(0), a.s_head = out.stride(1);
  const int rc = call(g_score, a, x.dev, status);
  if (rc != 0) return PyLong_FromLong(rc);
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// scores, kv_lens, cu_q, page_size, count, first, recent, out, status -> selected
PyObject* select(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_TYPE(n == 9, "9 arguments");
  Args x{args};
  spec_cache_select_args a = {};
  const Tensor& s = x.tensor("scores");
  TORCH_CHECK_VALUE(s.scalar_type() == at::kFloat && s.dim() == 3 && s.size(0) <= INT_MAX &&
                        s.size(1) <= INT_MAX && s.size(2) <= INT_MAX &&
                        (s.stride(2) == 1 || s.size(2) == 1),
                    "scores must be float32 [tokens, kv_heads, columns] with adjacent columns, "
                    "not ", s.scalar_type(), " ", s.sizes());
  a.num_tokens = (int)s.size(0), a.kv_heads = (int)s.size(1), a.width = (int)s.size(2);
  a.scores = (const float*)s.data_ptr();
  a.s_token = s.stride(0), a.s_head = s.stride(1);
  const Tensor& lens = x.ints("kv_lens", -1);
  TORCH_CHECK_VALUE(lens.numel() < INT_MAX, "requests: ", lens.numel());
  a.B = (int)lens.numel();
  a.kv_lens = (const int*)lens.data_ptr();
  a.cu_q = (const int*)x.ints("cu_q", a.B + 1ll).data_ptr();
  a.page_size = x.small("page_size");
  a.count = x.small("count");
  a.first = x.small("first");
  a.recent = x.small("recent");
  TORCH_CHECK_VALUE(a.count >= 1, "count = ", a.count);
  const int64_t size[3] = {a.num_tokens, a.kv_heads, a.count};
  Tensor out;
  if (x.none()) {
    ++x.x;
  } else {
    out = x.ints("out", size[0] * size[1] * size[2]);
    TORCH_CHECK_VALUE(out.dim() == 3 && out.size(0) == size[0] && out.size(1) == size[1],
                      "out must be [", size[0], ", ", size[1], ", ", size[2], "], not ",
                      out.sizes());
  }
  unsigned* status = x.status();
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)x.dev);
  if (!out.defined()) out = empty(size, at::kInt, x.dev);
  a.selected = (int*)out.data_ptr();
  const int rc = call(g_select, a, x.dev, status);
  if (rc != 0) return PyLong_FromLong(rc);
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// q, k_pages, v_pages, block_table, kv_lens, cu_q, selected, scale, out, return_lse, status
// -> out, or (out, lse)
PyObject* attend_selected(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_TYPE(n == 11, "11 arguments");
  Args x{args};
  spec_cache_attend_selected_args a = {};
  const Tensor& q = x.tensor("q");
  const Tensor& kp = x.tensor("k_pages");
  const Tensor& vp = x.tensor("v_pages");
  a.dtype = dtype_of(q);
  check_pages(kp, vp);
  check_pool("k_pages", kp);
  take_heads(a, q, kp.size(2), kp.size(3), kp.scalar_type());
  take_keys(a, kp);
  take_values(a, vp);
  take_requests(x, a, false);
  const Tensor& sel = x.ints("selected", -1);
  TORCH_CHECK_VALUE(sel.dim() == 3 && sel.size(0) == a.num_tokens && sel.size(1) == a.kv_heads &&
                        sel.size(2) >= 1 && sel.size(2) <= INT_MAX,
                    "selected must be [", a.num_tokens, ", ", a.kv_heads, ", count], not ",
                    sel.sizes());
  a.count = (int)sel.size(2);
  a.selected = (const int*)sel.data_ptr();
  a.scale = 1.0f / std::sqrt((float)std::max(a.dim, 1));
  if (x.none()) ++x.x; else a.scale = x.number();
  Tensor out, lse;
  if (x.none()) {
    ++x.x;
  } else {
    out = x.tensor("out");
    check_rows("out", out, a.num_tokens, a.heads, a.dim, q.scalar_type());
  }
  const int return_lse = PyObject_IsTrue(*x.x++);
  if (return_lse < 0) throw python_error();
  unsigned* status = x.status();
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)x.dev);
  if (!out.defined()) out = empty({a.num_tokens, a.heads, a.dim}, q.scalar_type(), x.dev);
  if (return_lse) lse = empty({a.num_tokens, a.heads}, at::kFloat, x.dev);
  a.out = out.data_ptr(), a.out_token = out.stride(0), a.out_head = out.stride(1);
  a.lse = return_lse ? (float*)lse.data_ptr() : nullptr;
  const int rc = call(g_selected, a, x.dev, status);
  if (rc != 0) return PyLong_FromLong(rc);
  if (!return_lse) return THPVariable_Wrap(out);
  PyObject* r = PyTuple_New(2);
  if (!r) throw python_error();
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(out));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(lse));
  return r;
  END_HANDLE_TH_ERRORS
}

// q, k_pages, block_table, kv_lens, cu_q, lse, weights, max_q, scale, decay, status -> None
PyObject* weigh(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_TYPE(n == 11, "11 arguments");
  Args x{args};
  spec_cache_weigh_args a = {};
  const Tensor& q = x.tensor("q");
  const Tensor& kp = x.tensor("k_pages");
  a.dtype = dtype_of(q);
  check_pool("k_pages", kp);
  take_heads(a, q, kp.size(2), kp.size(3), kp.scalar_type());
  take_keys(a, kp);
  take_requests(x, a, false);
  const Tensor& lse = x.tensor("lse");
  TORCH_CHECK_VALUE(lse.scalar_type() == at::kFloat && lse.is_contiguous() && lse.dim() == 2 &&
                        lse.size(0) == a.num_tokens && lse.size(1) == a.heads,
                    "lse must be contiguous float32 [", a.num_tokens, ", ", a.heads, "], not ",
                    lse.scalar_type(), " ", lse.sizes());
  a.lse = (const float*)lse.data_ptr();
  const Tensor& w = x.tensor("weights");
  check_weights(w, kp);
  a.weights = (float*)w.data_ptr();
  a.w_page = w.stride(0), a.w_head = w.stride(1);
  take_max_q(x, a, a.num_tokens);
  a.scale = 1.0f / std::sqrt((float)std::max(a.dim, 1));
  if (x.none()) ++x.x; else a.scale = x.number();
  a.decay = x.number();
  unsigned* status = x.status();
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)x.dev);
  const int rc = call(g_weigh, a, x.dev, status);
  if (rc != 0) return PyLong_FromLong(rc);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// k_pages, v_pages, weights, block_table, lens, budget, free_pages, free_count, first, recent,
// status -> (lens, free_count)
PyObject* evict(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_TYPE(n == 11, "11 arguments");
  Args x{args};
  spec_cache_evict_args a = {};
  const Tensor& kp = x.tensor("k_pages");
  const Tensor& vp = x.tensor("v_pages");
  a.dtype = dtype_of(kp);
  check_pages(kp, vp);
  check_pool("k_pages", kp);
  TORCH_CHECK_VALUE(kp.size(0) <= INT_MAX, "pages: ", kp.size(0));
  a.kv_heads = (int)kp.size(2), a.dim = (int)kp.size(3);
  a.page_size = (int)kp.size(1);
  a.num_pages = (int)kp.size(0);
  a.k_pages = kp.data_ptr();
  a.kp_page = kp.stride(0), a.kp_token = kp.stride(1), a.kp_head = kp.stride(2);
  take_values(a, vp);
  const Tensor& w = x.tensor("weights");
  check_weights(w, kp);
  a.weights = (float*)w.data_ptr();
  a.w_page = w.stride(0), a.w_head = w.stride(1);
  PyObject* const* at_table = x.x++;
  const Tensor& lens = x.ints("lens", -1);
  const int64_t B = lens.numel();
  TORCH_CHECK_VALUE(B < INT_MAX, "requests: ", B);
  Args table_arg{at_table, x.dev};
  const Tensor& table = table_arg.table(B, a.table_stride);
  TORCH_CHECK_VALUE(table.size(1) <= INT_MAX, "block_table ", table.sizes());
  a.B = (int)B;
  a.width = (int)table.size(1);
  a.block_table = (const int*)table.data_ptr();
  a.lens = (const int*)lens.data_ptr();
  a.budget = (const int*)x.ints("budget", B).data_ptr();
  a.free_pages = (int*)x.ints("free_pages", a.num_pages).data_ptr();
  a.free_count = (const int*)x.ints("free_count", 1).data_ptr();
  a.first = x.small("first");
  a.recent = x.small("recent");
  unsigned* status = x.status();
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)x.dev);
  const long long need = g_evict_workspace(&a);
  if (need < 0) return PyLong_FromLongLong(need);
  const Tensor few = empty({4 * (B + 1)}, at::kByte, x.dev);
  const Tensor workspace = empty({need}, at::kByte, x.dev);
  const Tensor out[2] = {part(few, 0, B, at::kInt), part(few, 4 * B, 1, at::kInt)};
  a.lens_out = (int*)out[0].data_ptr();
  a.free_count_out = (int*)out[1].data_ptr();
  a.workspace = workspace.data_ptr();
  a.workspace_bytes = (size_t)need;
  const int rc = call(g_evict, a, x.dev, status);
  if (rc != 0) return PyLong_FromLong(rc);
  PyObject* r = PyTuple_New(2);
  if (!r) throw python_error();
  for (int i = 0; i < 2; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(out[i]));
  return r;
  END_HANDLE_TH_ERRORS
}

// The addresses of the library's spec_cache_step, _append, _attend, _attend_workspace, _bounds,
// _score, _select, _attend_selected, _weigh, _evict, _evict_workspace.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 11) return PyErr_Format(PyExc_TypeError, "11 arguments");
  void* fn[11];
  for (int i = 0; i < 11; ++i) {
    fn[i] = PyLong_AsVoidPtr(args[i]);
    if (!fn[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
      return nullptr;
    }
  }
  g_step = (decltype(g_step))fn[0];
  g_append = (decltype(g_append))fn[1];
  g_attend = (decltype(g_attend))fn[2];
  g_workspace = (decltype(g_workspace))fn[3];
  g_bounds = (decltype(g_bounds))fn[4];
  g_score = (decltype(g_score))fn[5];
  g_select = (decltype(g_select))fn[6];
  g_selected = (decltype(g_selected))fn[7];
  g_weigh = (decltype(g_weigh))fn[8];
  g_evict = (decltype(g_evict))fn[9];
  g_evict_workspace = (decltype(g_evict_workspace))fn[10];
  Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"bind", (PyCFunction)(void*)bind, METH_FASTCALL, nullptr},
    {"step", (PyCFunction)(void*)step, METH_FASTCALL, nullptr},
    {"append", (PyCFunction)(void*)append, METH_FASTCALL, nullptr},
    {"attend", (PyCFunction)(void*)attend, METH_FASTCALL, nullptr},
    {"bounds", (PyCFunction)(void*)bounds, METH_FASTCALL, nullptr},
    {"score", (PyCFunction)(void*)score, METH_FASTCALL, nullptr},
    {"select", (PyCFunction)(void*)select, METH_FASTCALL, nullptr},
    {"attend_selected", (PyCFunction)(void*)attend_selected, METH_FASTCALL, nullptr},
    {"weigh", (PyCFunction)(void*)weigh, METH_FASTCALL, nullptr},
    {"evict", (PyCFunction)(void*)evict, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_cache_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cache_binding() { return PyModule_Create(&g_module); }
