// Torch binding of the 4-bit cache's entry points (kronq_kv4_append, _gather,
// _attention): the checks of the tensors, the outputs and workspaces that are not
// given, and the call into libkronq.so on the current stream.
//
// These run once per layer and token, and a decode step's kernels take a few
// microseconds themselves; the same checks in Python with ctypes took 13 to 18 us a
// call, here 2 to 4.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <string>

#include "../../include/kronq.h"

namespace {

namespace py = pybind11;
using at::Tensor;
using Maybe = std::optional<Tensor>;

PyObject* g_error = nullptr;      // abi.KronqError

void check(const char* fn, int code) {
  if (code == KRONQ_OK) return;
  py::object e = py::reinterpret_borrow<py::object>(g_error)(fn, code);
  PyErr_SetObject(g_error, e.ptr());
  throw py::error_already_set();
}

[[noreturn]] void bad(const std::string& what) { throw py::value_error(what); }

std::string shape(const Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

int dtype_code(const Tensor& t, const char* name, bool fp32) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return KRONQ_BF16;
    case at::kHalf: return KRONQ_FP16;
    case at::kFloat:
      if (fp32) return KRONQ_FP32;
      [[fallthrough]];
    default:
      bad(std::string(name) + " must be bfloat16" + (fp32 ? ", float16 or float32" : " or float16") + ", got " +
          c10::toString(t.scalar_type()));
  }
}

// The device all tensors of a call have to be on: the current one.
struct Device {
  c10::DeviceIndex index;
  explicit Device(const Tensor& t, const char* name) {
    if (!t.is_cuda()) bad(std::string(name) + " must be a CUDA tensor");
    index = t.get_device();
    const auto cur = c10::cuda::current_device();
    if (index != cur)
      bad(std::string(name) + " is on cuda:" + std::to_string(index) + ", the current device is cuda:" +
          std::to_string(cur));
  }
  void same(const Tensor& t, const char* name) const {
    if (!t.is_cuda() || t.get_device() != index)
      bad(std::string(name) + " is on " + t.device().str() + ", expected cuda:" + std::to_string(index));
  }
};

// A T x heads x D tensor with a contiguous last dimension.
void rows(const Tensor& t, const char* name, at::ScalarType type, int64_t T, int64_t D, const Device& dev) {
  if (t.scalar_type() != type)
    bad(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
  if (t.dim() != 3 || t.size(0) != T || t.size(2) != D)
    bad(std::string(name) + " has shape " + shape(t) + ", expected (" + std::to_string(T) + ", heads, " +
        std::to_string(D) + ")");
  if (t.stride(2) != 1) bad(std::string(name) + " needs unit stride along its last dimension");
  dev.same(t, name);
}

// A contiguous tensor of `count` elements (none: NULL).
template <class P>
P* vector(const Maybe& t, const char* name, at::ScalarType type, int64_t count, const Device& dev) {
  if (!t) return nullptr;
  if (t->scalar_type() != type || t->numel() != count || !t->is_contiguous())
    bad(std::string(name) + " must hold " + std::to_string(count) + " " + c10::toString(type) +
        " elements in order, got " + c10::toString(t->scalar_type()) + " " + shape(*t));
  dev.same(*t, name);
  return static_cast<P*>(t->data_ptr());
}

// The (cache, batch) part of a call.
struct Cache {
  uint8_t* data;
  int64_t pages, ld, max_pages, B;
  int page, heads, D;
  const int32_t *table, *q_start, *kv_len;

  Cache(const Tensor& cache, const Tensor& bt, const Tensor& qs, const Tensor& kv, int64_t head_dim,
        const Device& dev) {
    if (cache.scalar_type() != at::kByte || cache.dim() != 3 || !cache.is_contiguous())
      bad("cache must be a contiguous uint8 tensor of 3 dims (pages, heads, bytes)");
    if (bt.scalar_type() != at::kInt || qs.scalar_type() != at::kInt || kv.scalar_type() != at::kInt)
      bad("block_table, q_start and kv_len must be int32");
    if (bt.dim() != 2 || qs.dim() != 1 || kv.dim() != 1) bad("block_table has 2 dims, q_start and kv_len have 1");
    B = bt.size(0);
    max_pages = bt.size(1);
    if (qs.size(0) != B + 1 || kv.size(0) != B)
      bad("block_table has " + std::to_string(B) + " rows, q_start " + std::to_string(qs.size(0)) + " entries (" +
          std::to_string(B + 1) + " expected), kv_len " + std::to_string(kv.size(0)) + " (" + std::to_string(B) +
          " expected)");
    if ((max_pages > 1 && bt.stride(1) != 1) || !qs.is_contiguous() || !kv.is_contiguous())
      bad("block_table, q_start and kv_len need unit stride along their last dimension");
    ld = B > 1 ? bt.stride(0) : max_pages;
    if (ld < max_pages) bad("block_table's rows overlap");
    pages = cache.size(0);
    if (cache.size(1) > INT32_MAX || head_dim > INT32_MAX || cache.size(2) / (head_dim + 8) > INT32_MAX)
      bad("cache has shape " + shape(cache));
    heads = (int)cache.size(1);
    D = (int)head_dim;
    page = (int)(cache.size(2) / (head_dim + 8));
    if ((int64_t)page * (head_dim + 8) != cache.size(2))
      bad("a cache block of " + std::to_string(cache.size(2)) + " bytes does not hold whole tokens of head_dim " +
          std::to_string(head_dim));
    dev.same(cache, "cache");
    dev.same(bt, "block_table");
    dev.same(qs, "q_start");
    dev.same(kv, "kv_len");
    data = cache.data_ptr<uint8_t>();
    table = bt.data_ptr<int32_t>();
    q_start = qs.data_ptr<int32_t>();
    kv_len = kv.data_ptr<int32_t>();
  }
};

// The current stream: outputs and workspaces that are allocated here belong to it too, so a
// call cannot be given another one.
void* stream_of(const Device& dev) { return c10::cuda::getCurrentCUDAStream(dev.index).stream(); }

// 3-dim inputs before their sizes are used
void three(const Tensor& t, const char* name) {
  if (t.dim() != 3) bad(std::string(name) + " must have 3 dims, got " + shape(t));
}

std::optional<Tensor> append(const Maybe& q, const Tensor& k, const Tensor& v, const Tensor& cache,
                             const Tensor& block_table, const Tensor& q_start, const Tensor& kv_len, Maybe q_out,
                             const Maybe& table, bool interleaved, const Maybe& positions, const Maybe& signs,
                             const Maybe& info) {
  three(k, "k");
  const int dt = dtype_code(k, "k", false);
  const auto type = k.scalar_type();
  const int64_t T = k.size(0), heads = k.size(1), D = k.size(2);
  const Device dev(k, "k");
  rows(k, "k", type, T, D, dev);
  rows(v, "v", type, T, D, dev);
  const Cache c(cache, block_table, q_start, kv_len, D, dev);
  if (v.size(1) != heads || c.heads != heads) bad("k, v and the cache differ in their heads");
  int q_heads = 0;
  if (q) {
    rows(*q, "q", type, T, D, dev);
    if (q->size(1) > INT32_MAX) bad("q has shape " + shape(*q));
    q_heads = (int)q->size(1);
    if (!q_out) {
      q_out = at::empty(q->sizes(), q->options());
    } else {
      if (q_out->scalar_type() != type || q_out->sizes() != q->sizes() || !q_out->is_contiguous())
        bad("q_out must be contiguous with q's type and shape");
      dev.same(*q_out, "q_out");
    }
  } else if (q_out) {
    bad("q and q_out go together");
  }
  int64_t n_rows = 0, rot = 0;
  if (table) {
    if (table->dim() != 2 || table->size(1) > INT32_MAX) bad("table must have 2 dims (positions, rot), got " + shape(*table));
    n_rows = table->size(0);
    rot = table->size(1);
  }
  const float* tp = vector<float>(table, "table", at::kFloat, n_rows * rot, dev);
  const int32_t* pp = vector<int32_t>(positions, "positions", at::kInt, T, dev);
  const int8_t* sp = vector<int8_t>(signs, "signs", at::kChar, D, dev);
  int32_t* ip = vector<int32_t>(info, "info", at::kInt, 1, dev);
  check("kronq_kv4_append",
        kronq_kv4_append(q ? q->data_ptr() : nullptr, q ? q->stride(0) : 0, q ? q->stride(1) : 0, k.data_ptr(),
                         k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1), dt, T, q_heads,
                         q_heads ? q_out->data_ptr() : nullptr, tp, n_rows, (int)rot, interleaved, pp, sp, c.data,
                         c.pages, c.page, c.heads, c.D, c.table, c.ld, c.max_pages, c.q_start, c.kv_len, c.B, ip,
                         stream_of(dev)));
  return q_out;
}

void gather(const Tensor& cache, const Tensor& block_table, const Tensor& q_start, const Tensor& kv_len,
            const Tensor& k_out, const Tensor& v_out, const Maybe& info) {
  three(k_out, "k_out");
  const int dt = dtype_code(k_out, "k_out", true);
  const Device dev(k_out, "k_out");
  if (!k_out.is_contiguous()) bad("k_out must be contiguous");
  if (v_out.scalar_type() != k_out.scalar_type() || v_out.sizes() != k_out.sizes() || !v_out.is_contiguous())
    bad("v_out must be contiguous with k_out's type and shape");
  dev.same(v_out, "v_out");
  const Cache c(cache, block_table, q_start, kv_len, k_out.size(2), dev);
  if (k_out.size(1) != c.heads) bad("k_out and the cache differ in their heads");
  int32_t* ip = vector<int32_t>(info, "info", at::kInt, 1, dev);
  check("kronq_kv4_gather",
        kronq_kv4_gather(k_out.data_ptr(), v_out.data_ptr(), dt, k_out.size(0), c.data, c.pages, c.page, c.heads, c.D,
                         c.table, c.ld, c.max_pages, c.q_start, c.kv_len, c.B, ip, stream_of(dev)));
}

std::pair<Tensor, Tensor> gather_new(const Tensor& cache, const Tensor& block_table, const Tensor& q_start,
                                     const Tensor& kv_len, int64_t tokens, int64_t head_dim, at::ScalarType type,
                                     const Maybe& info) {
  three(cache, "cache");
  if (tokens < 0 || head_dim <= 0) bad("tokens and head_dim must not be negative");
  const auto options = cache.options().dtype(type);
  const std::array<int64_t, 3> sizes = {tokens, cache.size(1), head_dim};
  Tensor k = at::empty(sizes, options), v = at::empty(sizes, options);
  gather(cache, block_table, q_start, kv_len, k, v, info);
  return {k, v};
}

Tensor attention(const Tensor& q, const Tensor& cache, const Tensor& block_table, const Tensor& q_start,
                 const Tensor& kv_len, Maybe out, Maybe ws, std::optional<double> scale, bool causal, int64_t window,
                 int64_t sinks, const Maybe& lse, const Maybe& info) {
  three(q, "q");
  const int dt = dtype_code(q, "q", false);
  const int64_t T = q.size(0), q_heads = q.size(1), D = q.size(2);
  const Device dev(q, "q");
  rows(q, "q", q.scalar_type(), T, D, dev);
  const Cache c(cache, block_table, q_start, kv_len, D, dev);
  if (q_heads > INT32_MAX) bad("q has shape " + shape(q));
  if (window < 0 || sinks < 0) bad("window and sinks must not be negative");
  if (!out) {
    out = at::empty(q.sizes(), q.options());
  } else {
    rows(*out, "out", q.scalar_type(), T, D, dev);
    if (out->size(1) != q_heads) bad("out has shape " + shape(*out) + ", expected " + shape(q));
  }
  if (lse && (lse->dim() != 2 || lse->size(0) != T || lse->size(1) != q_heads))
    bad("lse has shape " + shape(*lse) + ", expected (" + std::to_string(T) + ", " + std::to_string(q_heads) + ")");
  float* lp = vector<float>(lse, "lse", at::kFloat, T * q_heads, dev);
  int32_t* ip = vector<int32_t>(info, "info", at::kInt, 1, dev);
  if (!ws) {
    const size_t n = kronq_kv4_attention_workspace_size(T, (int)q_heads, c.heads, c.D, c.B);
    ws = at::empty({(int64_t)(n > 256 ? n : 256)}, q.options().dtype(at::kByte));
  } else {
    if (!ws->is_contiguous()) bad("ws must be contiguous");
    dev.same(*ws, "ws");
  }
  const int far = 1 << 30;      // wider than any sequence
  check("kronq_kv4_attention",
        kronq_kv4_attention(q.data_ptr(), q.stride(0), q.stride(1), dt, T, (int)q_heads, c.data, c.pages, c.page,
                            c.heads, c.D, c.table, c.ld, c.max_pages, c.q_start, c.kv_len, c.B,
                            (float)(scale ? *scale : 1.0 / std::sqrt((double)D)), causal,
                            (int)std::min<int64_t>(window, far), (int)std::min<int64_t>(sinks, far), out->data_ptr(),
                            out->stride(0), out->stride(1), lp, ip, ws->data_ptr(),
                            (size_t)ws->numel() * ws->element_size(), stream_of(dev)));
  return *out;
}

}  // namespace

PYBIND11_MODULE(_kv4, m) {
  m.doc() = "Torch binding of kronq_kv4_append, kronq_kv4_gather and kronq_kv4_attention (include/kronq.h).";
  m.def("set_error", [](const py::object& cls) {
    Py_XDECREF(g_error);
    g_error = py::object(cls).release().ptr();
  });
  m.def("append", &append);
  m.def("gather", &gather);
  m.def("gather_new", &gather_new);
  m.def("attention", &attention);
}
