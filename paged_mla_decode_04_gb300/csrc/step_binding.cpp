// Python binding of the prefill-step, shared-prefix and compact-store calls: checks the
// tensors and calls the C entry points of include/mla_decode.h.
//
// A step's calls come once per layer with a dozen tensors each, and a small
// step's kernels take less time than marshalling those through ctypes did (10 to
// 13 us a call, 7 of them checks and conversions). Here they take below one.
// The library itself stays free of Python and PyTorch: its entry points arrive
// as addresses (bind).
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <exception>
#include <string>

#include "../../include/mla_decode.h"

namespace {

decltype(&mla_extend_tables) extend_tables_fn = nullptr;
decltype(&mla_rope_write) rope_write_fn = nullptr;
decltype(&mla_prefill) prefill_fn = nullptr;
decltype(&mla_decode_shared) decode_shared_fn = nullptr;
decltype(&mla_decode_plan_shared) plan_shared_fn = nullptr;
decltype(&mla_decode_workspace_size_shared) shared_size_fn = nullptr;
decltype(&mla_quant_write) quant_write_fn = nullptr;
decltype(&mla_quant_read) quant_read_fn = nullptr;

constexpr int64_t kLatentDim = 576, kCkvDim = 512, kNopeDim = 128, kRopeDim = 64, kQkDim = 192, kVDim = 128;
constexpr auto kI32 = at::kInt, kI64 = at::kLong, kBf16 = at::kBFloat16, kF32 = at::kFloat;

struct ValueError {
  std::string what;
};
struct PythonError {};  // one is set already

[[noreturn]] void refuse(const std::string& what) { throw ValueError{what}; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a CUDA tensor");
  return THPVariable_Unpack(o);
}

// Pointer of a contiguous tensor on the current device.
void* here(const at::Tensor& t, const char* name, int device) {
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  if (t.get_device() != device)
    refuse(std::string(name) + " is on cuda:" + std::to_string(t.get_device()) + ", the current device is cuda:" +
           std::to_string(device));
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  return t.data_ptr();
}

template <typename T>
T* here(const at::Tensor& t, const char* name, at::ScalarType type, int device) {
  void* p = here(t, name, device);
  if (t.scalar_type() != type)
    refuse(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
  return static_cast<T*>(p);
}

template <typename T = void>
T* here(PyObject* o, const char* name, at::ScalarType type, int device) {
  return here<T>(tensor(o, name), name, type, device);
}

template <typename T = void>
T* here_or_none(PyObject* o, const char* name, at::ScalarType type, int device) {
  return o == Py_None ? nullptr : here<T>(o, name, type, device);
}

// A workspace for the status word alone: decode's and prefill's begin with it.
void* status_workspace(PyObject* o, int device) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, "workspace");
  void* p = here(t, "workspace", device);
  if (t.nbytes() < 256) refuse("workspace must hold 256 bytes at least");
  return p;
}

int int_of(int64_t v, const char* name) {
  if (v > INT_MAX || v < INT_MIN) refuse(std::string(name) + " is out of range");
  return static_cast<int>(v);
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return v;
}

int integer32(PyObject* o, const char* name) { return int_of(integer(o), name); }

float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return static_cast<float>(v);
}

void* stream_of(PyObject* o, int device) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
  if (!h) throw PythonError{};
  void* p = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (PyErr_Occurred()) throw PythonError{};
  return p;
}

mla_kv_pool pool_of(PyObject* data, PyObject* scale, int device) {
  const at::Tensor& d = tensor(data, "pool");
  if (d.dim() != 4 || d.size(3) != kLatentDim) refuse("pool must be [num_layers, num_pages, page_size, 576]");
  const auto type = d.scalar_type();
  if (type != kBf16 && type != at::kByte) refuse("pool dtype must be bfloat16 or uint8 (e4m3 codes)");
  mla_kv_pool p = {};
  p.data = here(d, "pool", device);
  p.num_layers = int_of(d.size(0), "num_layers");
  p.num_pages = int_of(d.size(1), "num_pages");
  p.page_size = int_of(d.size(2), "page_size");
  p.dtype = type == kBf16 ? MLA_DTYPE_BF16 : MLA_DTYPE_FP8_E4M3;
  p.kv_scale = real(scale);
  return p;
}

mla_quant_pool store_of(PyObject* data, int device) {
  const at::Tensor& d = tensor(data, "store");
  const int64_t row = d.dim() == 4 ? d.size(3) : 0;
  if (d.scalar_type() != at::kByte || (row != MLA_QUANT_E4M3_ROW && row != MLA_QUANT_E2M1_ROW))
    refuse("store must be uint8 [num_layers, num_pages, page_size, 656 (e4m3) or 416 (e2m1)]");
  mla_quant_pool p = {};
  p.data = here(d, "store", device);
  p.num_layers = int_of(d.size(0), "num_layers");
  p.num_pages = int_of(d.size(1), "num_pages");
  p.page_size = int_of(d.size(2), "page_size");
  p.format = row == MLA_QUANT_E4M3_ROW ? MLA_QUANT_E4M3 : MLA_QUANT_E2M1;
  return p;
}

const int64_t* slots_of(PyObject* o, const char* name, int64_t rows, int device) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != 1 || t.numel() != rows) refuse(std::string(name) + " must be [rows]");
  return here<int64_t>(t, name, kI64, device);
}

// Runs a call's body: its status code as an int, or an exception.
template <typename F>
PyObject* call(Py_ssize_t got, Py_ssize_t want, F&& body) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, got);
    return nullptr;
  }
  try {
    return PyLong_FromLong(body());
  } catch (const ValueError& e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (const PythonError&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

template <typename F>
int without_gil(F&& f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = f();
  Py_END_ALLOW_THREADS;
  return rc;
}

PyObject* extend_tables(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return call(n, 15, [&] {
    const int dev = c10::cuda::current_device();
    const at::Tensor &lens = tensor(v[0], "context_lens"), &add = tensor(v[1], "new_lens"), &free = tensor(v[2], "free_pages"),
                     &count = tensor(v[3], "free_count"), &table = tensor(v[4], "block_table"),
                     &slots = tensor(v[7], "slot_mapping"), &indptr = tensor(v[8], "q_indptr"), &state = tensor(v[9], "state");
    const int64_t batch = lens.numel(), tokens = slots.numel();
    if (lens.dim() != 1 || add.dim() != 1 || add.numel() != batch) refuse("context_lens and new_lens must be [batch]");
    if (table.dim() != 2 || table.size(0) != batch) refuse("block_table must be [batch, max_blocks]");
    if (slots.dim() != 1) refuse("slot_mapping and positions must be [max_tokens]");
    if (v[10] != Py_None) {
      const at::Tensor& p = tensor(v[10], "positions");
      if (p.dim() != 1 || p.numel() != tokens) refuse("slot_mapping and positions must be [max_tokens]");
    }
    if (indptr.dim() != 1 || indptr.numel() != batch + 1) refuse("q_indptr must be [batch + 1]");
    if ((v[11] == Py_None) != (v[12] == Py_None)) refuse("give page_indptr and page_ids together");
    int64_t max_ids = 0;
    if (v[11] != Py_None) {
      const at::Tensor& p = tensor(v[11], "page_indptr");
      if (p.dim() != 1 || p.numel() != batch + 1) refuse("page_indptr must be [batch + 1]");
      max_ids = tensor(v[12], "page_ids").numel();
    }
    if (count.numel() < 1 || state.numel() < 2) refuse("free_count needs one element and state two");
    const int page_size = integer32(v[5], "page_size"), num_pages = integer32(v[6], "num_pages");
    const auto* lens_p = here<int32_t>(lens, "context_lens", kI32, dev);
    const auto* add_p = here<int32_t>(add, "new_lens", kI32, dev);
    const auto* free_p = here<int32_t>(free, "free_pages", kI32, dev);
    const auto* count_p = here<int32_t>(count, "free_count", kI32, dev);
    auto* table_p = here<int32_t>(table, "block_table", kI32, dev);
    auto* slots_p = here<int64_t>(slots, "slot_mapping", kI64, dev);
    auto* positions_p = here_or_none<int32_t>(v[10], "positions", kI32, dev);
    auto* indptr_p = here<int32_t>(indptr, "q_indptr", kI32, dev);
    auto* page_indptr_p = here_or_none<int32_t>(v[11], "page_indptr", kI32, dev);
    auto* ids_p = here_or_none<int32_t>(v[12], "page_ids", kI32, dev);
    auto* state_p = here<int32_t>(state, "state", kI32, dev);
    void* ws = status_workspace(v[13], dev);
    void* stream = stream_of(v[14], dev);
    const int b = int_of(batch, "batch"), capacity = int_of(free.numel(), "free_pages"), width = int_of(table.size(1), "max_blocks"),
              t = int_of(tokens, "max_tokens"), ids = int_of(max_ids, "max_page_ids");
    return without_gil([&] {
      return extend_tables_fn(lens_p, add_p, b, page_size, num_pages, free_p, count_p, capacity, table_p, width, slots_p,
                              positions_p, t, indptr_p, page_indptr_p, ids_p, ids, state_p, ws, stream);
    });
  });
}

// The rope dims [tokens, heads, 64] of queries: a view whose (token, head) rows lie
// at one pitch.
struct HeadRows {
  void* p = nullptr;
  int64_t pitch = 0, heads = 0;
};

HeadRows head_rows(PyObject* o, const char* name, int64_t tokens, int device) {
  const at::Tensor& t = tensor(o, name);
  if (!t.is_cuda() || t.get_device() != device) refuse(std::string(name) + " must be a CUDA tensor on the current device");
  if (t.scalar_type() != kBf16 || t.dim() != 3 || t.size(0) != tokens || t.size(2) != kRopeDim)
    refuse(std::string(name) + " must be bfloat16 [tokens, heads, 64]");
  HeadRows r;
  r.heads = t.size(1);
  const bool many_heads = r.heads > 1, many_tokens = tokens > 1;
  if (t.stride(2) != 1 || (many_heads && many_tokens && t.stride(0) != r.heads * t.stride(1)))
    refuse(std::string(name) + ": the (token, head) rows must lie at one pitch");
  r.pitch = many_heads ? t.stride(1) : many_tokens ? t.stride(0) : kRopeDim;
  r.p = t.data_ptr();
  return r;
}

PyObject* rope_write(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return call(n, 15, [&]() -> int {
    const int dev = c10::cuda::current_device();
    PyObject *data = v[0], *scale = v[1], *rows = v[3], *slots = v[4], *weight = v[7], *axis_of = v[11];
    const at::Tensor &pos = tensor(v[5], "positions"), &cos_sin = tensor(v[6], "cos_sin");
    if (pos.dim() != 1 && pos.dim() != 2) refuse("positions must be [tokens] or [axes, tokens]");
    const int64_t axes = pos.dim() == 2 ? pos.size(0) : 1, tokens = pos.size(-1);
    if (cos_sin.dim() != 2 || cos_sin.size(1) != kRopeDim) refuse("cos_sin must be [positions, 64]");
    const int64_t* slots_p = nullptr;
    const void *rows_p = nullptr, *weight_p = nullptr;
    mla_kv_pool pool = {};
    if (slots != Py_None) {
      const at::Tensor& t = tensor(slots, "slot_mapping");
      if (t.dim() != 1 || t.numel() != tokens) refuse("slot_mapping must be [tokens]");
      slots_p = here<int64_t>(t, "slot_mapping", kI64, dev);
    }
    if (rows != Py_None) {
      const at::Tensor& t = tensor(rows, "rows");
      if (data == Py_None || !slots_p || t.dim() != 2 || t.size(0) != tokens || t.size(1) != kLatentDim)
        refuse("rows [tokens, 576] go with pool and slot_mapping");
      rows_p = here<void>(t, "rows", kBf16, dev);
      pool = pool_of(data, scale, dev);
    }
    if (weight != Py_None) {
      const at::Tensor& t = tensor(weight, "norm_weight");
      if (t.numel() != kCkvDim) refuse("norm_weight must be [512]");
      weight_p = here<void>(t, "norm_weight", kBf16, dev);
    }
    const uint8_t* axis_p = nullptr;
    if (axis_of != Py_None) {
      if (!PyBytes_Check(axis_of) || PyBytes_GET_SIZE(axis_of) != kRopeDim / 2)
        refuse("pair_axis must name an axis for each of the 32 pairs");
      axis_p = reinterpret_cast<const uint8_t*>(PyBytes_AS_STRING(axis_of));
      for (int j = 0; j < kRopeDim / 2; ++j)
        if (axis_p[j] >= axes) refuse("pair_axis names an axis that positions lacks");
    }
    HeadRows q, o;
    if (v[9] != Py_None) {
      q = o = head_rows(v[9], "q_rope", tokens, dev);
      if (v[10] != Py_None) {
        o = head_rows(v[10], "q_out", tokens, dev);
        if (o.heads != q.heads) refuse("q_rope and q_out must be [tokens, heads, 64]");
      }
      if (q.heads == 0) q.p = o.p = nullptr;
    } else if (v[10] != Py_None) {
      refuse("q_out goes with q_rope");
    } else if (rows == Py_None) {
      refuse("give rows, q_rope or both");
    }
    if (tokens == 0 || (!q.p && !rows_p)) return MLA_OK;
    const int layer = integer32(v[2], "layer"), interleaved = PyObject_IsTrue(v[12]);
    if (interleaved < 0) throw PythonError{};
    const float eps = real(v[8]);
    const auto* pos_p = here<int32_t>(pos, "positions", kI32, dev);
    const auto* cs_p = here<float>(cos_sin, "cos_sin", kF32, dev);
    void* ws = status_workspace(v[13], dev);
    void* stream = stream_of(v[14], dev);
    const int t = int_of(tokens, "tokens"), ax = int_of(axes, "axes"), table = int_of(cos_sin.size(0), "positions"),
              heads = int_of(q.heads, "heads");
    return without_gil([&] {
      return rope_write_fn(rows_p ? &pool : nullptr, layer, rows_p, slots_p, t, pos_p, ax, axis_p, cs_p, table, interleaved,
                           weight_p, eps, q.p, q.pitch, o.p, o.pitch, heads, ws, stream);
    });
  });
}

PyObject* prefill(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return call(n, 18, [&] {
    const int dev = c10::cuda::current_device();
    const at::Tensor &q = tensor(v[3], "q"), &indptr = tensor(v[4], "q_indptr"), &lens = tensor(v[5], "context_lens"),
                     &uk = tensor(v[7], "w_uk"), &uv = tensor(v[8], "w_uv"), &work = tensor(v[9], "workspace"),
                     &out = tensor(v[10], "out");
    if (q.dim() != 3 || q.size(2) != kQkDim) refuse("q must be [rows, heads, 192]");
    const int64_t rows = q.size(0), heads = q.size(1), batch = lens.numel();
    const bool has_lse = v[16] != Py_None;
    if (!out.sizes().equals({rows, heads, kVDim}) || (has_lse && !tensor(v[16], "lse").sizes().equals({rows, heads})))
      refuse("out must be [rows, heads, 128], lse [rows, heads]");
    if (lens.dim() != 1) refuse("context_lens must be [batch]");
    if (indptr.dim() != 1 || indptr.numel() != batch + 1) refuse("q_indptr must be [batch + 1]");
    if (!uk.sizes().equals({heads, kNopeDim, kCkvDim}) || !uv.sizes().equals({heads, kCkvDim, kVDim}))
      refuse("w_uk [heads, 128, 512] and w_uv [heads, 512, 128] expected");
    const int32_t *page_indptr = nullptr, *ids = nullptr;
    int64_t max_blocks = 0;
    if (v[12] != Py_None) {
      const at::Tensor& t = tensor(v[12], "block_table");
      if (t.dim() != 2 || t.size(0) != batch) refuse("block_table must be [batch, max_blocks]");
      ids = here<int32_t>(t, "block_table", kI32, dev);
      max_blocks = t.size(1);
    } else {
      if (v[13] == Py_None || v[14] == Py_None) refuse("give block_table, or page_indptr [batch+1] and page_ids");
      const at::Tensor& t = tensor(v[13], "page_indptr");
      if (t.dim() != 1 || t.numel() != batch + 1) refuse("give block_table, or page_indptr [batch+1] and page_ids");
      page_indptr = here<int32_t>(t, "page_indptr", kI32, dev);
      ids = here<int32_t>(v[14], "page_ids", kI32, dev);
    }
    const mla_kv_pool pool = pool_of(v[0], v[1], dev);
    const int layer = integer32(v[2], "layer"), window = integer32(v[15], "window");
    const int64_t max_kv = integer(v[11]);
    const float scale = real(v[6]);
    const auto* q_p = here<void>(q, "q", kBf16, dev);
    const auto* indptr_p = here<int32_t>(indptr, "q_indptr", kI32, dev);
    const auto* lens_p = here<int32_t>(lens, "context_lens", kI32, dev);
    const auto *uk_p = here<void>(uk, "w_uk", kBf16, dev), *uv_p = here<void>(uv, "w_uv", kBf16, dev);
    void *work_p = here(work, "workspace", dev), *out_p = here<void>(out, "out", kBf16, dev);
    float* lse_p = here_or_none<float>(v[16], "lse", kF32, dev);
    void* stream = stream_of(v[17], dev);
    const int blocks = int_of(max_blocks, "max_blocks"), b = int_of(batch, "batch"), r = int_of(rows, "rows"),
              h = int_of(heads, "heads");
    const size_t bytes = work.nbytes();
    return without_gil([&] {
      return prefill_fn(&pool, layer, q_p, indptr_p, page_indptr, ids, blocks, lens_p, b, r, max_kv, h, uk_p, uv_p, scale,
                        window, work_p, bytes, out_p, lse_p, stream);
    });
  });
}

PyObject* plan_shared(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return call(n, 9, [&] {
    const int dev = c10::cuda::current_device();
    const at::Tensor &lens = tensor(v[0], "context_lens"), &indptr = tensor(v[1], "prefix_indptr"),
                     &prefix = tensor(v[2], "prefix_lens"), &work = tensor(v[6], "workspace");
    if (lens.dim() != 1 || prefix.dim() != 1 || indptr.dim() != 1 || indptr.numel() != prefix.numel() + 1)
      refuse("context_lens [batch], prefix_lens [prefixes] and prefix_indptr [prefixes + 1] expected");
    const int q_len = integer32(v[3], "q_len"), heads = integer32(v[4], "num_heads"), page = integer32(v[5], "page_size"),
              clusters = integer32(v[7], "num_clusters");
    const auto* lens_p = here<int32_t>(lens, "context_lens", kI32, dev);
    const auto* indptr_p = here<int32_t>(indptr, "prefix_indptr", kI32, dev);
    const auto* prefix_p = here<int32_t>(prefix, "prefix_lens", kI32, dev);
    void* work_p = here(work, "workspace", dev);
    void* stream = stream_of(v[8], dev);
    const int batch = int_of(lens.numel(), "batch"), prefixes = int_of(prefix.numel(), "prefixes");
    const size_t bytes = work.nbytes();
    return without_gil([&] {
      return plan_shared_fn(lens_p, indptr_p, prefix_p, batch, prefixes, q_len, heads, page, clusters, work_p, bytes, stream);
    });
  });
}

PyObject* decode_shared(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return call(n, 13, [&]() -> int {
    const int dev = c10::cuda::current_device();
    const at::Tensor &q = tensor(v[3], "q"), &work = tensor(v[6], "workspace"), &out = tensor(v[7], "out");
    if (q.dim() != 4 || q.size(3) != kLatentDim) refuse("q must be [batch, q_len, heads, 576]");
    const int64_t batch = q.size(0), q_len = q.size(1), heads = q.size(2);
    const bool has_lse = v[11] != Py_None;
    if (!out.sizes().equals({batch, q_len, heads, kCkvDim}) || (has_lse && !tensor(v[11], "lse").sizes().equals({batch, q_len, heads})))
      refuse("out must be [batch, q_len, heads, 512], lse [batch, q_len, heads]");
    const int32_t *page_indptr = nullptr, *ids = nullptr;
    int64_t max_blocks = 0;
    if (v[8] != Py_None) {
      const at::Tensor& t = tensor(v[8], "block_table");
      if (t.dim() != 2 || t.size(0) != batch) refuse("block_table must be [batch, max_blocks]");
      ids = here<int32_t>(t, "block_table", kI32, dev);
      max_blocks = t.size(1);
    } else {
      if (v[9] == Py_None || v[10] == Py_None) refuse("give block_table, or page_indptr [batch+1] and page_ids");
      const at::Tensor& t = tensor(v[9], "page_indptr");
      if (t.dim() != 1 || t.numel() != batch + 1) refuse("give block_table, or page_indptr [batch+1] and page_ids");
      page_indptr = here<int32_t>(t, "page_indptr", kI32, dev);
      ids = here<int32_t>(v[10], "page_ids", kI32, dev);
    }
    const mla_kv_pool pool = pool_of(v[0], v[1], dev);
    const int layer = integer32(v[2], "layer"), prefixes = integer32(v[4], "num_prefixes");
    const float scale = real(v[5]);
    const auto* q_p = here<void>(q, "q", kBf16, dev);
    void *work_p = here(work, "workspace", dev), *out_p = here<void>(out, "out", kBf16, dev);
    float* lse_p = here_or_none<float>(v[11], "lse", kF32, dev);
    void* stream = stream_of(v[12], dev);
    const int blocks = int_of(max_blocks, "max_blocks"), b = int_of(batch, "batch"), l = int_of(q_len, "q_len"),
              h = int_of(heads, "heads");
    const size_t bytes = work.nbytes();
    return without_gil([&] {
      // (the plan looked at the workspace's size; another one's is refused here)
      if (b > 0 && prefixes > 0 && bytes < shared_size_fn(b, l, h, prefixes)) return MLA_ERR_WORKSPACE;
      return decode_shared_fn(&pool, layer, q_p, page_indptr, ids, blocks, b, l, h, prefixes, scale, work_p, out_p, lse_p, stream);
    });
  });
}

PyObject* quant_write(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return call(n, 6, [&]() -> int {
    const int dev = c10::cuda::current_device();
    const mla_quant_pool store = store_of(v[0], dev);
    const int layer = integer32(v[1], "layer");
    const at::Tensor& rows = tensor(v[2], "rows");
    if (rows.dim() != 2 || rows.size(1) != kLatentDim) refuse("rows must be [rows, 576]");
    const void* rows_p = here<void>(rows, "rows", kBf16, dev);
    const int64_t* slots_p = slots_of(v[3], "slot_mapping", rows.size(0), dev);
    void* ws = status_workspace(v[4], dev);
    void* stream = stream_of(v[5], dev);
    const int t = int_of(rows.size(0), "rows");
    return without_gil([&] { return quant_write_fn(&store, layer, rows_p, slots_p, t, ws, stream); });
  });
}

PyObject* quant_read(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return call(n, 10, [&]() -> int {
    const int dev = c10::cuda::current_device();
    const mla_quant_pool store = store_of(v[0], dev);
    const int layer = integer32(v[1], "layer");
    const int64_t count = tensor(v[2], "slots").numel();
    const int64_t* slots_p = slots_of(v[2], "slots", count, dev);
    void* rows_p = nullptr;
    const int64_t* into_p = nullptr;
    mla_kv_pool pool = {};
    int into_layer = 0;
    const bool into = v[4] != Py_None;
    if (into == (v[3] != Py_None)) refuse("give rows, or pool with pool_slots");
    if (into) {
      pool = pool_of(v[4], v[5], dev);
      into_layer = integer32(v[6], "pool_layer");
      into_p = slots_of(v[7], "pool_slots", count, dev);
    } else {
      const at::Tensor& rows = tensor(v[3], "rows");
      if (v[7] != Py_None) refuse("pool_slots go with pool");
      if (rows.dim() != 2 || rows.size(0) != count || rows.size(1) != kLatentDim) refuse("rows must be [slots, 576]");
      rows_p = here<void>(rows, "rows", kBf16, dev);
    }
    void* ws = status_workspace(v[8], dev);
    void* stream = stream_of(v[9], dev);
    const int t = int_of(count, "slots");
    return without_gil([&] {
      return quant_read_fn(&store, layer, slots_p, t, into ? &pool : nullptr, into_layer, into_p, rows_p, ws, stream);
    });
  });
}

void entry_points(PyObject* const* v, void** p, int count) {
  for (int i = 0; i < count; ++i) {
    p[i] = PyLong_AsVoidPtr(v[i]);
    if (!p[i]) {
      if (PyErr_Occurred()) throw PythonError{};
      refuse("an entry point is missing");
    }
  }
}

// The library's entry points: mla_extend_tables, mla_rope_write, mla_prefill.
PyObject* bind(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return call(n, 3, [&] {
    void* p[3];
    entry_points(v, p, 3);
    extend_tables_fn = reinterpret_cast<decltype(extend_tables_fn)>(p[0]);
    rope_write_fn = reinterpret_cast<decltype(rope_write_fn)>(p[1]);
    prefill_fn = reinterpret_cast<decltype(prefill_fn)>(p[2]);
    return 0;
  });
}

// Those of the shared prefixes and the store: mla_decode_plan_shared, mla_decode_shared,
// mla_decode_workspace_size_shared, mla_quant_write, mla_quant_read.
PyObject* bind_shared(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return call(n, 5, [&] {
    void* p[5];
    entry_points(v, p, 5);
    plan_shared_fn = reinterpret_cast<decltype(plan_shared_fn)>(p[0]);
    decode_shared_fn = reinterpret_cast<decltype(decode_shared_fn)>(p[1]);
    shared_size_fn = reinterpret_cast<decltype(shared_size_fn)>(p[2]);
    quant_write_fn = reinterpret_cast<decltype(quant_write_fn)>(p[3]);
    quant_read_fn = reinterpret_cast<decltype(quant_read_fn)>(p[4]);
    return 0;
  });
}

}  // namespace

PyMODINIT_FUNC PyInit__step_binding() {
  static PyMethodDef methods[] = {
      {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
      {"extend_tables", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(extend_tables)), METH_FASTCALL, nullptr},
      {"rope_write", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope_write)), METH_FASTCALL, nullptr},
      {"prefill", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(prefill)), METH_FASTCALL, nullptr},
      {"bind_shared", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind_shared)), METH_FASTCALL, nullptr},
      {"plan_shared", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(plan_shared)), METH_FASTCALL, nullptr},
      {"decode_shared", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode_shared)), METH_FASTCALL, nullptr},
      {"quant_write", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quant_write)), METH_FASTCALL, nullptr},
      {"quant_read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quant_read)), METH_FASTCALL, nullptr},
      {nullptr, nullptr, 0, nullptr}};
  static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_step_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};
  return PyModule_Create(&module);
}
