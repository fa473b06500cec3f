// calls.cpp -- the decode-step calls' way from torch tensors to the C ABI.
//
// A decode step makes these calls once for each layer, and on small batches the kernels take less
// time than Python needs to read a dozen tensors' properties and to convert the arguments (25 us a
// call on the host, measured; 5 to 8 us here). So this module does what the rest of the binding does in
// Python: it checks shapes, types and strides, turns tensors into pointers, allocates outputs and
// keeps the attention's workspaces. No step of the work runs here.
//
// Functions take their arguments by position (the Python functions give them names and defaults),
// raise ValueError for what the tensors' properties forbid, and return the outputs, or the status
// of a C call that failed as an int.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <string>
#include <vector>

#include "../../include/nvfp4kv.h"

namespace {

struct Refused {
  std::string what;
};
[[noreturn]] void refuse(const std::string& what) { throw Refused{what}; }

struct Args {
  PyObject* const* v;
  const at::Tensor& tensor(int i, const char* what) const {
    if (!THPVariable_Check(v[i])) refuse(std::string(what) + " must be a tensor");
    return THPVariable_Unpack(v[i]);
  }
  bool none(int i) const { return v[i] == Py_None; }
  int64_t integer(int i) const {
    const long long x = PyLong_AsLongLong(v[i]);
    if (x == -1 && PyErr_Occurred()) throw PyErr_Occurred();
    return x;
  }
  int32_t int32(int i, const char* what) const {
    const int64_t x = integer(i);
    if (x < INT32_MIN || x > INT32_MAX) refuse(std::string(what) + " is out of range");
    return static_cast<int32_t>(x);
  }
  double real(int i) const {
    const double x = PyFloat_AsDouble(v[i]);
    if (x == -1.0 && PyErr_Occurred()) throw PyErr_Occurred();
    return x;
  }
};

int32_t fits32(int64_t n, const char* what) {
  if (n > INT32_MAX) refuse(std::string(what) + " is out of range");
  return static_cast<int32_t>(n);
}

std::string name(const at::Device& d) { return d.str(); }

const at::Tensor& first(const at::Tensor& t) {
  if (!t.is_cuda()) refuse("nvfp4 ops take CUDA tensors only");
  return t;
}

int32_t dtype_code(const at::Tensor& t) {
  if (t.scalar_type() == at::kHalf) return NVFP4_F16;
  if (t.scalar_type() == at::kBFloat16) return NVFP4_BF16;
  refuse(std::string("expected float16 or bfloat16, got ") + c10::toString(t.scalar_type()));
}

// A contiguous tensor of a type on the call's device.
void* address(const at::Tensor& t, at::ScalarType type, const at::Device& device, const char* what) {
  if (t.scalar_type() != type || t.device() != device || !t.is_contiguous())
    refuse(std::string(what) + " must be a contiguous " + c10::toString(type) + " tensor on " + name(device));
  return t.data_ptr();
}
template <typename T>
T* address(const Args& a, int i, at::ScalarType type, const at::Device& device, const char* what, bool optional = false) {
  if (optional && a.none(i)) return nullptr;
  return static_cast<T*>(address(a.tensor(i, what), type, device, what));
}

// Rows [n, heads, head_dim] whose heads and elements are contiguous.
struct Rows {
  int64_t n, heads, stride;
  void* data;
};
Rows rows_of(const at::Tensor& t, at::ScalarType type, const at::Device& device, const char* what, int64_t heads,
             int64_t head_dim) {
  if (t.dim() != 3 || t.scalar_type() != type || t.device() != device)
    refuse(std::string(what) + " must be a [n, heads, head_dim] " + c10::toString(type) + " tensor on " + name(device));
  const auto size = t.sizes(), stride = t.strides();
  if (size[2] != head_dim || (heads >= 0 && size[1] != heads))
    refuse(std::string(what) + " must have " + (heads >= 0 ? std::to_string(heads) : "its") + " heads of " +
           std::to_string(head_dim) + " elements");
  if (stride[2] != 1 || (stride[1] != size[2] && size[1] > 1))
    refuse(std::string(what) + " must have contiguous heads and elements");
  return {size[0], size[1], size[0] > 1 ? stride[0] : size[1] * size[2], t.data_ptr()};
}

// One cache's codes and scales.
struct Cache {
  nvfp4_paged_cache c;
  int64_t a, b, last;  // the codes' inner sizes
};
Cache cache_of(const at::Tensor& data, const at::Tensor& sf, const at::Device& device) {
  if (data.scalar_type() != at::kByte || (sf.scalar_type() != at::kByte && sf.scalar_type() != at::kFloat8_e4m3fn))
    refuse("paged caches are uint8 codes and uint8 / float8_e4m3fn scales");
  if (data.dim() != 4 || sf.dim() != 4) refuse("a paged cache tensor is 4-D [pages, ., ., head_dim // 2|16]");
  const auto d = data.sizes(), s = sf.sizes(), ds = data.strides(), ss = sf.strides();
  if (data.device() != device || sf.device() != device || s[0] != d[0] || s[1] != d[1] || s[2] != d[2] ||
      s[3] * 8 != d[3])
    refuse("codes [pages, ., ., D/2] and scales [pages, ., ., D/16] must match, on " + name(device));
  if (ds[3] != 1 || ds[2] != d[3] || ds[1] != d[2] * d[3] || ss[3] != 1 || ss[2] != s[3] || ss[1] != s[2] * s[3])
    refuse("paged cache pages must be contiguous inside (page stride may be larger)");
  return {{static_cast<uint8_t*>(data.data_ptr()), static_cast<uint8_t*>(sf.data_ptr()), ds[0], ss[0], d[0]}, d[1], d[2], d[3]};
}
struct Geometry {
  int32_t page_size, heads, head_dim;
};
Geometry geometry_of(const Cache& c, int32_t layout) {
  const bool nhd = layout == NVFP4_NHD;
  return {fits32(nhd ? c.a : c.b, "page_size"), fits32(nhd ? c.b : c.a, "num_kv_heads"), fits32(2 * c.last, "head_dim")};
}

struct Tables {
  void* data;
  int32_t type, width;
};
Tables tables_of(const at::Tensor& t, int64_t batch, const at::Device& device) {
  const auto type = t.scalar_type();
  if (t.dim() != 2 || t.size(0) != batch || (type != at::kInt && type != at::kLong) || t.device() != device ||
      !t.is_contiguous())
    refuse("block_tables must be a contiguous [" + std::to_string(batch) + ", max_pages] int32/int64 tensor on " + name(device));
  return {t.data_ptr(), type == at::kLong ? NVFP4_I64 : NVFP4_I32, fits32(t.size(1), "max_pages")};
}

float* device_scale(const Args& a, int i, const at::Device& device) {
  if (THPVariable_Check(a.v[i])) {
    const at::Tensor& t = THPVariable_Unpack(a.v[i]);
    if (t.scalar_type() == at::kFloat && t.device() == device && t.numel() >= 1) return static_cast<float*>(t.data_ptr());
  }
  refuse("k_scale/v_scale must be float32 CUDA tensors");
}

// The attention's workspaces (its counters have to stay as the last call left them), one per (device, stream):
// calls on one stream run one at a time, so they can share one; a larger one takes its place when a call needs
// it. A stream goes by its id, which is never given again, not by its handle; cudaStreamPerThread is another
// stream in each thread. At most kMostKept and kMostKeptBytes are kept (64 of the decode calls', which take up to 10 MB, or
// 16 of the prompts', which take up to 41): those that were not used for longest go back to torch's
// allocator, which hands their memory to the same stream only, and so after the calls that use it. A call that is
// being captured gets its own from the graph's memory, so that a graph never depends on what later calls do with
// these. The GIL guards the list, which is never destroyed (the process's end is no time to free device memory).
constexpr size_t kMostKept = 64;
constexpr int64_t kMostKeptBytes = int64_t(656) << 20;
struct Kept {
  int device;
  unsigned long long stream;
  uint64_t thread;
  at::Tensor memory;
};
std::vector<Kept>& kept() {  // the last one used first
  static auto* list = new std::vector<Kept>();
  return *list;
}
uint64_t this_thread() {
  static std::atomic<uint64_t> threads{0};
  thread_local const uint64_t number = ++threads;
  return number;
}

at::Tensor attention_workspace(const at::Device& device, cudaStream_t stream, int64_t bytes) {
  const bool capturing = c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None;
  Kept k{device.index(), 0, stream == cudaStreamPerThread ? this_thread() : 0, {}};
  if (!capturing && cudaStreamGetId(stream, &k.stream) != cudaSuccess) refuse("the current stream has no id");
  auto find = [&] {
    auto& list = kept();
    return std::find_if(list.begin(), list.end(), [&](const Kept& x) {
      return x.stream == k.stream && x.device == k.device && x.thread == k.thread;
    });
  };
  if (!capturing) {
    const auto at = find();
    if (at != kept().end()) {
      std::rotate(kept().begin(), at, at + 1);
      if (kept().front().memory.numel() >= bytes) return kept().front().memory;
    }
  }
  k.memory = at::empty({bytes}, at::TensorOptions().dtype(at::kByte).device(device));
  if (cudaMemsetAsync(k.memory.data_ptr(), 0, NVFP4_COUNTER_BYTES, stream) != cudaSuccess)
    refuse("the workspace's counters could not be cleared");
  if (!capturing) {
    const auto at = find();
    if (at != kept().end()) kept().erase(at);
    kept().insert(kept().begin(), k);
    int64_t held = 0;
    for (const Kept& x : kept()) held += x.memory.numel();
    for (; kept().size() > 1 && (kept().size() > kMostKept || held > kMostKeptBytes); kept().pop_back())
      held -= kept().back().memory.numel();
  }
  return k.memory;
}

cudaStream_t stream_of(const at::Device& device) { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }

PyObject* pair(const at::Tensor& x, const at::Tensor& y) {
  PyObject* a = THPVariable_Wrap(x);
  PyObject* b = THPVariable_Wrap(y);
  PyObject* r = a && b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return r;
}

// No exception leaves a call: torch's own become what torch raises for them (OutOfMemoryError among them).
template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F body) {
  HANDLE_TH_ERRORS
  try {
    if (given != wanted) refuse("wrong number of arguments");
    return body();
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (PyObject*) {  // set already
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

// query, key, value, q_weight, k_weight, cos_sin, batch_indices, positions, k codes, v codes, k scales, v scales,
// kv_indices, kv_indptr, kv_last_page_len, k_scale, v_scale, layout, eps, interleaved, recipe (None or (e4m3_max,
// err_mode, fast)), out, dev_status, rotary_positions, rotary_axes
PyObject* qk_norm_rope_append(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded(n, 25, [&]() -> PyObject* {
    const Args a{argv};
    const at::Tensor& q = first(a.tensor(0, "query"));
    const at::Device device = q.device();
    const c10::cuda::CUDAGuard on(device);
    const auto type = q.scalar_type();
    const int32_t code = dtype_code(q);
    const Cache k = cache_of(a.tensor(8, "k_cache"), a.tensor(10, "k scales"), device);
    const Cache v = cache_of(a.tensor(9, "v_cache"), a.tensor(11, "v scales"), device);
    if (k.a != v.a || k.b != v.b || k.last != v.last) refuse("the K and V caches must have the same page shape");
    const int32_t layout = a.int32(17, "kv_layout");
    const Geometry g = geometry_of(k, layout);
    const Rows qr = rows_of(q, type, device, "query", -1, g.head_dim);
    const Rows kr = rows_of(a.tensor(1, "key"), type, device, "key", g.heads, g.head_dim);
    const Rows vr = rows_of(a.tensor(2, "value"), type, device, "value", g.heads, g.head_dim);
    const at::Tensor &bi = a.tensor(6, "batch_indices"), &pos = a.tensor(7, "positions");
    if (kr.n != qr.n || vr.n != qr.n || bi.numel() != qr.n || pos.numel() != qr.n)
      refuse("query, key, value, batch_indices and positions must have as many rows");
    const void* w[2];
    for (int i = 0; i < 2; ++i) {
      w[i] = address<void>(a, 3 + i, type, device, i ? "k_weight" : "q_weight", true);
      if (w[i] && a.tensor(3 + i, "").numel() != g.head_dim) refuse("a norm's weights must have head_dim elements");
    }
    const float* table = address<float>(a, 5, at::kFloat, device, "cos_sin", true);
    int64_t table_rows = 0;
    int32_t rotary = 0;
    if (!a.none(5)) {
      const at::Tensor& t = a.tensor(5, "cos_sin");
      if (t.dim() != 2) refuse("cos_sin must be [positions, rotary_dim]");
      table_rows = t.size(0);
      rotary = fits32(t.size(1), "rotary_dim");
    }
    const at::Tensor &indices = a.tensor(12, "kv_indices"), &indptr = a.tensor(13, "kv_indptr");
    const int64_t batch = indptr.numel() - 1;
    if (!a.none(14) && a.tensor(14, "").numel() < batch) refuse("kv_last_page_len must have one entry per request");
    float ks = 1.0f, vs = 1.0f;
    const float *kd = nullptr, *vd = nullptr;
    if (THPVariable_Check(argv[15]) || THPVariable_Check(argv[16])) {
      kd = device_scale(a, 15, device);
      vd = device_scale(a, 16, device);
    } else {
      ks = static_cast<float>(a.real(15));
      vs = static_cast<float>(a.real(16));
    }
    nvfp4_4over6_config recipe{};
    const bool has_recipe = !a.none(20);
    if (has_recipe) {
      int mode = 0, fast = 0;
      if (!PyArg_ParseTuple(argv[20], "fii", &recipe.e4m3_max, &mode, &fast)) return nullptr;
      recipe.err_mode = mode;
      recipe.err_use_fast_math = fast;
    }
    at::Tensor out;
    Rows o;
    if (a.none(21)) {
      out = at::empty({qr.n, qr.heads, g.head_dim}, q.options());
      o = {qr.n, qr.heads, qr.heads * g.head_dim, out.data_ptr()};
    } else {
      out = a.tensor(21, "out");
      o = rows_of(out, type, device, "out", qr.heads, g.head_dim);
      if (o.n != qr.n) refuse("out must have query's shape");
    }
    const int32_t Hq = fits32(qr.heads, "num_qo_heads"), requests = fits32(batch, "batch_size");
    const float eps = static_cast<float>(a.real(18));
    const int32_t interleaved = PyObject_IsTrue(argv[19]) == 1;
    const int32_t* bi_ptr = static_cast<int32_t*>(address(bi, at::kInt, device, "batch_indices"));
    const int32_t* pos_ptr = static_cast<int32_t*>(address(pos, at::kInt, device, "positions"));
    const int32_t* idx_ptr = static_cast<int32_t*>(address(indices, at::kInt, device, "kv_indices"));
    const int32_t* ptr_ptr = static_cast<int32_t*>(address(indptr, at::kInt, device, "kv_indptr"));
    const int32_t* last_ptr = address<int32_t>(a, 14, at::kInt, device, "kv_last_page_len", true);
    int32_t* status = address<int32_t>(a, 22, at::kInt, device, "dev_status", true);
    const nvfp4_4over6_config* r = has_recipe ? &recipe : nullptr;
    nvfp4_status st;
    if (a.none(23) && a.none(24)) {
      st = nvfp4_qk_norm_rope_append_paged(qr.data, kr.data, vr.data, code, qr.n, Hq, g.heads, g.head_dim, qr.stride, kr.stride,
                                           vr.stride, w[0], w[1], eps, table, table_rows, rotary, interleaved, bi_ptr, pos_ptr,
                                           k.c, v.c, g.page_size, layout, idx_ptr, indices.numel(), ptr_ptr, last_ptr, requests,
                                           ks, vs, kd, vd, r, o.data, o.stride, status, stream_of(device));
    } else {
      if (a.none(23) || a.none(24)) refuse("rotary_positions and rotary_axes go together");
      const at::Tensor &ap = a.tensor(23, "rotary_positions"), &ax = a.tensor(24, "rotary_axes");
      if (ap.dim() != 2 || ap.size(1) != qr.n) refuse("rotary_positions must be [axes, n] with a column for each row");
      if (ax.numel() != rotary / 2) refuse("rotary_axes must have an entry for each of cos_sin's rotary_dim / 2 pairs");
      st = nvfp4_qk_norm_rope_axes_append_paged(
          qr.data, kr.data, vr.data, code, qr.n, Hq, g.heads, g.head_dim, qr.stride, kr.stride, vr.stride, w[0], w[1], eps,
          table, table_rows, rotary, interleaved, static_cast<int32_t*>(address(ap, at::kInt, device, "rotary_positions")),
          fits32(ap.size(0), "axes"), static_cast<uint8_t*>(address(ax, at::kByte, device, "rotary_axes")), bi_ptr, pos_ptr,
          k.c, v.c, g.page_size, layout, idx_ptr, indices.numel(), ptr_ptr, last_ptr, requests, ks, vs, kd, vd, r, o.data,
          o.stride, status, stream_of(device));
    }
    if (st != NVFP4_OK) return PyLong_FromLong(st);
    return THPVariable_Wrap(out);
  });
}

// k codes, k scales, block_tables, seq_lens, key_bounds, first_positions, layout, dev_status
PyObject* page_key_bounds(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const Args a{argv};
    const at::Tensor& data = first(a.tensor(0, "k_cache"));
    const at::Device device = data.device();
    const c10::cuda::CUDAGuard on(device);
    const Cache k = cache_of(data, a.tensor(1, "k scales"), device);
    const int32_t layout = a.int32(6, "kv_layout");
    const Geometry g = geometry_of(k, layout);
    const at::Tensor &lens = a.tensor(3, "seq_lens"), &bounds = a.tensor(4, "key_bounds");
    const int64_t batch = lens.numel();
    if (bounds.dim() != 4 || bounds.size(0) != k.c.num_pages || bounds.size(1) != g.heads || bounds.size(2) != 2 ||
        bounds.size(3) != g.head_dim)
      refuse("key_bounds must be [num_pages, num_kv_heads, 2, head_dim]");
    if (!a.none(5) && a.tensor(5, "first_positions").numel() != batch) refuse("first_positions must have one entry per request");
    const Tables t = tables_of(a.tensor(2, "block_tables"), batch, device);
    const nvfp4_status st = nvfp4_page_key_bounds(
        k.c, g.page_size, g.heads, g.head_dim, layout, t.data, t.type, t.width,
        static_cast<int32_t*>(address(lens, at::kInt, device, "seq_lens")),
        address<int32_t>(a, 5, at::kInt, device, "first_positions", true), fits32(batch, "batch_size"),
        address(bounds, at::kHalf, device, "key_bounds"), address<int32_t>(a, 7, at::kInt, device, "dev_status", true),
        stream_of(device));
    if (st != NVFP4_OK) return PyLong_FromLong(st);
    Py_RETURN_NONE;
  });
}

// query, key_bounds, block_tables, seq_lens, page_size, max_selected, sink, recent, selected, count, dev_status
PyObject* select_pages(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const Args a{argv};
    const at::Tensor& q = first(a.tensor(0, "query"));
    const at::Device device = q.device();
    const c10::cuda::CUDAGuard on(device);
    const at::Tensor& bounds = a.tensor(1, "key_bounds");
    if (bounds.dim() != 4 || bounds.size(2) != 2) refuse("key_bounds must be [num_pages, num_kv_heads, 2, head_dim]");
    const int64_t heads = bounds.size(1), head_dim = bounds.size(3);
    const Rows r = rows_of(q, q.scalar_type(), device, "query", -1, head_dim);
    const at::Tensor& lens = a.tensor(3, "seq_lens");
    if (lens.numel() != r.n) refuse("seq_lens must have one entry per request");
    const Tables t = tables_of(a.tensor(2, "block_tables"), r.n, device);
    const int32_t k = a.int32(5, "max_selected");
    at::Tensor selected, count;
    if (a.none(8)) {
      const auto options = at::TensorOptions().dtype(at::kInt).device(device);
      selected = at::empty({r.n, heads, k < 0 ? 0 : k}, options);
      count = at::empty({r.n, heads}, options);
    } else {
      selected = a.tensor(8, "selected_pages");
      count = a.tensor(9, "num_selected");
      if (selected.dim() != 3 || selected.size(0) != r.n || selected.size(1) != heads || selected.size(2) != k ||
          count.dim() != 2 || count.size(0) != r.n || count.size(1) != heads)
        refuse("out must be ([B, H, max_selected], [B, H]) int32 tensors");
    }
    int64_t bytes = 0;
    nvfp4_status st = nvfp4_select_pages_workspace_bytes(fits32(r.n, "batch_size"), fits32(heads, "num_kv_heads"), t.width, &bytes);
    if (st != NVFP4_OK) return PyLong_FromLong(st);
    const cudaStream_t stream = stream_of(device);
    // the scores, for this call: nothing later reads them, and they grow with the table's width
    const at::Tensor ws = at::empty({bytes}, at::TensorOptions().dtype(at::kByte).device(device));
    st = nvfp4_select_pages(
        r.data, dtype_code(q), r.stride, fits32(r.heads, "num_qo_heads"), static_cast<int32_t>(heads),
        fits32(head_dim, "head_dim"), address(bounds, at::kHalf, device, "key_bounds"), bounds.size(0),
        a.int32(4, "page_size"), t.data, t.type, t.width, static_cast<int32_t*>(address(lens, at::kInt, device, "seq_lens")),
        static_cast<int32_t>(r.n), k, a.int32(6, "num_sink_pages"), a.int32(7, "num_recent_pages"),
        static_cast<int32_t*>(address(selected, at::kInt, device, "selected_pages")),
        static_cast<int32_t*>(address(count, at::kInt, device, "num_selected")),
        address<int32_t>(a, 10, at::kInt, device, "dev_status", true), ws.data_ptr(), ws.numel(), stream);
    if (st != NVFP4_OK) return PyLong_FromLong(st);
    return pair(selected, count);
  });
}

// query, k codes, v codes, k scales, v scales, block_tables, seq_lens, selected, count (None: all pages), k_scale,
// v_scale, layout, sm_scale (None: head_dim ** -0.5), soft cap, window_left, out, lse, dev_status, num_sink_tokens
PyObject* attention(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded(n, 19, [&]() -> PyObject* {
    const Args a{argv};
    const at::Tensor& q = first(a.tensor(0, "query"));
    const at::Device device = q.device();
    const c10::cuda::CUDAGuard on(device);
    const auto type = q.scalar_type();
    const int32_t code = dtype_code(q);
    const Cache k = cache_of(a.tensor(1, "k_cache"), a.tensor(3, "k scales"), device);
    const Cache v = cache_of(a.tensor(2, "v_cache"), a.tensor(4, "v scales"), device);
    if (k.a != v.a || k.b != v.b || k.last != v.last) refuse("the K and V caches must have the same page shape");
    const int32_t layout = a.int32(11, "kv_layout");
    const Geometry g = geometry_of(k, layout);
    const Rows r = rows_of(q, type, device, "query", -1, g.head_dim);
    const at::Tensor& lens = a.tensor(6, "seq_lens");
    if (lens.numel() != r.n) refuse("seq_lens must have one entry per request");
    const Tables t = tables_of(a.tensor(5, "block_tables"), r.n, device);
    const float *gk = device_scale(a, 9, device), *gv = device_scale(a, 10, device);
    at::Tensor out, lse;
    if (a.none(15)) {
      out = at::empty({r.n, r.heads, g.head_dim}, q.options());
    } else {
      out = a.tensor(15, "out");
      if (out.dim() != 3 || out.size(0) != r.n || out.size(1) != r.heads || out.size(2) != g.head_dim)
        refuse("out must be [batch, num_qo_heads, head_dim]");
    }
    if (a.none(16)) {
      lse = at::empty({r.n, r.heads}, q.options().dtype(at::kFloat));
    } else {
      lse = a.tensor(16, "lse");
      if (lse.dim() != 2 || lse.size(0) != r.n || lse.size(1) != r.heads) refuse("lse must be [batch, num_qo_heads]");
    }
    const int32_t Hq = fits32(r.heads, "num_qo_heads"), batch = fits32(r.n, "batch_size");
    int64_t bytes = 0;
    nvfp4_status st = nvfp4_paged_attention_workspace_bytes(Hq, g.heads, g.head_dim, &bytes);
    if (st != NVFP4_OK) return PyLong_FromLong(st);
    const cudaStream_t stream = stream_of(device);
    const at::Tensor ws = attention_workspace(device, stream, bytes);
    const float sm = a.none(12) ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(g.head_dim))) : static_cast<float>(a.real(12));
    const float cap = static_cast<float>(a.real(13));
    const int32_t* len_ptr = static_cast<int32_t*>(address(lens, at::kInt, device, "seq_lens"));
    void* out_ptr = address(out, type, device, "out");
    float* lse_ptr = static_cast<float*>(address(lse, at::kFloat, device, "lse"));
    int32_t* status = address<int32_t>(a, 17, at::kInt, device, "dev_status", true);
    if (a.none(7)) {
      const int32_t window = a.int32(14, "window_left"), sinks = a.int32(18, "num_sink_tokens");
      if (sinks == 0)
        st = nvfp4_paged_attention_decode(r.data, code, r.stride, Hq, k.c, v.c, g.page_size, g.heads, g.head_dim, layout,
                                          t.data, t.type, t.width, len_ptr, batch, gk, gv, sm, cap, window, out_ptr, lse_ptr,
                                          status, ws.data_ptr(), ws.numel(), stream);
      else
        st = nvfp4_paged_attention_decode_sinks(r.data, code, r.stride, Hq, k.c, v.c, g.page_size, g.heads, g.head_dim,
                                                layout, t.data, t.type, t.width, len_ptr, batch, gk, gv, sm, cap, window,
                                                sinks, out_ptr, lse_ptr, status, ws.data_ptr(), ws.numel(), stream);
    } else {
      const at::Tensor &sel = a.tensor(7, "selected_pages"), &num = a.tensor(8, "num_selected");
      if (sel.dim() != 3 || sel.size(0) != r.n || sel.size(1) != g.heads || num.dim() != 2 || num.size(0) != r.n ||
          num.size(1) != g.heads)
        refuse("selected_pages must be [B, H, max_selected] and num_selected [B, H]");
      st = nvfp4_sparse_paged_attention_decode(
          r.data, code, r.stride, Hq, k.c, v.c, g.page_size, g.heads, g.head_dim, layout, t.data, t.type, t.width,
          len_ptr, batch, static_cast<int32_t*>(address(sel, at::kInt, device, "selected_pages")),
          static_cast<int32_t*>(address(num, at::kInt, device, "num_selected")), fits32(sel.size(2), "max_selected"), gk,
          gv, sm, cap, out_ptr, lse_ptr, status, ws.data_ptr(), ws.numel(), stream);
    }
    if (st != NVFP4_OK) return PyLong_FromLong(st);
    return pair(out, lse);
  });
}

// query, k codes, v codes, k scales, v scales, qo_indptr, block_tables, seq_lens, k_scale, v_scale, layout, causal,
// sm_scale (None: head_dim ** -0.5), soft cap, window_left, num_sink_tokens, out, lse, dev_status
PyObject* prefill(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded(n, 19, [&]() -> PyObject* {
    const Args a{argv};
    const at::Tensor& q = first(a.tensor(0, "query"));
    const at::Device device = q.device();
    const c10::cuda::CUDAGuard on(device);
    const auto type = q.scalar_type();
    const int32_t code = dtype_code(q);
    const Cache k = cache_of(a.tensor(1, "k_cache"), a.tensor(3, "k scales"), device);
    const Cache v = cache_of(a.tensor(2, "v_cache"), a.tensor(4, "v scales"), device);
    if (k.a != v.a || k.b != v.b || k.last != v.last) refuse("the K and V caches must have the same page shape");
    const int32_t layout = a.int32(10, "kv_layout");
    const Geometry g = geometry_of(k, layout);
    const Rows r = rows_of(q, type, device, "query", -1, g.head_dim);
    const at::Tensor &indptr = a.tensor(5, "qo_indptr"), &lens = a.tensor(7, "seq_lens");
    const int64_t batch = lens.numel();
    if (indptr.numel() != batch + 1) refuse("qo_indptr must have one entry more than seq_lens");
    const Tables t = tables_of(a.tensor(6, "block_tables"), batch, device);
    const float *gk = device_scale(a, 8, device), *gv = device_scale(a, 9, device);
    at::Tensor out, lse;
    if (a.none(16)) {
      out = at::empty({r.n, r.heads, g.head_dim}, q.options());
    } else {
      out = a.tensor(16, "out");
      if (out.dim() != 3 || out.size(0) != r.n || out.size(1) != r.heads || out.size(2) != g.head_dim)
        refuse("out must be [nnz, num_qo_heads, head_dim]");
    }
    if (a.none(17)) {
      lse = at::empty({r.n, r.heads}, q.options().dtype(at::kFloat));
    } else {
      lse = a.tensor(17, "lse");
      if (lse.dim() != 2 || lse.size(0) != r.n || lse.size(1) != r.heads) refuse("lse must be [nnz, num_qo_heads]");
    }
    int64_t bytes = 0;
    nvfp4_status st = nvfp4_paged_attention_prefill_workspace_bytes(g.head_dim, &bytes);
    if (st != NVFP4_OK) return PyLong_FromLong(st);
    const cudaStream_t stream = stream_of(device);
    const at::Tensor ws = attention_workspace(device, stream, bytes);
    const float sm = a.none(12) ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(g.head_dim))) : static_cast<float>(a.real(12));
    st = nvfp4_paged_attention_prefill(
        r.data, code, r.n, r.stride, fits32(r.heads, "num_qo_heads"),
        static_cast<int32_t*>(address(indptr, at::kInt, device, "qo_indptr")), k.c, v.c, g.page_size, g.heads, g.head_dim, layout,
        t.data, t.type, t.width, static_cast<int32_t*>(address(lens, at::kInt, device, "seq_lens")), fits32(batch, "batch_size"),
        gk, gv, PyObject_IsTrue(argv[11]) == 1, sm, static_cast<float>(a.real(13)), a.int32(14, "window_left"),
        a.int32(15, "num_sink_tokens"), address(out, type, device, "out"),
        static_cast<float*>(address(lse, at::kFloat, device, "lse")), address<int32_t>(a, 18, at::kInt, device, "dev_status", true),
        ws.data_ptr(), ws.numel(), stream);
    if (st != NVFP4_OK) return PyLong_FromLong(st);
    return pair(out, lse);
  });
}

// The attention's workspaces that are kept, the last one used first: (device, stream's id, thread of a
// per-thread stream, bytes).
PyObject* workspaces(PyObject*, PyObject* const*, Py_ssize_t n) {
  return guarded(n, 0, []() -> PyObject* {
    PyObject* list = PyList_New(0);
    for (const Kept& k : kept()) {
      PyObject* item = list ? Py_BuildValue("iKKL", k.device, k.stream, static_cast<unsigned long long>(k.thread),
                                            static_cast<long long>(k.memory.numel()))
                            : nullptr;
      if (!item || PyList_Append(list, item) < 0) Py_CLEAR(list);
      Py_XDECREF(item);
      if (!list) break;
    }
    return list;
  });
}

PyMethodDef kMethods[] = {
    {"qk_norm_rope_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(qk_norm_rope_append)), METH_FASTCALL, nullptr},
    {"page_key_bounds", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(page_key_bounds)), METH_FASTCALL, nullptr},
    {"select_pages", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(select_pages)), METH_FASTCALL, nullptr},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(attention)), METH_FASTCALL, nullptr},
    {"prefill", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(prefill)), METH_FASTCALL, nullptr},
    {"workspaces", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(workspaces)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "nvfp4kv_calls", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_nvfp4kv_calls() { return PyModule_Create(&kModule); }
