// fa_torch.cpp -- the tensor-level calls of the package (module _fa_torch): checks of torch
// tensors, allocation of outputs and workspaces, and the C-ABI call of include/fa_decoder.h.
//
// A single token's operators take a few microseconds on the GPU, and the same checks written in
// Python cost 25 to 60 us a call on the host (a Grace core); here they cost one or two. Nothing is
// computed here and no CUDA call is made besides those of the library and torch's allocator. The
// library's functions are handed in as addresses (bind), so that the module serves either build.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/as_strided.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>
#include <stdexcept>
#include <string>
#include <utility>

#include "fa_decoder.h"

namespace {

struct Library {
  decltype(&fa_qk_norm_rope) norm_rope = nullptr;
  decltype(&fa_qk_norm_rope_bwd) norm_rope_bwd = nullptr;
  decltype(&fa_qk_norm_rope_bwd_workspace_bytes) norm_rope_bwd_bytes = nullptr;
  decltype(&fa_paged_append) append = nullptr;
  decltype(&fa_fwd_paged) attend = nullptr;
  decltype(&fa_fwd_paged_workspace_bytes) attend_bytes = nullptr;
} lib;

// A refusal: TypeError or ValueError in Python.
struct Refusal {
  PyObject* type;
  std::string text;
};
[[noreturn]] void bad_type(const std::string& text) { throw Refusal{PyExc_TypeError, text}; }
[[noreturn]] void bad_value(const std::string& text) { throw Refusal{PyExc_ValueError, text}; }

std::string shape_text(at::IntArrayRef s) {
  std::string t = "[";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + "]";
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) bad_type(std::string(what) + " must be a tensor");
  return THPVariable_Unpack(o);
}
// an undefined tensor for None
at::Tensor optional_tensor(PyObject* o, const char* what) { return o == Py_None ? at::Tensor() : tensor(o, what); }

int as_int(int64_t n, const char* what) {
  if (n > 0x7fffffffLL) bad_value(std::string(what) + " is too large");
  return (int)n;
}
int as_int(PyObject* o, const char* what) {
  const long long n = PyLong_AsLongLong(o);
  if (n == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    bad_type(std::string(what) + " must be an integer");
  }
  if (n > 0x7fffffffLL || n < -0x7fffffffLL) bad_value(std::string(what) + " is too large");
  return (int)n;
}
float as_float(PyObject* o, const char* what) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    bad_type(std::string(what) + " must be a number");
  }
  return (float)x;
}

bool as_bool(PyObject* o, const char* what) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) {
    PyErr_Clear();
    bad_type(std::string(what) + " must be a truth value");
  }
  return x;
}

fa_dtype type_code(const at::Tensor& t, const char* what) {
  if (t.scalar_type() == at::kBFloat16) return FA_BF16;
  if (t.scalar_type() == at::kHalf) return FA_F16;
  bad_type(std::string(what) + " must be float16 or bfloat16");
}

// fa_heads of a [..., tokens, heads, d] tensor (3 or 4 dimensions). The stride of an axis of one
// element is never used, and torch may report any.
fa_heads heads_of(const at::Tensor& t, const char* what, const at::Tensor& like, at::IntArrayRef shape = {},
                  bool written = false) {
  if (t.scalar_type() != like.scalar_type()) bad_type(std::string(what) + " must have the other tensors' dtype");
  const auto size = t.sizes();
  const auto stride = t.strides();
  if (!shape.empty() && size != shape)
    bad_value(std::string(what) + " must be " + shape_text(shape) + ", not " + shape_text(size));
  const int n = (int)t.dim();
  if (stride[n - 1] != 1 && size[n - 1] > 1)
    bad_value(std::string("the elements of a row of ") + what + " must be adjacent (stride 1)");
  long long s[3] = {0, 0, 0};
  for (int i = 0; i < n - 1; ++i) {
    if (size[i] <= 1) continue;
    s[i + 4 - n] = stride[i];
    if (written && stride[i] == 0) bad_value(std::string("the rows of ") + what + " must not overlap");
  }
  return fa_heads{t.data_ptr(), s[0], s[1], s[2], as_int(size[n - 2], "the number of heads")};
}

// Every tensor (undefined: not given) is a CUDA tensor on the first one's device.
struct OneDevice {
  const at::Tensor& first;
  explicit OneDevice(const at::Tensor& t) : first(t) { also(t); }
  OneDevice& also(const at::Tensor& t) {
    if (t.defined() && (!t.is_cuda() || t.device() != first.device()))
      bad_value("the tensors must be CUDA tensors on one device");
    return *this;
  }
};

const int* index_of(const at::Tensor& t, const char* what, at::IntArrayRef shape) {
  if (t.scalar_type() != at::kInt) bad_type(std::string(what) + " must be int32");
  if (t.sizes() != shape || !t.is_contiguous())
    bad_value(std::string(what) + " must be contiguous " + shape_text(shape) + ", not " + shape_text(t.sizes()));
  return static_cast<const int*>(t.data_ptr());
}

// fa_rope of a [length, rot_dim] fp32 table (undefined: no rotation)
fa_rope rope_of(const at::Tensor& t, bool interleaved, int64_t d) {
  if (!t.defined()) return fa_rope{nullptr, 0, 0, 0};
  if (t.scalar_type() != at::kFloat) bad_type("rope must be float32");
  if (t.dim() != 2 || !t.is_contiguous() || t.size(1) % 16 || t.size(1) > d)
    bad_value("rope must be a contiguous [length, rot_dim] table, rot_dim a multiple of 16 up to d");
  // torch has no address for a table without rows, and a null pointer would mean no rotation: this
  // one is never read, for no position lies below a length of 0
  alignas(16) static const float no_rows[4] = {};
  return fa_rope{t.numel() ? static_cast<const float*>(t.data_ptr()) : no_rows,
                 as_int(t.size(0), "the table's length"), (int)t.size(1), interleaved};
}

// fa_paged_kv of [num_pages, Hkv, page_size, d] tensors with the same strides
fa_paged_kv cache_of(const at::Tensor& k, const at::Tensor& v, const at::Tensor& like) {
  if (k.scalar_type() != like.scalar_type() || v.scalar_type() != like.scalar_type())
    bad_type("the cache must have the other tensors' dtype");
  if (k.dim() != 4 || k.sizes() != v.sizes())
    bad_value("k_pages and v_pages must both be [num_pages, Hkv, page_size, d]");
  long long s[4];
  for (int i = 0; i < 4; ++i) {
    s[i] = k.size(i) <= 1 ? 0 : k.stride(i);
    if (k.size(i) > 1 && k.stride(i) != v.stride(i)) bad_value("k_pages and v_pages must have the same strides");
  }
  if (k.size(3) > 1 && s[3] != 1) bad_value("the elements of a cached row must be adjacent (stride 1)");
  return fa_paged_kv{k.data_ptr(), v.data_ptr(), s[0], s[1], s[2], as_int(k.size(0), "the number of pages"),
                     as_int(k.size(2), "the page size"), as_int(k.size(1), "the number of heads"),
                     as_int(k.size(3), "the head dimension")};
}

// Nothing here is recorded by autograd: an input that requires a gradient would lose it unseen.
void not_recorded(std::initializer_list<std::pair<const at::Tensor*, const char*>> inputs) {
  if (!at::GradMode::is_enabled()) return;
  for (const auto& [t, what] : inputs)
    if (t->requires_grad())
      bad_value(std::string(what) + " requires grad and the call is not recorded by autograd: make it under "
                                    "torch.no_grad(), or pass the tensor detached");
}

// The device and stream of a call: what is allocated inside belongs to that stream.
struct Launch {
  c10::cuda::CUDAGuard device;
  std::optional<c10::cuda::CUDAStreamGuard> inner;
  void* stream;
  Launch(const at::Tensor& t, PyObject* s) : device(t.device()) {
    if (s == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
      return;
    }
    int64_t part[3];
    const char* names[3] = {"stream_id", "device_index", "device_type"};
    for (int i = 0; i < 3; ++i) {
      PyObject* o = PyObject_GetAttrString(s, names[i]);
      part[i] = o ? PyLong_AsLongLong(o) : -1;
      Py_XDECREF(o);
      if (PyErr_Occurred()) {
        PyErr_Clear();
        bad_type("stream must be a torch.cuda.Stream");
      }
    }
    const auto st = c10::cuda::CUDAStream::unpack3(part[0], (c10::DeviceIndex)part[1], (c10::DeviceType)part[2]);
    if (st.device_index() != t.get_device()) bad_value("stream must be on the tensors' device");
    inner.emplace(st);
    stream = st.stream();
  }
};

// (the allocator's own call: at::empty's dispatch costs another 0.2 us each)
at::Tensor fresh(const at::Tensor& t, at::IntArrayRef size, at::ScalarType type) {
  return at::detail::empty_cuda(size, t.options().dtype(type));
}
at::Tensor rows_like(const at::Tensor& t) { return fresh(t, t.sizes(), t.scalar_type()); }

// Device memory for the length of a call, from torch's allocator (so from the graph's own pool
// while one is captured): given back when the call returns, for later work on the same stream.
struct Scratch {
  void* ptr = nullptr;
  size_t size = 0;
  void take(size_t n, void* stream) {
    if (!n) return;
    ptr = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(n, static_cast<cudaStream_t>(stream));
    size = n;
  }
  Scratch() = default;
  Scratch(const Scratch&) = delete;
  Scratch& operator=(const Scratch&) = delete;
  ~Scratch() {
    if (ptr) c10::cuda::CUDACachingAllocator::raw_delete(ptr);
  }
};

PyObject* tuple_of(std::initializer_list<at::Tensor> ts) {
  PyObject* out = PyTuple_New((Py_ssize_t)ts.size());
  Py_ssize_t i = 0;
  for (const auto& t : ts) PyTuple_SET_ITEM(out, i++, THPVariable_Wrap(t));
  return out;
}

// Runs f, turning refusals and C++ exceptions into Python ones.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  try {
    if (n != want) bad_type("wrong number of arguments");
    return f();
  } catch (const Refusal& r) {
    PyErr_SetString(r.type, r.text.c_str());
  } catch (const c10::OutOfMemoryError& e) {  // the type that torch's own calls raise
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "an unknown C++ exception");
  }
  return nullptr;
}

void check_qk(const at::Tensor& q, const at::Tensor& k, const at::Tensor& wq, const at::Tensor& wk) {
  if (q.dim() != 4 || k.dim() != 4 || q.size(0) != k.size(0) || q.size(1) != k.size(1) || q.size(3) != k.size(3))
    bad_value("q and k must be [B, N, H, d] with the same B, N and d");
  if (wq.scalar_type() != q.scalar_type() || wk.scalar_type() != q.scalar_type())
    bad_type("wq and wk must have q's dtype");
  const int64_t d = q.size(3);
  if (wq.dim() != 1 || wk.dim() != 1 || wq.size(0) != d || wk.size(0) != d || !wq.is_contiguous() ||
      !wk.is_contiguous())
    bad_value("wq and wk must be contiguous [d]");
}

// (q, k, wq, wk, rope, positions, eps, interleaved, q_out, k_out, stream)
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &wq = tensor(a[2], "wq"), &wk = tensor(a[3], "wk");
    const at::Tensor table = optional_tensor(a[4], "rope"), pos = optional_tensor(a[5], "positions");
    at::Tensor qo = optional_tensor(a[8], "q_out"), ko = optional_tensor(a[9], "k_out");
    const fa_dtype dt = type_code(q, "q and k");
    check_qk(q, k, wq, wk);
    const int B = as_int(q.size(0), "B"), N = as_int(q.size(1), "N"), d = as_int(q.size(3), "d");
    const fa_heads hq = heads_of(q, "q", q), hk = heads_of(k, "k", q);
    const fa_rope rp = rope_of(table, as_bool(a[7], "interleaved"), d);
    const int* positions = pos.defined() ? index_of(pos, "positions", {B, N}) : nullptr;
    const float eps = as_float(a[6], "eps");
    fa_heads oq{}, ok{};
    if (qo.defined()) oq = heads_of(qo, "q_out", q, q.sizes(), true);
    if (ko.defined()) ok = heads_of(ko, "k_out", q, k.sizes(), true);
    OneDevice(q).also(k).also(wq).also(wk).also(table).also(pos).also(qo).also(ko);
    not_recorded({{&q, "q"}, {&k, "k"}, {&wq, "wq"}, {&wk, "wk"}});
    Launch on(q, a[10]);
    if (!qo.defined()) oq = heads_of(qo = rows_like(q), "q_out", q);
    if (!ko.defined()) ok = heads_of(ko = rows_like(k), "k_out", q);
    const int rc = lib.norm_rope(&hq, &hk, &oq, &ok, B, N, d, wq.data_ptr(), wk.data_ptr(), eps, &rp, positions, dt,
                                 on.stream);
    return rc == FA_OK ? tuple_of({qo, ko}) : PyLong_FromLong(rc);
  });
}

// (dq_out, dk_out, q, k, wq, wk, rope, positions, eps, interleaved, dq, dk, stream)
PyObject* norm_rope_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    const at::Tensor &gq = tensor(a[0], "dq_out"), &gk = tensor(a[1], "dk_out");
    const at::Tensor &q = tensor(a[2], "q"), &k = tensor(a[3], "k"), &wq = tensor(a[4], "wq"), &wk = tensor(a[5], "wk");
    const at::Tensor table = optional_tensor(a[6], "rope"), pos = optional_tensor(a[7], "positions");
    at::Tensor dq = optional_tensor(a[10], "dq"), dk = optional_tensor(a[11], "dk");
    const fa_dtype dt = type_code(q, "q and k");
    check_qk(q, k, wq, wk);
    const int B = as_int(q.size(0), "B"), N = as_int(q.size(1), "N"), d = as_int(q.size(3), "d");
    const fa_heads hq = heads_of(q, "q", q), hk = heads_of(k, "k", q);
    const fa_heads hgq = heads_of(gq, "dq_out", q, q.sizes()), hgk = heads_of(gk, "dk_out", q, k.sizes());
    const fa_rope rp = rope_of(table, as_bool(a[9], "interleaved"), d);
    const int* positions = pos.defined() ? index_of(pos, "positions", {B, N}) : nullptr;
    const float eps = as_float(a[8], "eps");
    fa_heads oq{}, ok{};
    if (dq.defined()) oq = heads_of(dq, "dq", q, q.sizes(), true);
    if (dk.defined()) ok = heads_of(dk, "dk", q, k.sizes(), true);
    OneDevice(q).also(k).also(wq).also(wk).also(table).also(pos).also(gq).also(gk).also(dq).also(dk);
    Launch on(q, a[12]);
    if (!dq.defined()) oq = heads_of(dq = rows_like(q), "dq", q);
    if (!dk.defined()) ok = heads_of(dk = rows_like(k), "dk", q);
    // a set without heads leaves its weights' gradient unwritten: zero
    const at::Tensor dw = hq.H && hk.H ? fresh(q, {2, d}, at::kFloat) : at::zeros({2, d}, q.options().dtype(at::kFloat));
    Scratch ws;
    ws.take(lib.norm_rope_bwd_bytes(d), on.stream);
    float* w = static_cast<float*>(dw.data_ptr());
    const int rc = lib.norm_rope_bwd(&hgq, &hgk, &hq, &hk, &oq, &ok, w, w + d, B, N, d, wq.data_ptr(), wk.data_ptr(),
                                     eps, &rp, positions, dt, ws.ptr, ws.size, on.stream);
    if (rc != FA_OK) return PyLong_FromLong(rc);
    c10::impl::ExcludeDispatchKeyGuard plain(c10::autograd_dispatch_keyset_with_ADInplaceOrView);
    return tuple_of({dq, dk, at::as_strided(dw, {d}, {1}, 0), at::as_strided(dw, {d}, {1}, d)});
  });
}

// The int32 arrays of a batch over a paged cache
struct Batch {
  int B, width;
  const int *cu, *lens, *table;
  Batch(const at::Tensor& block_table, const at::Tensor& cu_seqlens, const at::Tensor& seq_lens) {
    if (seq_lens.dim() != 1) bad_value("seq_lens must be [B]");
    const int64_t b = seq_lens.size(0);
    B = as_int(b, "B");
    lens = index_of(seq_lens, "seq_lens", {b});
    cu = index_of(cu_seqlens, "cu_seqlens", {b + 1});
    if (block_table.dim() != 2) bad_value("block_table must be [B, pages per sequence]");
    table = index_of(block_table, "block_table", {b, block_table.size(1)});
    width = as_int(block_table.size(1), "the table's width");
  }
};

// (k, v, k_pages, v_pages, block_table, cu_seqlens, seq_lens, rope, interleaved, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &kp = tensor(a[2], "k_pages"),
                     &vp = tensor(a[3], "v_pages"), &table = tensor(a[4], "block_table"),
                     &cu = tensor(a[5], "cu_seqlens"), &lens = tensor(a[6], "seq_lens");
    const at::Tensor rope = optional_tensor(a[7], "rope");
    const fa_dtype dt = type_code(k, "k and v");
    if (k.dim() != 3) bad_value("k and v must be [T, Hkv, d]");
    const fa_heads hk = heads_of(k, "k", k), hv = heads_of(v, "v", k, k.sizes());
    const fa_paged_kv kv = cache_of(kp, vp, k);
    if (kv.Hkv != hk.H || kv.d != k.size(2)) bad_value("the cache must have k's heads and head dimension");
    for (int i = 0; i < 3; ++i)
      if (kp.size(i) > 1 && kp.stride(i) == 0) bad_value("the rows of the cache must not overlap");
    const Batch batch(table, cu, lens);
    const fa_rope rp = rope_of(rope, as_bool(a[8], "interleaved"), k.size(2));
    OneDevice(k).also(v).also(kp).also(vp).also(table).also(cu).also(lens).also(rope);
    not_recorded({{&k, "k"}, {&v, "v"}, {&kp, "k_pages"}, {&vp, "v_pages"}});
    Launch on(k, a[9]);
    const int rc = lib.append(&kv, &hk, &hv, batch.B, as_int(k.size(0), "T"), batch.cu, batch.lens, batch.table,
                              batch.width, &rp, dt, on.stream);
    return PyLong_FromLong(rc);
  });
}

// (q, k_pages, v_pages, block_table, cu_seqlens, seq_lens, max_q, causal, scale, out, lse, workspace, stream)
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    const at::Tensor &q = tensor(a[0], "q"), &kp = tensor(a[1], "k_pages"), &vp = tensor(a[2], "v_pages"),
                     &table = tensor(a[3], "block_table"), &cu = tensor(a[4], "cu_seqlens"),
                     &lens = tensor(a[5], "seq_lens");
    at::Tensor out = optional_tensor(a[9], "out"), lse = optional_tensor(a[10], "lse");
    const at::Tensor ws = optional_tensor(a[11], "workspace");
    const fa_dtype dt = type_code(q, "q");
    if (q.dim() != 3) bad_value("q must be [T, Hq, d]");
    const int T = as_int(q.size(0), "T");
    const fa_heads hq = heads_of(q, "q", q);
    const fa_paged_kv kv = cache_of(kp, vp, q);
    if (kv.d != q.size(2)) bad_value("the cache must have q's head dimension");
    const Batch batch(table, cu, lens);
    const int max_q = as_int(a[6], "max_q");
    const bool causal = as_bool(a[7], "causal");
    const float scale = a[8] == Py_None ? (float)(1.0 / std::sqrt((double)kv.d)) : as_float(a[8], "scale");
    fa_heads ho{};
    if (out.defined()) ho = heads_of(out, "out", q, q.sizes(), true);
    if (lse.defined() && (lse.scalar_type() != at::kFloat || lse.dim() != 2 || lse.size(0) != T ||
                          lse.size(1) != hq.H || !lse.is_contiguous()))
      bad_value("lse must be a contiguous [T, Hq] float32 tensor");
    if (ws.defined() && (ws.scalar_type() != at::kByte || !ws.is_contiguous()))
      bad_value("workspace must be a contiguous uint8 tensor");
    OneDevice(q).also(kp).also(vp).also(table).also(cu).also(lens).also(out).also(lse).also(ws);
    not_recorded({{&q, "q"}, {&kp, "k_pages"}, {&vp, "v_pages"}});
    Launch on(q, a[12]);
    if (!out.defined()) ho = heads_of(out = rows_like(q), "out", q);
    if (!lse.defined()) lse = fresh(q, {T, hq.H}, at::kFloat);
    const bool narrow = (int64_t)batch.width * kv.page_size <= FA_PAGED_WHOLE_KEYS;  // needs no workspace
    Scratch own;
    if (!ws.defined() && !narrow) own.take(lib.attend_bytes(hq.H, kv.Hkv, kv.d, max_q), on.stream);
    const int rc = lib.attend(&kv, &hq, &ho, static_cast<float*>(lse.data_ptr()), batch.B, T, max_q, batch.cu,
                              batch.lens, batch.table, batch.width, scale, causal, dt,
                              ws.defined() ? ws.data_ptr() : own.ptr, ws.defined() ? (size_t)ws.numel() : own.size,
                              on.stream);
    return rc == FA_OK ? tuple_of({out, lse}) : PyLong_FromLong(rc);
  });
}

// bind(addresses of the six library functions in Library's order)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    void* f[6];
    for (int i = 0; i < 6; ++i) {
      f[i] = PyLong_AsVoidPtr(a[i]);
      if (!f[i]) bad_value("a function is missing");
    }
    lib.norm_rope = reinterpret_cast<decltype(lib.norm_rope)>(f[0]);
    lib.norm_rope_bwd = reinterpret_cast<decltype(lib.norm_rope_bwd)>(f[1]);
    lib.norm_rope_bwd_bytes = reinterpret_cast<decltype(lib.norm_rope_bwd_bytes)>(f[2]);
    lib.append = reinterpret_cast<decltype(lib.append)>(f[3]);
    lib.attend = reinterpret_cast<decltype(lib.attend)>(f[4]);
    lib.attend_bytes = reinterpret_cast<decltype(lib.attend_bytes)>(f[5]);
    Py_RETURN_NONE;
  });
}

#define FAST(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST("bind", bind),     FAST("norm_rope", norm_rope), FAST("norm_rope_backward", norm_rope_backward),
                         FAST("append", append), FAST("attend", attend),       {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fa_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_torch() { return PyModule_Create(&module); }
