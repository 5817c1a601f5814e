// The tensor front end of the paged latent cache: checks of arguments, outputs and
// workspaces, and the call into the C ABI, for calls that take a few microseconds
// on the GPU. (In Python the same checks cost 6 to 14 us a call, more than the
// kernels of a decode step.) The functions take their arguments by position; the
// public ones, with their defaults and documentation, are in ops.py.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>

#include "../../include/indexcache.h"

namespace {

constexpr int64_t kDqk = 576, kDv = 512, kRowBytes = 656;
constexpr size_t kStatusBytes = 256;
PyObject* g_error = nullptr;  // _abi.ICError

#define NEED(cond, ...) TORCH_CHECK_VALUE(cond, __VA_ARGS__)

const at::Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " is not a tensor");
  return THPVariable_Unpack(o);
}
const at::Tensor* maybe(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }
template <typename T>
T* data(const at::Tensor& t) { return static_cast<T*>(t.data_ptr()); }
template <typename T>
T* data(const at::Tensor* t) { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }

// The device of the call: x's, which the others share.
c10::Device device_of(const at::Tensor& x, std::initializer_list<const at::Tensor*> others) {
  NEED(x.is_cuda(), "lightning_indexer_cross_b200 ops need CUDA tensors (no CPU path exists)");
  for (const at::Tensor* t : others)
    if (t) {
      NEED(t->is_cuda(), "lightning_indexer_cross_b200 ops need CUDA tensors (no CPU path exists)");
      NEED(t->device() == x.device(), "tensors on different devices: ", x.device(), " and ", t->device());
    }
  return x.device();
}

ic_stream_t stream_of(c10::Device d) {
  return reinterpret_cast<ic_stream_t>(c10::cuda::getCurrentCUDAStream(d.index()).stream());
}

bool vector_of(const at::Tensor& t, at::ScalarType type, int64_t n) {
  return t.dim() == 1 && t.size(0) == n && t.scalar_type() == type && t.is_contiguous();
}

struct Cache {
  void* data;
  ic_dtype_t dtype;
  int64_t pages, page_size, stride;  // stride in bytes
};
Cache cache_of(const at::Tensor& c) {
  constexpr const char* kForm = "the cache is [num_pages, page_size, 576] bf16 or [num_pages, page_size, 656] uint8";
  NEED(c.dim() == 3, kForm);
  const bool fp8 = c.scalar_type() == at::kByte;
  const int64_t row = fp8 ? kRowBytes : kDqk;
  NEED(c.size(2) == row && (fp8 || c.scalar_type() == at::kBFloat16), kForm);
  NEED(c.stride(2) == 1 && (c.stride(1) == row || c.size(1) <= 1), "the rows of a page are dense");
  const int64_t stride = c.size(0) > 1 ? c.stride(0) : c.size(1) * row;
  return {c.data_ptr(), fp8 ? IC_FP8_E4M3 : IC_BF16, c.size(0), c.size(1), fp8 ? stride : 2 * stride};
}

struct Table {
  const int32_t* data;
  int64_t rows, width, stride;
};
Table table_of(const at::Tensor& t) {
  NEED(t.dim() == 2 && t.scalar_type() == at::kInt, "block_table is int32 [B, width]");
  const int64_t stride = t.size(0) > 1 ? t.stride(0) : t.size(1);
  NEED((t.stride(1) == 1 || t.size(1) <= 1) && stride >= t.size(1), "block_table is dense along a row");
  return {data<int32_t>(t), t.size(0), t.size(1), stride};
}

// Sizes that the C ABI takes as int.
int as_int(int64_t v) {
  NEED(v >= 0 && v < (int64_t(1) << 31), "a size of ", v, " is too large");
  return static_cast<int>(v);
}

// The given byte workspace, or a new one of which only the status word is cleared.
at::Tensor workspace_of(const at::Tensor* ws, size_t bytes, c10::Device d) {
  if (ws) {
    NEED(ws->dim() == 1 && ws->scalar_type() == at::kByte && ws->is_contiguous(), "the workspace is a uint8 vector");
    return *ws;
  }
  at::Tensor t = at::empty({static_cast<int64_t>(std::max(bytes, kStatusBytes))}, at::TensorOptions().dtype(at::kByte).device(d));
  t.narrow(0, 0, kStatusBytes).zero_();
  return t;
}

bool failed(ic_status_t s, const char* where) {
  if (s == IC_OK) return false;
  PyObject* e = PyObject_CallFunction(g_error, "is", static_cast<int>(s), where);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return true;
}

PyObject* wrong_count(const char* name, Py_ssize_t n, int want) {
  return PyErr_Format(PyExc_TypeError, "%s takes %d arguments, %zd given", name, want, n);
}

int64_t as_long(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
float as_float(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return static_cast<float>(v);
}
bool as_bool(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}
ic_rope_layout_t layout_of(PyObject* o) { return static_cast<ic_rope_layout_t>(as_long(o)); }

PyObject* new_ref(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// x, pos, freq, rot_off, layout, mscale, transpose, out
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8) return wrong_count("rope", n, 8);
  const at::Tensor &x = tensor(a[0], "x"), &pos = tensor(a[1], "pos"), &freq = tensor(a[2], "freq");
  const at::Tensor* given = maybe(a[7], "out");
  const c10::Device dev = device_of(x, {&pos, &freq, given});
  const bool f32 = x.scalar_type() == at::kFloat;
  NEED(x.dim() == 3 && (f32 || x.scalar_type() == at::kBFloat16), "x is [T, H, D], bf16 or fp32");
  const int64_t T = x.size(0), H = x.size(1), D = x.size(2), rot = 2 * freq.numel(), off = as_long(a[3]);
  NEED(x.stride(2) == 1 || D == 1, "x is dense along D");
  NEED(vector_of(pos, at::kLong, T), "pos is int64 [T], dense");
  NEED(vector_of(freq, at::kDouble, freq.numel()), "freq is float64 [rot_dim / 2], dense");
  NEED(off >= 0 && off <= D - rot, "the rotated dims lie in the head");
  const c10::cuda::OptionalCUDAGuard guard(dev);
  at::Tensor out;
  if (given) {
    out = *given;
    NEED(out.sizes() == x.sizes() && out.scalar_type() == x.scalar_type() && (out.stride(2) == 1 || D == 1),
         "out is like x, dense along D");
  } else {
    out = at::empty({T, H, D}, x.options());
  }
  if (T > 0 && H > 0 &&
      failed(ic_rope(x.data_ptr(), x.stride(0), x.stride(1), data<int64_t>(pos), data<double>(freq),
                     as_float(a[5]), layout_of(a[4]), as_bool(a[6]),
                     f32 ? IC_F32 : IC_BF16, T, as_int(H), as_int(D), as_int(off), as_int(rot), out.data_ptr(),
                     out.stride(0), out.stride(1), stream_of(dev)),
             "ic_rope"))
    return nullptr;
  return given ? new_ref(a[7]) : THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// kv, slots, cache, pos, freq, layout, mscale, workspace
PyObject* latent_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8) return wrong_count("latent_append", n, 8);
  const at::Tensor &kv = tensor(a[0], "kv"), &slots = tensor(a[1], "slots"), &cache = tensor(a[2], "cache");
  const at::Tensor *pos = maybe(a[3], "pos"), *freq = maybe(a[4], "freq"), *given = maybe(a[7], "workspace");
  const c10::Device dev = device_of(kv, {&slots, &cache, pos, freq, given});
  const Cache c = cache_of(cache);
  NEED(kv.dim() == 2 && kv.size(1) == kDqk && kv.stride(1) == 1 && kv.scalar_type() == at::kBFloat16,
       "kv is bf16 [T, 576], dense along a row");
  const int64_t T = kv.size(0);
  NEED(vector_of(slots, at::kLong, T), "slots is int64 [T], dense");
  NEED((pos == nullptr) == (freq == nullptr), "pos and freq come together");
  NEED(!pos || vector_of(*pos, at::kLong, T), "pos is int64 [T], dense");
  NEED(!freq || vector_of(*freq, at::kDouble, (kDqk - kDv) / 2), "freq is float64 [32], dense");
  const c10::cuda::OptionalCUDAGuard guard(dev);
  at::Tensor ws = workspace_of(given, ic_latent_append_workspace_size(), dev);
  if (T > 0 &&
      failed(ic_latent_append(kv.data_ptr(), kv.stride(0), data<int64_t>(slots), data<int64_t>(pos), data<double>(freq),
                              as_float(a[6]), layout_of(a[5]), T, c.dtype, c.data, c.pages,
                              as_int(c.page_size), c.stride, ws.data_ptr(), ws.numel(), stream_of(dev)),
             "ic_latent_append"))
    return nullptr;
  return given ? new_ref(a[7]) : THPVariable_Wrap(std::move(ws));
  END_HANDLE_TH_ERRORS
}

// cache, block_table, cu_len, out, workspace
PyObject* latent_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 5) return wrong_count("latent_read", n, 5);
  const at::Tensor &cache = tensor(a[0], "cache"), &table = tensor(a[1], "block_table"), &cu = tensor(a[2], "cu_len"),
                   &out = tensor(a[3], "out");
  const at::Tensor* given = maybe(a[4], "workspace");
  const c10::Device dev = device_of(cache, {&table, &cu, &out, given});
  const Cache c = cache_of(cache);
  const Table t = table_of(table);
  NEED(vector_of(cu, at::kLong, t.rows + 1), "cu_len is int64 [B + 1], dense");
  NEED(out.dim() == 2 && out.size(1) == kDqk && out.scalar_type() == at::kBFloat16 && out.is_contiguous(),
       "out is bf16 [R, 576], dense");
  const c10::cuda::OptionalCUDAGuard guard(dev);
  if (out.size(0) > 0 && t.rows > 0) {
    const at::Tensor ws = workspace_of(given, ic_latent_read_workspace_size(), dev);
    if (failed(ic_latent_read(c.data, c.dtype, c.pages, as_int(c.page_size), c.stride, t.data, t.stride, as_int(t.width),
                              data<int64_t>(cu), as_int(t.rows), out.data_ptr(), out.size(0), ws.data_ptr(), ws.numel(),
                              stream_of(dev)),
               "ic_latent_read"))
      return nullptr;
  }
  return new_ref(a[3]);
  END_HANDLE_TH_ERRORS
}

// Checks the arguments that the two attentions share; makes the outputs that are not given.
struct Outputs {
  at::Tensor out, lse;
  ic_dtype_t dtype;
};
Outputs outputs_of(const at::Tensor& q, const at::Tensor* sink, const at::Tensor* gate, long code, const at::Tensor* out,
                   const at::Tensor* lse, bool want_lse) {
  const auto lead = q.sizes().slice(0, q.dim() - 1);
  c10::SmallVector<int64_t, 4> wide(lead.begin(), lead.end());
  wide.push_back(kDv);
  NEED(q.size(-1) == kDqk && q.scalar_type() == at::kBFloat16 && q.is_contiguous(), "q is bf16 [..., H, 576], dense");
  NEED(!sink || vector_of(*sink, at::kFloat, q.size(-2)), "sink is fp32 [H], dense");
  NEED(!gate || (gate->sizes() == at::IntArrayRef(wide) && gate->scalar_type() == at::kBFloat16 && gate->is_contiguous()),
       "gate is bf16 [..., H, 512], dense");
  Outputs o;
  if (out) {
    o.dtype = out->scalar_type() == at::kFloat ? IC_F32 : IC_BF16;
    NEED(out->sizes() == at::IntArrayRef(wide) && out->is_contiguous() &&
             (o.dtype == IC_F32 || out->scalar_type() == at::kBFloat16),
         "out is [..., H, 512], bf16 or fp32, dense");
    o.out = *out;
  } else {
    o.dtype = static_cast<ic_dtype_t>(code);
    o.out = at::empty(wide, q.options().dtype(code == IC_F32 ? at::kFloat : at::kBFloat16));
  }
  if (lse) {
    NEED(lse->sizes() == lead && lse->scalar_type() == at::kFloat && lse->is_contiguous(), "lse is fp32 [..., H], dense");
    o.lse = *lse;
  } else if (want_lse) {
    o.lse = at::empty(lead, q.options().dtype(at::kFloat));
  }
  return o;
}
PyObject* pair_of(Outputs& o, PyObject* out, PyObject* lse) {
  PyObject* first = out != Py_None ? new_ref(out) : THPVariable_Wrap(o.out);
  PyObject* second = lse != Py_None ? new_ref(lse) : o.lse.defined() ? THPVariable_Wrap(o.lse) : new_ref(Py_None);
  PyObject* t = PyTuple_New(2);
  PyTuple_SET_ITEM(t, 0, first);
  PyTuple_SET_ITEM(t, 1, second);
  return t;
}

// q, cache, block_table, lens, sink, gate, sm_scale, dtype code, out, lse, want_lse, workspace
PyObject* latent_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 12) return wrong_count("latent_decode", n, 12);
  const at::Tensor &q = tensor(a[0], "q"), &cache = tensor(a[1], "cache"), &table = tensor(a[2], "block_table"),
                   &lens = tensor(a[3], "lens");
  const at::Tensor *sink = maybe(a[4], "sink"), *gate = maybe(a[5], "gate"), *out = maybe(a[8], "out"),
                   *lse = maybe(a[9], "lse"), *given = maybe(a[11], "workspace");
  const c10::Device dev = device_of(q, {&cache, &table, &lens, sink, gate, out, lse, given});
  const Cache c = cache_of(cache);
  const Table t = table_of(table);
  NEED(q.dim() == 3 || q.dim() == 4, "q is [B, H, 576] or [B, Q, H, 576]");
  const int64_t B = q.size(0), H = q.size(-2), Q = q.dim() == 4 ? q.size(1) : 1;
  NEED(t.rows == B && vector_of(lens, at::kLong, B), "block_table is [B, width], lens int64 [B], dense");
  const c10::cuda::OptionalCUDAGuard guard(dev);
  Outputs o = outputs_of(q, sink, gate, as_long(a[7]), out, lse, as_bool(a[10]));
  if (B > 0 && Q > 0 && H > 0) {
    const int b = as_int(B), nq = as_int(Q), h = as_int(H), width = as_int(t.width), ps = as_int(c.page_size);
    const at::Tensor ws = workspace_of(given, given ? 0 : ic_latent_decode_workspace_size(b, nq, h, int64_t(width) * ps), dev);
    if (failed(ic_latent_decode(q.data_ptr(), c.data, c.dtype, c.pages, ps, c.stride, t.data, t.stride, width,
                                data<int64_t>(lens), data<float>(sink), data<void>(gate),
                                as_float(a[6]), b, nq, h, o.dtype, o.out.data_ptr(),
                                o.lse.defined() ? data<float>(o.lse) : nullptr, ws.data_ptr(), ws.numel(), stream_of(dev)),
               "ic_latent_decode"))
      return nullptr;
  }
  return pair_of(o, a[8], a[9]);
  END_HANDLE_TH_ERRORS
}

// q, cache, slots, sink, gate, sm_scale, dtype code, out, lse, want_lse, workspace
PyObject* latent_sparse_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 11) return wrong_count("latent_sparse_decode", n, 11);
  const at::Tensor &q = tensor(a[0], "q"), &cache = tensor(a[1], "cache"), &slots = tensor(a[2], "slots");
  const at::Tensor *sink = maybe(a[3], "sink"), *gate = maybe(a[4], "gate"), *out = maybe(a[7], "out"),
                   *lse = maybe(a[8], "lse"), *given = maybe(a[10], "workspace");
  const c10::Device dev = device_of(q, {&cache, &slots, sink, gate, out, lse, given});
  const Cache c = cache_of(cache);
  NEED(c.dtype == IC_FP8_E4M3, "the cache holds e4m3 rows");
  NEED(q.dim() == 3, "q is [B, H, 576]");
  const int64_t B = q.size(0), H = q.size(1);
  NEED(slots.dim() == 2 && slots.size(0) == B && slots.scalar_type() == at::kInt && slots.is_contiguous(),
       "slots is int32 [B, k], dense");
  const c10::cuda::OptionalCUDAGuard guard(dev);
  Outputs o = outputs_of(q, sink, gate, as_long(a[6]), out, lse, as_bool(a[9]));
  if (B > 0 && H > 0) {
    const int b = as_int(B), h = as_int(H), k = as_int(slots.size(1));
    const at::Tensor ws = workspace_of(given, given ? 0 : ic_latent_sparse_workspace_size(b, h, k), dev);
    if (failed(ic_latent_sparse_decode(q.data_ptr(), c.data, c.pages, as_int(c.page_size), c.stride, data<int32_t>(slots),
                                       k, data<float>(sink), data<void>(gate), as_float(a[5]),
                                       b, h, o.dtype, o.out.data_ptr(), o.lse.defined() ? data<float>(o.lse) : nullptr,
                                       ws.data_ptr(), ws.numel(), stream_of(dev)),
               "ic_latent_sparse_decode"))
      return nullptr;
  }
  return pair_of(o, a[7], a[8]);
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error);
  g_error = cls;
  Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(rope),          FAST(latent_append),        FAST(latent_read),
                         FAST(latent_decode), FAST(latent_sparse_decode), {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_front", "Tensor front end of the paged latent cache.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__front() {
  PyObject* m = PyModule_Create(&module);
  // the tensors' layout is that torch's: ops.py calls nothing here under another
  if (m && PyModule_AddStringConstant(m, "torch_version", IC_TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
