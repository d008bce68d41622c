// pkv_torch.cpp -- the per-step calls of the Python binding, on torch tensors.
//
// Checks of dtype, device and layout, allocation of outputs and the call through the C ABI
// (include/pkv.h), nothing else. These calls run once per layer and step: with the same checks
// in Python and ctypes a small call spent 9 to 25 us on the host, most of it longer than on the
// GPU. A call takes its arguments in order (the Python functions around it give them names,
// defaults and documentation) and returns its outputs, or the library's status as an int when
// that is not PKV_OK.
//
// Every tensor has to be on the caches' device, which need not be the current one. With a stream
// given, outputs are allocated on that stream.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <sstream>
#include <string>

#include "pkv.h"

namespace {

constexpr int64_t kGroup = PKV_FP8_GROUP;

struct Fail {  // becomes a Python exception
  PyObject *type;
  std::string text;
};

template <class... Parts>
[[noreturn]] void fail(PyObject *type, const Parts &...parts) {
  std::ostringstream s;
  (s << ... << parts);
  throw Fail{type, s.str()};
}

// ------------------------------------------------------------------------------ arguments
const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o))
    fail(PyExc_TypeError, name, " must be a tensor, got ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}
bool given(PyObject *o) { return o != Py_None; }

int64_t integer(PyObject *o, const char *name) {
  PyObject *i = PyNumber_Index(o);
  if (!i) {
    PyErr_Clear();
    fail(PyExc_TypeError, name, " must be an integer");
  }
  const long long v = PyLong_AsLongLong(i);
  Py_DECREF(i);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    fail(PyExc_ValueError, name, " is out of range");
  }
  return v;
}
int32_t integer32(PyObject *o, const char *name) {
  const int64_t v = integer(o, name);
  if (v < INT32_MIN || v > INT32_MAX) fail(PyExc_ValueError, name, " is out of range");
  return (int32_t)v;
}
int32_t size32(int64_t v, const char *name) {
  if (v > INT32_MAX) fail(PyExc_ValueError, name, " is too large");
  return (int32_t)v;
}
float number(PyObject *o, const char *name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    fail(PyExc_TypeError, name, " must be a number");
  }
  return (float)v;
}

// ------------------------------------------------------------------------------ checks
void need(const at::Tensor &t, const char *name, at::ScalarType dtype, int index) {
  if (!t.is_cuda()) fail(PyExc_ValueError, name, " must be a CUDA tensor");
  if (t.scalar_type() != dtype)
    fail(PyExc_TypeError, name, " must be ", c10::toString(dtype), ", got ",
         c10::toString(t.scalar_type()));
  if (t.get_device() != index)
    fail(PyExc_ValueError, name, " is on ", t.device().str(), ", the caches on cuda:", index);
}
void need_shape(const at::Tensor &t, const char *name, at::ScalarType dtype, int index,
                at::IntArrayRef shape) {
  need(t, name, dtype, index);
  if (t.sizes() != shape || !t.is_contiguous())
    fail(PyExc_ValueError, name, " must be a contiguous tensor of shape ", shape, ", got ",
         t.sizes());
}

struct Cache {
  const at::Tensor &k, &v;
  const float *k_scale = nullptr, *v_scale = nullptr;
  float *k_scale_w = nullptr, *v_scale_w = nullptr;
  int index = 0;
  int64_t num_blocks = 0;
  int32_t block_size = 0, hkv = 0, d = 0;
};

// The pools of a cache: bf16, or e4m3 with their scales.
Cache cache(PyObject *ko, PyObject *vo, PyObject *kso, PyObject *vso) {
  Cache c{tensor(ko, "k_cache"), tensor(vo, "v_cache")};
  const bool fp8 = given(kso) || given(vso);
  if (given(kso) != given(vso)) fail(PyExc_ValueError, "k_scale and v_scale go together");
  const auto dtype = fp8 ? at::kFloat8_e4m3fn : at::kBFloat16;
  if (!c.k.is_cuda()) fail(PyExc_ValueError, "k_cache must be a CUDA tensor");
  c.index = c.k.get_device();
  need(c.k, "k_cache", dtype, c.index);
  need(c.v, "v_cache", dtype, c.index);
  if (c.k.dim() != 4 || c.k.sizes() != c.v.sizes())
    fail(PyExc_ValueError, "caches must be [NB, bs, Hkv, D], the same for K and V, got ",
         c.k.sizes(), " and ", c.v.sizes());
  if (!c.k.is_contiguous() || !c.v.is_contiguous())
    fail(PyExc_ValueError, "caches must be contiguous");
  c.num_blocks = c.k.size(0);
  c.block_size = size32(c.k.size(1), "block size");
  c.hkv = size32(c.k.size(2), "number of KV heads");
  c.d = size32(c.k.size(3), "head dimension");
  if (fp8) {
    const int64_t shape[3] = {c.num_blocks, c.hkv, c.block_size / kGroup};
    const at::Tensor &ks = tensor(kso, "k_scale"), &vs = tensor(vso, "v_scale");
    need_shape(ks, "k_scale", at::kFloat, c.index, shape);
    need_shape(vs, "v_scale", at::kFloat, c.index, shape);
    c.k_scale = c.k_scale_w = ks.data_ptr<float>();
    c.v_scale = c.v_scale_w = vs.data_ptr<float>();
  }
  return c;
}
void need_fp8(PyObject *kso, PyObject *vso) {
  if (!given(kso) || !given(vso)) fail(PyExc_ValueError, "k_scale and v_scale must be given");
}

struct Lists {
  const int32_t *context_lens, *tables;
  int32_t batch, width;
};
const int32_t *table(PyObject *o, const char *name, int index, int64_t batch, int32_t &width) {
  const at::Tensor &t = tensor(o, name);
  if (t.dim() != 2) fail(PyExc_ValueError, name, " must be a [B, W] int32 tensor");
  width = size32(t.size(1), name);
  need_shape(t, name, at::kInt, index, {batch < 0 ? t.size(0) : batch, t.size(1)});
  return t.data_ptr<int32_t>();
}
const int32_t *ints(PyObject *o, const char *name, int index, at::IntArrayRef shape) {
  const at::Tensor &t = tensor(o, name);
  need_shape(t, name, at::kInt, index, shape);
  return t.data_ptr<int32_t>();
}
Lists lists(PyObject *context_lens, PyObject *tables, int index) {
  Lists l{};
  const at::Tensor &c = tensor(context_lens, "context_lens");
  if (c.dim() != 1) fail(PyExc_ValueError, "context_lens must be a [B] int32 tensor");
  l.batch = size32(c.size(0), "batch");
  l.context_lens = ints(context_lens, "context_lens", index, {l.batch});
  l.tables = table(tables, "block_tables", index, l.batch, l.width);
  return l;
}

// [T, Hkv, D] bf16 rows, each token's dense; the token stride.
int64_t rows(const at::Tensor &t, const char *name, const Cache &c) {
  need(t, name, at::kBFloat16, c.index);
  if (t.dim() != 3 || t.size(1) != c.hkv || t.size(2) != c.d)
    fail(PyExc_ValueError, name, " must be [T, ", c.hkv, ", ", c.d, "], got ", t.sizes());
  if (t.stride(2) != 1 || (c.hkv > 1 && t.stride(1) != c.d))
    fail(PyExc_ValueError, name, ": each token's heads must be dense");
  return t.size(0) > 1 ? t.stride(0) : (int64_t)c.hkv * c.d;
}

// A [B, Hkv, >= length] fp32 tensor of dense rows one stride apart; the stride.
int64_t weight_rows(const at::Tensor &t, const char *name, int64_t batch, int64_t hkv,
                    int64_t length, int index) {
  need(t, name, at::kFloat, index);
  if (t.dim() != 3 || t.size(0) != batch || t.size(1) != hkv || t.size(2) < length ||
      (t.size(2) > 1 && t.stride(2) != 1) ||
      (batch > 1 && hkv > 1 && t.stride(0) != hkv * t.stride(1)))
    fail(PyExc_ValueError, name, " must be [", batch, ", ", hkv, ", >= ", length,
         "] with dense, evenly spaced rows, got ", t.sizes(), " with strides ", t.strides());
  return hkv > 1 ? t.stride(1) : batch > 1 ? t.stride(0) : t.size(2);
}

struct Weights {
  const float *in = nullptr;
  float *out = nullptr;
  int64_t in_stride = 0, out_stride = 0;
};
// (without an output: in place)
Weights weights(PyObject *in, PyObject *out, int64_t batch, int64_t hkv, int64_t length,
                int index) {
  Weights w;
  if (given(in)) {
    const at::Tensor &t = tensor(in, "weights");
    w.in_stride = weight_rows(t, "weights", batch, hkv, length, index);
    w.in = t.data_ptr<float>();
  }
  if (given(out)) {
    const at::Tensor &t = tensor(out, "weights_out");
    w.out_stride = weight_rows(t, "weights_out", batch, hkv, length, index);
    w.out = t.data_ptr<float>();
    if (w.in == w.out && w.in_stride != w.out_stride)
      fail(PyExc_ValueError, "weights and weights_out overlap with different strides");
  } else if (given(in)) {
    w.out = const_cast<float *>(w.in);
    w.out_stride = w.in_stride;
  }
  return w;
}

// ------------------------------------------------------------------------------ the call
// The device and the stream of a call: for None the device's current stream.
struct On {
  c10::cuda::OptionalCUDAGuard device;
  std::optional<c10::cuda::CUDAStreamGuard> stream_guard;
  void *stream = nullptr;
  On(int index, PyObject *o) {
    device.set_index((c10::DeviceIndex)index);
    if (!given(o)) {
      stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
      return;
    }
    PyObject *handle = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
    if (handle) {
      stream = PyLong_AsVoidPtr(handle);
      Py_DECREF(handle);
    }
    if (PyErr_Occurred()) {
      PyErr_Clear();
      fail(PyExc_TypeError, "stream must be a torch.cuda.Stream or a cudaStream_t as an integer");
    }
    stream_guard.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream),
                                                          (c10::DeviceIndex)index));
  }
};

at::Tensor empty(at::IntArrayRef shape, at::ScalarType dtype, int index) {
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(at::kCUDA, (c10::DeviceIndex)index));
}
// The given output, or a new one.
at::Tensor output(PyObject *o, const char *name, at::IntArrayRef shape, at::ScalarType dtype,
                  int index) {
  if (!given(o)) return empty(shape, dtype, index);
  const at::Tensor &t = tensor(o, name);
  need_shape(t, name, dtype, index, shape);
  return t;
}
PyObject *object(PyObject *given_one, const at::Tensor &t) {
  return given(given_one) ? Py_NewRef(given_one) : THPVariable_Wrap(t);
}

// The given decode workspace, or a new one with its work counter at zero.
at::Tensor workspace_of(PyObject *o, size_t bytes, int index) {
  if (given(o)) {
    const at::Tensor &t = tensor(o, "workspace");
    if (!t.is_cuda() || t.get_device() != index || !t.is_contiguous())
      fail(PyExc_ValueError, "workspace must be a contiguous tensor on cuda:", index);
    return t;
  }
  at::Tensor t = empty({(int64_t)std::max<size_t>(bytes, 16)}, at::kByte, index);
  t.narrow(0, 0, 16).zero_();
  return t;
}

PyObject *status_or(pkv_status s, PyObject *result) {
  if (s == PKV_OK) return result;
  Py_XDECREF(result);
  return PyLong_FromLong(s);
}

// ------------------------------------------------------------------------------ the functions
PyObject *kv_store_fp8(PyObject *const *a) {
  need_fp8(a[6], a[7]);
  const Cache c = cache(a[4], a[5], a[6], a[7]);
  const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
  const int64_t ks = rows(k, "k", c), vs = rows(v, "v", c);
  if (k.size(0) != v.size(0)) fail(PyExc_ValueError, "k and v must hold the same tokens");
  const Lists l = lists(a[2], a[3], c.index);
  const int32_t *cu = given(a[8]) ? ints(a[8], "cu_seqlens", c.index, {(int64_t)l.batch + 1}) : nullptr;
  On on(c.index, a[9]);
  return status_or(pkv_kv_store_fp8(k.data_ptr(), ks, v.data_ptr(), vs, cu, l.context_lens,
                                    l.tables, l.width, l.batch, k.size(0), c.k.data_ptr(),
                                    c.v.data_ptr(), c.k_scale_w, c.v_scale_w, c.hkv, c.d,
                                    c.block_size, c.num_blocks, on.stream),
                   Py_NewRef(Py_None));
}

PyObject *kv_gather_fp8(PyObject *const *a) {
  need_fp8(a[2], a[3]);
  const Cache c = cache(a[0], a[1], a[2], a[3]);
  int32_t width = 0;
  const int32_t *tables = table(a[4], "block_table", c.index, -1, width);
  const int32_t n = size32(tensor(a[4], "block_table").size(0), "block_table");
  const int32_t *cu = ints(a[5], "cu_seqlens_k", c.index, {(int64_t)n + 1});
  const int64_t total = integer(a[6], "total_k");
  if (total < 0) fail(PyExc_ValueError, "total_k must not be negative");
  On on(c.index, a[9]);
  const int64_t shape[3] = {total, c.hkv, c.d};
  const at::Tensor k = output(a[7], "k_out", shape, at::kBFloat16, c.index);
  const at::Tensor v = output(a[8], "v_out", shape, at::kBFloat16, c.index);
  const pkv_status s =
      pkv_kv_gather_fp8(c.k.data_ptr(), c.v.data_ptr(), c.k_scale, c.v_scale, tables, width, cu, n,
                        total, k.data_ptr(), v.data_ptr(), c.hkv, c.d, c.block_size, c.num_blocks,
                        on.stream);
  if (s != PKV_OK) return PyLong_FromLong(s);
  PyObject *ko = object(a[7], k), *vo = object(a[8], v);
  return ko && vo ? Py_BuildValue("(NN)", ko, vo) : nullptr;
}

// What every decode call takes: q, and the output it gives.
struct Decode {
  Lists l;
  int32_t hq;
  const at::Tensor &q;
};
Decode decode(PyObject *qo, PyObject *tables, PyObject *context_lens, const Cache &c) {
  const at::Tensor &q = tensor(qo, "q");
  need(q, "q", at::kBFloat16, c.index);
  if (q.dim() != 3 || q.size(2) != c.d || !q.is_contiguous())
    fail(PyExc_ValueError, "q must be a contiguous [B, Hq, ", c.d, "] tensor, got ", q.sizes());
  Decode r{lists(context_lens, tables, c.index), size32(q.size(1), "number of query heads"), q};
  if (q.size(0) != r.l.batch)
    fail(PyExc_ValueError, "q holds ", q.size(0), " sequences, context_lens ", r.l.batch);
  return r;
}

PyObject *paged_decode_attn_fp8(PyObject *const *a) {
  need_fp8(a[3], a[4]);
  const Cache c = cache(a[1], a[2], a[3], a[4]);
  const Decode r = decode(a[0], a[5], a[6], c);
  const int32_t longest = integer32(a[7], "max_context_len");
  const float scale = number(a[8], "scale");
  const int32_t splits = integer32(a[9], "num_splits");
  const Weights w = weights(a[10], a[11], r.l.batch, c.hkv, longest, c.index);
  On on(c.index, a[14]);
  const at::Tensor out = output(a[13], "out", r.q.sizes(), at::kBFloat16, c.index);
  const at::Tensor ws = workspace_of(
      a[12], given(a[12]) ? 0
                          : pkv_decode_fp8_workspace_bytes(r.l.batch, r.hq, c.hkv, c.d, longest,
                                                           splits, w.out != nullptr),
      c.index);
  const pkv_status s = pkv_paged_decode_attn_fp8(
      r.q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), c.k_scale, c.v_scale, r.l.tables, r.l.width,
      r.l.context_lens, r.l.batch, longest, r.hq, c.hkv, c.d, c.block_size, c.num_blocks, scale,
      splits, w.in, w.in_stride, w.out, w.out_stride, ws.data_ptr(), ws.nbytes(), out.data_ptr(),
      on.stream);
  return s == PKV_OK ? object(a[13], out) : PyLong_FromLong(s);
}

PyObject *paged_decode_attn_weights(PyObject *const *a) {
  const Cache c = cache(a[1], a[2], Py_None, Py_None);
  const Decode r = decode(a[0], a[3], a[4], c);
  const int32_t longest = integer32(a[5], "max_context_len");
  const float scale = number(a[6], "scale");
  const int32_t splits = integer32(a[8], "num_splits");
  if (!given(a[7]) && !given(a[9])) fail(PyExc_ValueError, "weights or weights_out must be given");
  const Weights w = weights(a[7], a[9], r.l.batch, c.hkv, longest, c.index);
  On on(c.index, a[12]);
  const at::Tensor out = output(a[11], "out", r.q.sizes(), at::kBFloat16, c.index);
  const at::Tensor ws = workspace_of(
      a[10], given(a[10]) ? 0
                          : pkv_decode_weights_workspace_bytes(r.l.batch, r.hq, c.hkv, c.d,
                                                               longest, splits),
      c.index);
  const pkv_status s = pkv_paged_decode_attn_weights(
      r.q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), r.l.tables, r.l.width, r.l.context_lens,
      r.l.batch, longest, r.hq, c.hkv, c.d, c.block_size, c.num_blocks, scale, splits, w.in,
      w.in_stride, w.out, w.out_stride, ws.data_ptr(), ws.nbytes(), out.data_ptr(), on.stream);
  return s == PKV_OK ? object(a[11], out) : PyLong_FromLong(s);
}

PyObject *kv_evict(PyObject *const *a) {
  const Cache c = cache(a[7], a[8], a[9], a[10]);
  const Lists l = lists(a[1], a[3], c.index);
  const int32_t longest = integer32(a[2], "max_context_len");
  int32_t dst_width = 0;
  const int32_t *dst = table(a[4], "dst_block_tables", c.index, l.batch, dst_width);
  const int32_t budget = integer32(a[5], "budget"), recent = integer32(a[6], "recent");
  if (budget < 1 || recent < 0 || recent > budget)
    fail(PyExc_ValueError, "budget must be at least 1 and recent between 0 and budget");
  const at::Tensor &w = tensor(a[0], "weights");
  const int64_t w_stride = weight_rows(w, "weights", l.batch, c.hkv, longest, c.index);
  On on(c.index, a[14]);
  const int64_t shape[3] = {l.batch, c.hkv, budget};
  const at::Tensor kept = output(a[11], "kept", shape, at::kInt, c.index);
  at::Tensor w_out;
  int64_t w_out_stride = budget;
  if (given(a[12])) {
    w_out = tensor(a[12], "weights_out");
    w_out_stride = weight_rows(w_out, "weights_out", l.batch, c.hkv, budget, c.index);
  } else {
    w_out = empty(shape, at::kFloat, c.index);
  }
  const at::Tensor lens = output(a[13], "new_context_lens", {l.batch}, at::kInt, c.index);
  const pkv_status s = pkv_kv_evict(
      w.data_ptr<float>(), w_stride, l.context_lens, l.batch, longest, budget, recent, l.tables,
      l.width, dst, dst_width, c.k.data_ptr(), c.v.data_ptr(), c.k_scale_w, c.v_scale_w, c.hkv,
      c.d, c.block_size, c.num_blocks, kept.data_ptr<int32_t>(), w_out.data_ptr<float>(),
      w_out_stride, lens.data_ptr<int32_t>(), on.stream);
  if (s != PKV_OK) return PyLong_FromLong(s);
  PyObject *ko = object(a[11], kept), *wo = object(a[12], w_out), *lo = object(a[13], lens);
  return ko && wo && lo ? Py_BuildValue("(NNN)", ko, wo, lo) : nullptr;
}

// A Python function of exactly N arguments; no C++ exception leaves it.
template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments wanted, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Fail &f) {
    PyErr_SetString(f.type, f.text.c_str());
  } catch (const c10::OutOfMemoryError &e) {
    if (PyObject *torch = PyImport_ImportModule("torch")) {
      if (PyObject *type = PyObject_GetAttrString(torch, "OutOfMemoryError")) {
        PyErr_SetString(type, e.what_without_backtrace());
        Py_DECREF(type);
      }
      Py_DECREF(torch);
    }
  } catch (const std::exception &e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyCFunction method() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&entry<F, N>));
}

PyMethodDef g_methods[] = {
    {"kv_store_fp8", method<kv_store_fp8, 10>(), METH_FASTCALL, nullptr},
    {"kv_gather_fp8", method<kv_gather_fp8, 10>(), METH_FASTCALL, nullptr},
    {"paged_decode_attn_fp8", method<paged_decode_attn_fp8, 15>(), METH_FASTCALL, nullptr},
    {"paged_decode_attn_weights", method<paged_decode_attn_weights, 13>(), METH_FASTCALL, nullptr},
    {"kv_evict", method<kv_evict, 15>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_pkv_torch", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pkv_torch() { return PyModule_Create(&g_module); }
