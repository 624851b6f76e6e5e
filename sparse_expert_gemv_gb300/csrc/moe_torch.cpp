// Argument marshalling of the prompt and block operators between torch tensors
// and the C ABI of include/moe_prompt.h and include/moe_block.h, as a CPython extension: the checks of the
// tensors, the allocation of outputs, the current stream, one call. Nothing is
// computed here. It exists for latency: the smallest calls run 2 to 3 us on the
// GPU, and the same steps in Python with ctypes took 16.5 us a norm with four
// new outputs and 12.0 us a grouping; here they take 6.0 and 4.8.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Stream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <exception>
#include <optional>
#include <string>

#include "moe_block.h"
#include "moe_prompt.h"

namespace {

PyObject* g_error = nullptr;   // MoEError

// A Python exception is set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(type, format, args);
  va_end(args);
  throw Raised{};
}

const char* dtype_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kByte: return "torch.uint8";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kFloat: return "torch.float32";
    case at::kHalf: return "torch.float16";
    default: return c10::toString(t);
  }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return THPVariable_Unpack(o);
}

// A contiguous CUDA tensor of the given type and, where they are given, shape
// and device (that of `like`).
const at::Tensor& need(PyObject* o, at::ScalarType dtype, std::optional<at::IntArrayRef> shape,
                       const char* name, const at::Tensor* like = nullptr) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != dtype)
    raise(PyExc_TypeError, "%s: expected %s, got %s", name, dtype_name(dtype),
          dtype_name(t.scalar_type()));
  if (shape && t.sizes() != *shape) {
    const std::string want = c10::str(*shape), got = c10::str(t.sizes());
    raise(PyExc_ValueError, "%s: expected shape %s, got %s", name, want.c_str(), got.c_str());
  }
  if (!t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
  if (!t.is_cuda()) raise(PyExc_ValueError, "%s must be a CUDA tensor", name);
  if (like && t.device() != like->device()) {
    const std::string want = like->device().str(), got = t.device().str();
    raise(PyExc_ValueError, "%s: expected a tensor on %s, got one on %s", name, want.c_str(),
          got.c_str());
  }
  return t;
}

const at::Tensor& matrix(PyObject* o, at::ScalarType dtype, const char* name,
                         const at::Tensor* like = nullptr) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != 2)
    raise(PyExc_ValueError, "%s: expected two dimensions, got %lld", name, (long long)t.dim());
  return need(o, dtype, std::nullopt, name, like);
}

// The caller's output buffer, or a new one: of the current stream's memory, so
// the stream of the call has to be current (a block of another stream's may
// still be read there, and would return there while this call writes it).
at::Tensor output(PyObject* o, at::ScalarType dtype, at::IntArrayRef shape, const char* name,
                  const at::Tensor& like) {
  if (o != Py_None) return need(o, dtype, shape, name, &like);
  return at::detail::empty_cuda(shape, dtype, like.device(), std::nullopt);
}

int32_t int32_of(int64_t v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX)
    raise(PyExc_ValueError, "%s is out of range: %lld", name, (long long)v);
  return (int32_t)v;
}
int32_t int32_of(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return int32_of((int64_t)v, name);
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

template <typename T>
T* data(const at::Tensor& t) {
  return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
}

// The stream a call runs on: `o`, a torch.cuda.Stream of the tensor's device, or
// that device's current stream for None.
c10::cuda::CUDAStream stream_of(PyObject* o, const at::Tensor& t) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(t.device().index());
  if (!THPStream_Check(o)) raise(PyExc_TypeError, "stream must be a torch.cuda.Stream");
  const THPStream* s = reinterpret_cast<const THPStream*>(o);
  if (s->device_type != (int64_t)c10::DeviceType::CUDA || s->device_index != t.device().index())
    raise(PyExc_ValueError, "stream: expected one of %s", t.device().str().c_str());
  return c10::cuda::CUDAStream::unpack3(s->stream_id, (c10::DeviceIndex)s->device_index,
                                        (c10::DeviceType)s->device_type);
}

void check(moe_status_t st, const char* what) {
  if (st == MOE_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", (int)st, what);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

PyObject* wrap(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  PyObject* o = THPVariable_Wrap(t);
  if (!o) throw Raised{};
  return o;
}
template <typename... Ts>
PyObject* wrap_all(const Ts&... ts) {
  PyObject* tuple = PyTuple_New(sizeof...(ts));
  if (!tuple) throw Raised{};
  Py_ssize_t i = 0;
  try {
    (PyTuple_SET_ITEM(tuple, i++, wrap(ts)), ...);
  } catch (...) {
    Py_DECREF(tuple);
    throw;
  }
  return tuple;
}

// Runs `body`; C++ exceptions become Python ones.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& body) {
  try {
    if (n != want) raise(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return body();
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (x, weight, residual, eps, bf16, mxfp8, sum, y, codes, scales, stream)
//   -> (sum, y, codes, scales)
PyObject* add_rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    const at::Tensor& x = matrix(a[0], at::kBFloat16, "x");
    const int64_t T = x.size(0), H = x.size(1);
    const at::Tensor& weight = need(a[1], at::kBFloat16, at::IntArrayRef{H}, "weight", &x);
    const float eps = (float)PyFloat_AsDouble(a[3]);
    if (PyErr_Occurred()) throw Raised{};
    const bool bf16 = truth(a[4]), mxfp8 = truth(a[5]);
    if (!bf16 && !mxfp8)
      raise(PyExc_ValueError, "add_rms_norm: ask for bf16 rows, mxfp8 rows or both");
    at::Tensor residual, sum, y, codes, scales;
    if (a[2] != Py_None) residual = need(a[2], at::kBFloat16, x.sizes(), "residual", &x);
    const c10::cuda::CUDAStreamGuard on(stream_of(a[10], x));
    if (residual.defined() || a[6] != Py_None)
      sum = output(a[6], at::kBFloat16, x.sizes(), "sum", x);
    if (bf16) y = output(a[7], at::kBFloat16, x.sizes(), "y", x);
    if (mxfp8) {
      codes = output(a[8], at::kByte, x.sizes(), "codes", x);
      scales = output(a[9], at::kByte, {T, H / 32}, "scales", x);
    }
    check(moe_add_rms_norm(int32_of(T, "T"), int32_of(H, "H"), data<uint16_t>(x),
                           data<uint16_t>(residual), data<uint16_t>(weight), eps,
                           data<uint16_t>(sum), data<uint16_t>(y), data<uint8_t>(codes),
                           data<uint8_t>(scales), on.current_stream().stream()),
          "moe_add_rms_norm");
    return wrap_all(sum, y, codes, scales);
  });
}

// (ids, E, offsets, rows, slots, stream) -> (offsets, rows, slots)
PyObject* group_by_expert(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    const at::Tensor& ids = matrix(a[0], at::kInt, "ids");
    const int64_t T = ids.size(0), k = ids.size(1);
    const int32_t E = int32_of(a[1], "E");
    if (E < 1) raise(PyExc_ValueError, "E must be positive");
    const c10::cuda::CUDAStreamGuard on(stream_of(a[5], ids));
    at::Tensor offsets = output(a[2], at::kInt, {(int64_t)E + 1}, "offsets", ids);
    at::Tensor rows = output(a[3], at::kInt, {T * k}, "rows", ids);
    at::Tensor slots = output(a[4], at::kInt, ids.sizes(), "slots", ids);
    check(moe_group(int32_of(T, "T"), int32_of(k, "k"), E, data<int32_t>(ids),
                    data<int32_t>(offsets), data<int32_t>(rows), data<int32_t>(slots),
                    on.current_stream().stream()),
          "moe_group");
    return wrap_all(offsets, rows, slots);
  });
}

// (y, slots, w, residual, out, stream) -> out
PyObject* combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    const at::Tensor& y = matrix(a[0], at::kBFloat16, "y");
    const at::Tensor& slots = matrix(a[1], at::kInt, "slots", &y);
    const int64_t R = y.size(0), H = y.size(1), T = slots.size(0), k = slots.size(1);
    const at::Tensor& w = need(a[2], at::kFloat, slots.sizes(), "w", &y);
    at::Tensor residual;
    if (a[3] != Py_None)
      residual = need(a[3], at::kBFloat16, at::IntArrayRef{T, H}, "residual", &y);
    const c10::cuda::CUDAStreamGuard on(stream_of(a[5], y));
    at::Tensor out = output(a[4], at::kBFloat16, {T, H}, "out", y);
    check(moe_combine(int32_of(T, "T"), int32_of(k, "k"), int32_of(H, "H"), int32_of(R, "R"),
                      data<uint16_t>(y), data<int32_t>(slots), data<float>(w),
                      data<uint16_t>(residual), data<uint16_t>(out), on.current_stream().stream()),
          "moe_combine");
    return wrap(out);
  });
}

// (handle, device, E, N, K, silu_mul, a, a_scales, offsets, rows, out, out_scales, stream)
//   -> out, or (out, out_scales) with silu_mul
PyObject* product_run(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    moe_product_t handle = static_cast<moe_product_t>(PyLong_AsVoidPtr(a[0]));
    if (!handle && PyErr_Occurred()) throw Raised{};
    const int32_t device = int32_of(a[1], "device");
    const int64_t E = int32_of(a[2], "E"), N = int32_of(a[3], "N"), K = int32_of(a[4], "K");
    const bool silu = truth(a[5]);
    const at::Tensor& rows_of = matrix(a[6], at::kByte, "a");
    const int64_t A = rows_of.size(0);
    need(a[6], at::kByte, at::IntArrayRef{A, K}, "a");
    if (rows_of.device().index() != device)
      raise(PyExc_ValueError, "a: expected a tensor on cuda:%d, where the weights are, got one on %s",
            (int)device, rows_of.device().str().c_str());
    const at::Tensor& a_scales =
        need(a[7], at::kByte, at::IntArrayRef{A, K / 32}, "a_scales", &rows_of);
    const at::Tensor& offsets =
        need(a[8], at::kInt, at::IntArrayRef{E + 1}, "offsets", &rows_of);
    at::Tensor rows;
    int64_t R = A;
    if (a[9] != Py_None) {
      R = tensor(a[9], "rows").numel();
      rows = need(a[9], at::kInt, at::IntArrayRef{R}, "rows", &rows_of);
    }
    const c10::cuda::CUDAStreamGuard on(stream_of(a[12], rows_of));
    at::Tensor out = output(a[10], silu ? at::kByte : at::kBFloat16, {R, silu ? N / 2 : N}, "out",
                            rows_of);
    at::Tensor scales;
    if (silu)
      scales = output(a[11], at::kByte, {R, N / 64}, "out_scales", rows_of);
    else if (a[11] != Py_None)
      raise(PyExc_ValueError, "out_scales: only a product with silu_mul has scales");
    check(moe_product_run(handle, int32_of(R, "R"), int32_of(A, "A"), data<uint8_t>(rows_of),
                          data<uint8_t>(a_scales), data<int32_t>(offsets), data<int32_t>(rows),
                          silu ? nullptr : data<uint16_t>(out), silu ? data<uint8_t>(out) : nullptr,
                          data<uint8_t>(scales), on.current_stream().stream()),
          "moe_product_run");
    return silu ? wrap_all(out, scales) : wrap(out);
  });
}

// (logits, bias, k, groups, top_groups, scale, flags, ids, w, stream) -> (ids, w)
PyObject* route_experts(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const at::ScalarType type = tensor(a[0], "logits").scalar_type();
    const at::Tensor& logits = matrix(a[0], type == at::kBFloat16 ? type : at::kFloat, "logits");
    const int64_t T = logits.size(0), E = logits.size(1);
    at::Tensor bias;
    if (a[1] != Py_None) bias = need(a[1], at::kFloat, at::IntArrayRef{E}, "bias", &logits);
    const float scale = (float)PyFloat_AsDouble(a[5]);
    if (PyErr_Occurred()) throw Raised{};
    moe_route_config_t cfg{int32_of(E, "E"), int32_of(a[2], "k"), int32_of(a[3], "groups"),
                           int32_of(a[4], "top_groups"), scale, (uint32_t)int32_of(a[6], "flags")};
    if (type == at::kBFloat16) cfg.flags |= MOE_ROUTE_BF16;
    if (cfg.k < 1) raise(PyExc_ValueError, "k must be positive");
    const c10::cuda::CUDAStreamGuard on(stream_of(a[9], logits));
    at::Tensor ids = output(a[7], at::kInt, {T, cfg.k}, "ids", logits);
    at::Tensor w = output(a[8], at::kFloat, {T, cfg.k}, "w", logits);
    check(moe_route_experts(&cfg, int32_of(T, "T"), data<void>(logits), data<float>(bias),
                            data<int32_t>(ids), data<float>(w), on.current_stream().stream()),
          "moe_route_experts");
    return wrap_all(ids, w);
  });
}

// (x, residual, post, pre, gate, scale, residual_scale, eps, flags, bf16, mxfp8, sum, y, codes,
//  scales, stream) -> (sum, y, codes, scales)
PyObject* norm_add_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&] {
    const at::Tensor& x = matrix(a[0], at::kBFloat16, "x");
    const int64_t T = x.size(0), H = x.size(1);
    const at::Tensor& residual = need(a[1], at::kBFloat16, x.sizes(), "residual", &x);
    at::Tensor post, pre, gate, sum, y, codes, scales;
    if (a[2] != Py_None) post = need(a[2], at::kBFloat16, at::IntArrayRef{H}, "post_weight", &x);
    if (a[3] != Py_None) pre = need(a[3], at::kBFloat16, at::IntArrayRef{H}, "pre_weight", &x);
    float f[3];
    for (int i = 0; i < 3; ++i) {
      f[i] = (float)PyFloat_AsDouble(a[5 + i]);
      if (PyErr_Occurred()) throw Raised{};
    }
    uint32_t flags = (uint32_t)int32_of(a[8], "flags");
    if (a[4] != Py_None) {   // by its shape: a value per channel, per row or per element
      gate = tensor(a[4], "gate");
      if (gate.sizes() == at::IntArrayRef{T, H})
        flags |= MOE_NORM_GATE_FULL;
      else if (gate.sizes() == at::IntArrayRef{T, 1})
        flags |= MOE_NORM_GATE_ROW;
      else if (gate.sizes() != at::IntArrayRef{H}) {
        const std::string got = c10::str(gate.sizes());
        raise(PyExc_ValueError, "gate: expected a value per channel [H], row [T, 1] or element [T, H], got %s",
              got.c_str());
      }
      need(a[4], at::kBFloat16, std::nullopt, "gate", &x);
    }
    const bool bf16 = truth(a[9]), mxfp8 = truth(a[10]);
    if (pre.defined() && !bf16 && !mxfp8)
      raise(PyExc_ValueError, "norm_add_norm: ask for bf16 rows, mxfp8 rows or both");
    if (!pre.defined() && mxfp8)
      raise(PyExc_ValueError, "norm_add_norm: mxfp8 rows need a pre_weight");
    const c10::cuda::CUDAStreamGuard on(stream_of(a[15], x));
    sum = output(a[11], at::kBFloat16, x.sizes(), "sum", x);
    if (bf16 && pre.defined()) y = output(a[12], at::kBFloat16, x.sizes(), "y", x);
    if (mxfp8) {
      codes = output(a[13], at::kByte, x.sizes(), "codes", x);
      scales = output(a[14], at::kByte, {T, H / 32}, "scales", x);
    }
    check(moe_norm_add_norm(int32_of(T, "T"), int32_of(H, "H"), data<uint16_t>(x),
                            data<uint16_t>(residual), data<uint16_t>(post), data<uint16_t>(pre),
                            data<uint16_t>(gate), f[0], f[1], f[2], flags, data<uint16_t>(sum),
                            data<uint16_t>(y), data<uint8_t>(codes), data<uint8_t>(scales),
                            on.current_stream().stream()),
          "moe_norm_add_norm");
    return wrap_all(sum, y, codes, scales);
  });
}

// (handle, device, K, M, x, residual, out, float32, stream) -> out
PyObject* dense_run(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&] {
    moe_dense_t handle = static_cast<moe_dense_t>(PyLong_AsVoidPtr(a[0]));
    if (!handle && PyErr_Occurred()) throw Raised{};
    const int32_t device = int32_of(a[1], "device");
    const int64_t K = int32_of(a[2], "K"), M = int32_of(a[3], "M");
    const at::Tensor& x = matrix(a[4], at::kBFloat16, "x");
    const int64_t R = x.size(0);
    need(a[4], at::kBFloat16, at::IntArrayRef{R, K}, "x");
    if (x.device().index() != device)
      raise(PyExc_ValueError, "x: expected a tensor on cuda:%d, where the weight is, got one on %s",
            (int)device, x.device().str().c_str());
    at::Tensor residual;
    if (a[5] != Py_None)
      residual = need(a[5], at::kBFloat16, at::IntArrayRef{R, M}, "residual", &x);
    const bool float32 = truth(a[7]);
    const c10::cuda::CUDAStreamGuard on(stream_of(a[8], x));
    at::Tensor out = output(a[6], float32 ? at::kFloat : at::kBFloat16, {R, M}, "out", x);
    check(moe_dense_run(handle, int32_of(R, "R"), data<uint16_t>(x), data<uint16_t>(residual),
                        data<void>(out), float32, on.current_stream().stream()),
          "moe_dense_run");
    return wrap(out);
  });
}

// (MoEError): the exception of a refused call, made from (status, what)
PyObject* set_error(PyObject*, PyObject* error) {
  Py_INCREF(error);
  Py_XSETREF(g_error, error);
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"add_rms_norm", (PyCFunction)(void (*)(void))add_rms_norm, METH_FASTCALL, nullptr},
    {"group_by_expert", (PyCFunction)(void (*)(void))group_by_expert, METH_FASTCALL, nullptr},
    {"combine", (PyCFunction)(void (*)(void))combine, METH_FASTCALL, nullptr},
    {"product_run", (PyCFunction)(void (*)(void))product_run, METH_FASTCALL, nullptr},
    {"route_experts", (PyCFunction)(void (*)(void))route_experts, METH_FASTCALL, nullptr},
    {"norm_add_norm", (PyCFunction)(void (*)(void))norm_add_norm, METH_FASTCALL, nullptr},
    {"dense_run", (PyCFunction)(void (*)(void))dense_run, METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_moe_torch", nullptr, -1, kMethods,
                       nullptr,               nullptr,      nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__moe_torch(void) {
  PyObject* m = PyModule_Create(&kModule);
  if (m && PyModule_AddStringConstant(m, "built_for", MOE_BUILT_FOR) < 0) Py_CLEAR(m);
  return m;
}
