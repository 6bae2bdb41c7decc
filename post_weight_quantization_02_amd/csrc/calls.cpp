// The ordinary forms of the int8 and distillation calls from Python in one step: tensors in,
// outputs allocated, one C ABI call, tensors out.  In Python the same takes 8 to 13 us of a
// call whose kernels may take 3.
//
// Each function returns None where anything is not as it takes it -- a tensor's device, type,
// shape or strides, a gradient or tangent that is asked for, a trace, another current device,
// a status that is not ok -- and the binding's own path then does the call or says what is
// wrong with it.  Nothing is refused here.  Tensors are taken apart by the headers of the
// torch that this was built for, BUILT_FOR_TORCH, so the binding uses it with no other.
#include <torch/csrc/python_headers.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_strided.h>
#include <c10/core/GradMode.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gptq.h"

namespace {

// addresses in the library that the binding has loaded, and torch's own functions
struct {
  decltype(&gptq_int8_quantize) int8_quantize;
  decltype(&gptq_int8_matmul_workspace_size) int8_matmul_workspace_size;
  decltype(&gptq_int8_matmul) int8_matmul;
  decltype(&gptq_int8_matmul_grouped) int8_matmul_grouped;
  decltype(&gptq_distill_loss_workspace_size) distill_loss_workspace_size;
  decltype(&gptq_distill_loss) distill_loss;
} abi;
PyObject *tracing_state, *forward_ad, *level_name, *current_device, *raw_stream;

// why a call is left to Python
struct NotPlain {};
void want(bool ok) {
  if (!ok) throw NotPlain{};
}

struct Object {
  PyObject* o;
  explicit Object(PyObject* o) : o(o) { want(o != nullptr); }
  ~Object() { Py_XDECREF(o); }
};

const at::Tensor& tensor(PyObject* o) {
  want(THPVariable_Check(o));
  return THPVariable_Unpack(o);
}

int element_type(at::ScalarType t) {
  if (t == at::kFloat) return GPTQ_F32;
  if (t == at::kHalf) return GPTQ_F16;
  want(t == at::kBFloat16);
  return GPTQ_BF16;
}

// a strided tensor on `device` that neither autograd nor a wrapper has a word in
void check(const at::Tensor& t, c10::Device device, at::ScalarType type) {
  static const c10::DispatchKeySet others({c10::DispatchKey::Python, c10::DispatchKey::FuncTorchBatched,
                                           c10::DispatchKey::FuncTorchGradWrapper, c10::DispatchKey::Functionalize,
                                           c10::DispatchKey::Conjugate, c10::DispatchKey::Negative,
                                           c10::DispatchKey::ZeroTensor});
  want(t.defined() && !t.key_set().has_any(others) && t.layout() == at::kStrided && t.has_storage());
  want(t.device() == device && t.scalar_type() == type);
  want(!(t.requires_grad() && c10::GradMode::is_enabled()));
}
void check_rows(const at::Tensor& t, c10::Device device, at::ScalarType type, int64_t rows, int64_t cols) {
  check(t, device, type);
  want(t.dim() == 2 && t.size(0) == rows && t.size(1) == cols && t.stride(1) == 1 && (rows < 2 || t.stride(0) >= cols));
}
void check_whole(const at::Tensor& t, c10::Device device, at::ScalarType type, at::IntArrayRef shape) {
  check(t, device, type);
  want(t.sizes() == shape && t.is_contiguous());
}
int64_t pitch(const at::Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

// the current stream of a device that is the current one, with nothing that records or differentiates
void* stream_of(const at::Tensor& t) {
  want(t.is_cuda());
  want(Object(PyObject_CallNoArgs(tracing_state)).o == Py_None);
  want(PyLong_AsLong(Object(PyObject_GetAttr(forward_ad, level_name)).o) < 0);
  const Object device(PyLong_FromLong(t.device().index()));
  want(PyLong_AsLong(Object(PyObject_CallNoArgs(current_device)).o) == t.device().index());
  const Object stream(PyObject_CallOneArg(raw_stream, device.o));
  return PyLong_AsVoidPtr(stream.o);
}

at::ScalarType out_type(PyObject* o) {
  if (o == Py_None) return at::kFloat;
  want(THPDtype_Check(o));
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

template <typename F>
PyObject* plain_or_none(F&& call) {
  try {
    return call();
  } catch (const NotPlain&) {
  } catch (...) {       // no memory, say: the other path says so
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

// X
PyObject* int8_quantize(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return plain_or_none([&]() -> PyObject* {
    want(n_args == 1);
    const at::Tensor& X = tensor(a[0]);
    want(X.dim() == 2 && X.size(0) > 0 && X.size(1) > 0);
    const int64_t m = X.size(0), k = X.size(1), ld = (k + 127) / 128 * 128;
    check_rows(X, X.device(), X.scalar_type(), m, k);
    const int type = element_type(X.scalar_type());
    void* const stream = stream_of(X);
    at::Tensor codes = at::empty_strided({m, k}, {ld, 1}, X.options().dtype(at::kChar));
    at::Tensor scales = at::empty({m}, X.options().dtype(at::kFloat));
    want(abi.int8_quantize(X.data_ptr(), type, m, k, pitch(X), (int8_t*)codes.data_ptr(), ld, (float*)scales.data_ptr(),
                           stream) == GPTQ_OK);
    return PyTuple_Pack(2, Object(THPVariable_Wrap(codes)).o, Object(THPVariable_Wrap(scales)).o);
  });
}

// x_codes, x_scales, w_codes, w_scales, bias, out_dtype
PyObject* int8_matmul(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return plain_or_none([&]() -> PyObject* {
    want(n_args == 6);
    const at::Tensor &x = tensor(a[0]), &sx = tensor(a[1]), &w = tensor(a[2]), &sw = tensor(a[3]);
    want(x.dim() == 2 && w.dim() == 2 && x.size(0) > 0 && x.size(1) > 0 && w.size(0) > 0);
    const int64_t m = x.size(0), k = x.size(1), n = w.size(0);
    const c10::Device device = x.device();
    check_rows(x, device, at::kChar, m, k);
    check_rows(w, device, at::kChar, n, k);
    check_whole(sx, device, at::kFloat, {m});
    check_whole(sw, device, at::kFloat, {n});
    const at::ScalarType out = out_type(a[5]);
    const int type = element_type(out);
    const void* bias = nullptr;
    if (a[4] != Py_None) {
      check_whole(tensor(a[4]), device, out, {n});
      bias = tensor(a[4]).data_ptr();
    }
    void* const stream = stream_of(x);
    at::Tensor Y = at::empty({m, n}, x.options().dtype(out)), ws;
    const size_t need = abi.int8_matmul_workspace_size(m, n, k);
    if (need > 0) ws = at::empty({(int64_t)need}, x.options().dtype(at::kByte));
    want(abi.int8_matmul((const int8_t*)x.data_ptr(), pitch(x), (const float*)sx.data_ptr(), (const int8_t*)w.data_ptr(),
                         pitch(w), (const float*)sw.data_ptr(), m, n, k, bias, Y.data_ptr(), type, n,
                         need > 0 ? ws.data_ptr() : nullptr, need, stream) == GPTQ_OK);
    return THPVariable_Wrap(Y);
  });
}

// x_codes, x_scales, w_codes, w_scales, offsets, rows, bias, out_dtype
PyObject* int8_matmul_grouped(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return plain_or_none([&]() -> PyObject* {
    want(n_args == 8);
    const at::Tensor &x = tensor(a[0]), &sx = tensor(a[1]), &w = tensor(a[2]), &sw = tensor(a[3]), &off = tensor(a[4]);
    want(x.dim() == 2 && w.dim() == 3 && x.size(0) > 0 && x.size(1) > 0 && w.size(0) > 0 && w.size(1) > 0);
    const int64_t rows_x = x.size(0), k = x.size(1), experts = w.size(0), n = w.size(1);
    const c10::Device device = x.device();
    check_rows(x, device, at::kChar, rows_x, k);
    check(w, device, at::kChar);
    want(w.size(2) == k && w.stride(2) == 1);
    const int64_t ld_w = n > 1 ? w.stride(1) : k, stride_w = experts > 1 ? w.stride(0) : n * ld_w;
    want(ld_w >= k && stride_w >= n * ld_w);
    check_whole(sx, device, at::kFloat, {rows_x});
    check_whole(sw, device, at::kFloat, {experts, n});
    check_whole(off, device, at::kInt, {experts + 1});
    int64_t m = rows_x;
    const int32_t* rows = nullptr;
    if (a[5] != Py_None) {
      const at::Tensor& r = tensor(a[5]);
      want(r.dim() == 1 && r.size(0) > 0);
      m = r.size(0);
      check_whole(r, device, at::kInt, {m});
      rows = (const int32_t*)r.data_ptr();
    }
    const at::ScalarType out = out_type(a[7]);
    const int type = element_type(out);
    const void* bias = nullptr;
    if (a[6] != Py_None) {
      check_whole(tensor(a[6]), device, out, {experts, n});
      bias = tensor(a[6]).data_ptr();
    }
    void* const stream = stream_of(x);
    at::Tensor Y = at::empty({m, n}, x.options().dtype(out));
    want(abi.int8_matmul_grouped((const int8_t*)x.data_ptr(), pitch(x), (const float*)sx.data_ptr(), rows_x, rows, m,
                                 (const int32_t*)off.data_ptr(), experts, (const int8_t*)w.data_ptr(), ld_w, stride_w,
                                 (const float*)sw.data_ptr(), n, k, bias, Y.data_ptr(), type, n, stream) == GPTQ_OK);
    return THPVariable_Wrap(Y);
  });
}

// logits, ids, logprobs, temperature, tail, weights, want_grad
PyObject* distill_loss(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return plain_or_none([&]() -> PyObject* {
    want(n_args == 7);
    const at::Tensor &z = tensor(a[0]), &ids = tensor(a[1]), &lp = tensor(a[2]);
    want(z.dim() == 2 && ids.dim() == 2 && z.size(0) > 0 && z.size(1) > 0);
    const int64_t n = z.size(0), v = z.size(1), top = ids.size(1);
    const c10::Device device = z.device();
    check_rows(z, device, z.scalar_type(), n, v);
    const int type = element_type(z.scalar_type());
    check_whole(ids, device, at::kInt, {n, top});
    check_whole(lp, device, at::kFloat, {n, top});
    want(PyFloat_Check(a[3]) && PyBool_Check(a[4]) && PyBool_Check(a[6]));
    const float temperature = (float)PyFloat_AS_DOUBLE(a[3]);
    const float* weights = nullptr;
    if (a[5] != Py_None) {
      check_whole(tensor(a[5]), device, at::kFloat, {n});
      weights = (const float*)tensor(a[5]).data_ptr();
    }
    void* const stream = stream_of(z);
    at::Tensor loss = at::empty({n}, z.options().dtype(at::kFloat)), grad, ws;
    if (a[6] == Py_True) grad = at::empty({n, v}, z.options());
    const size_t need = abi.distill_loss_workspace_size(n, v);
    if (need > 0) ws = at::empty({(int64_t)need}, z.options().dtype(at::kByte));
    want(abi.distill_loss(z.data_ptr(), type, n, v, pitch(z), (const int32_t*)ids.data_ptr(), (const float*)lp.data_ptr(), top,
                          temperature, a[4] == Py_True, weights, (float*)loss.data_ptr(),
                          grad.defined() ? grad.data_ptr() : nullptr, v, need > 0 ? ws.data_ptr() : nullptr, need,
                          stream) == GPTQ_OK);
    const Object l(THPVariable_Wrap(loss));
    if (!grad.defined()) return PyTuple_Pack(2, l.o, Py_None);
    return PyTuple_Pack(2, l.o, Object(THPVariable_Wrap(grad)).o);
  });
}

// (addresses by name, torch._C._get_tracing_state, torch.autograd.forward_ad, torch._C._cuda_getDevice,
// torch._C._cuda_getCurrentRawStream)
PyObject* bind(PyObject*, PyObject* args) {
  PyObject* names;
  if (!PyArg_ParseTuple(args, "O!OOOO", &PyDict_Type, &names, &tracing_state, &forward_ad, &current_device, &raw_stream))
    return nullptr;
  bool ok = true;
  const auto set = [&](auto& to, const char* name) {
    PyObject* o = PyDict_GetItemString(names, name);
    void* p = o ? PyLong_AsVoidPtr(o) : nullptr;
    to = reinterpret_cast<std::decay_t<decltype(to)>>(p);
    ok = ok && p != nullptr;
  };
  set(abi.int8_quantize, "gptq_int8_quantize");
  set(abi.int8_matmul_workspace_size, "gptq_int8_matmul_workspace_size");
  set(abi.int8_matmul, "gptq_int8_matmul");
  set(abi.int8_matmul_grouped, "gptq_int8_matmul_grouped");
  set(abi.distill_loss_workspace_size, "gptq_distill_loss_workspace_size");
  set(abi.distill_loss, "gptq_distill_loss");
  level_name = PyUnicode_InternFromString("_current_level");
  for (PyObject* o : {tracing_state, forward_ad, current_device, raw_stream}) Py_INCREF(o);      // kept until the process ends
  if (!ok || level_name == nullptr) {
    PyErr_SetString(PyExc_RuntimeError, "an entry point is missing");
    return nullptr;
  }
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"int8_quantize", (PyCFunction)(void (*)(void))int8_quantize, METH_FASTCALL, nullptr},
    {"int8_matmul", (PyCFunction)(void (*)(void))int8_matmul, METH_FASTCALL, nullptr},
    {"int8_matmul_grouped", (PyCFunction)(void (*)(void))int8_matmul_grouped, METH_FASTCALL, nullptr},
    {"distill_loss", (PyCFunction)(void (*)(void))distill_loss, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", BUILT_FOR_TORCH) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
