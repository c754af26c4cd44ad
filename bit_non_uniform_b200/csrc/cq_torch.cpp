// cq_torch.cpp -- the host side of the INT8 calls on torch tensors.
//
// A decode step makes these calls one after another, and the small ones take
// 4 to 7 us on the GPU: through Python argument checks and ctypes the host
// needed 10 us for each and set the pace; here it needs about half.  Each
// function takes a call whose arguments are all as they should be (CUDA
// tensors of the current device, the right types and shapes, contiguous),
// allocates the outputs, launches on the current stream and returns the
// outputs, or libcq's status as an int.  For anything else it returns None and
// the Python binding goes its general way: that one says what is wrong, or
// switches device and stream.
#include <Python.h>

#include <ATen/cuda/CUDAContext.h>
#include <ATen/cuda/EmptyTensor.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "cq.h"

namespace {

const at::Tensor* tensor(PyObject* o) {
  return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr;
}

// A contiguous tensor of this type, shape and device.
bool is(const at::Tensor* t, at::ScalarType dtype, at::IntArrayRef shape, c10::DeviceIndex dev) {
  return t && t->scalar_type() == dtype && t->sizes() == shape && t->is_cuda() &&
         t->get_device() == dev && t->is_contiguous();
}

// Integer arguments; false when the object is not a plain int.
bool integer(PyObject* o, long& v) {
  if (!PyLong_CheckExact(o)) return false;
  v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return v >= INT32_MIN && v <= INT32_MAX;
}

// The workspace argument: None, or a contiguous tensor of the device.
bool scratch(PyObject* o, c10::DeviceIndex dev, void*& ptr, size_t& bytes) {
  ptr = nullptr;
  bytes = 0;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o);
  if (!t || !t->is_cuda() || t->get_device() != dev || !t->is_contiguous()) return false;
  ptr = t->data_ptr();
  bytes = t->nbytes();
  return true;
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType dtype, c10::DeviceIndex dev) {
  return at::detail::empty_cuda(shape, dtype, at::Device(at::kCUDA, dev), std::nullopt);
}

PyObject* result(int status, at::Tensor out) {
  if (status != CQ_OK) return PyLong_FromLong(status);
  return THPVariable_Wrap(std::move(out));
}

PyObject* none() { Py_RETURN_NONE; }

// (x or xq, absmax or None, wq, wscale, epilogue, out_dtype, workspace or None)
PyObject* product(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 7) return none();
  const at::Tensor *x = tensor(args[0]), *wq = tensor(args[2]), *ws = tensor(args[3]);
  long epi, dt;
  if (!x || !wq || x->dim() != 2 || wq->dim() != 2 || !x->is_cuda() || !integer(args[4], epi) ||
      !integer(args[5], dt) || (dt != CQ_DTYPE_F32 && dt != CQ_DTYPE_BF16))
    return none();
  const c10::DeviceIndex dev = x->get_device();
  if (dev != c10::cuda::current_device()) return none();
  const int64_t M = x->size(0), K = x->size(1), N = wq->size(0);
  const bool codes = args[1] != Py_None;
  const at::Tensor* am = codes ? tensor(args[1]) : nullptr;
  if (!is(x, codes ? at::kChar : at::kBFloat16, {M, K}, dev) || !is(wq, at::kChar, {N, K}, dev) ||
      !is(ws, at::kFloat, {N}, dev) || (codes && !is(am, at::kFloat, {M}, dev)))
    return none();
  void* wsp;
  size_t nws;
  if (!scratch(args[6], dev, wsp, nws)) return none();
  at::Tensor own;
  if (!codes && !wsp) {
    nws = cq_gemm_i8_workspace_size(M, N, K, static_cast<int>(epi));
    if (nws) {
      own = empty({static_cast<int64_t>(nws)}, at::kByte, dev);
      wsp = own.data_ptr();
    }
  }
  at::Tensor out = empty({M, epi == CQ_EPI_SWIGLU ? N / 2 : N},
                         dt == CQ_DTYPE_F32 ? at::kFloat : at::kBFloat16, dev);
  void* stream = at::cuda::getCurrentCUDAStream(dev).stream();
  const int8_t* w = static_cast<const int8_t*>(wq->data_ptr());
  const float* s = static_cast<const float*>(ws->data_ptr());
  const int st =
      codes ? cq_gemm_i8(static_cast<const int8_t*>(x->data_ptr()),
                         static_cast<const float*>(am->data_ptr()), M, w, s, N, K,
                         static_cast<int>(epi), static_cast<int>(dt), out.data_ptr(), wsp, nws,
                         stream)
            : cq_linear_i8(static_cast<const uint16_t*>(x->data_ptr()), M, w, s, N, K,
                           static_cast<int>(epi), static_cast<int>(dt), out.data_ptr(), wsp, nws,
                           stream);
  return result(st, std::move(out));
  END_HANDLE_TH_ERRORS
}

// (tokens, topk_ids, topk_w, w_gu, s_gu, w_dn, s_dn, out_dtype, workspace or None):
// the combined output only
PyObject* moe(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9) return none();
  const at::Tensor* t[7];
  for (int i = 0; i < 7; ++i)
    if (!(t[i] = tensor(args[i]))) return none();
  long dt;
  if (t[0]->dim() != 2 || t[1]->dim() != 2 || t[5]->dim() != 3 || !t[0]->is_cuda() ||
      !integer(args[7], dt) || (dt != CQ_DTYPE_F32 && dt != CQ_DTYPE_BF16))
    return none();
  const c10::DeviceIndex dev = t[0]->get_device();
  if (dev != c10::cuda::current_device()) return none();
  const int64_t T = t[0]->size(0), H = t[0]->size(1), k = t[1]->size(1), E = t[5]->size(0),
                I = t[5]->size(2);
  if (k > INT32_MAX || E > INT32_MAX || !is(t[0], at::kBFloat16, {T, H}, dev) ||
      !is(t[1], at::kInt, {T, k}, dev) || !is(t[2], at::kFloat, {T, k}, dev) ||
      !is(t[3], at::kChar, {E, 2 * I, H}, dev) || !is(t[4], at::kFloat, {E, 2 * I}, dev) ||
      !is(t[5], at::kChar, {E, H, I}, dev) || !is(t[6], at::kFloat, {E, H}, dev))
    return none();
  void* wsp;
  size_t nws;
  if (!scratch(args[8], dev, wsp, nws)) return none();
  at::Tensor own;
  if (!wsp) {
    nws = cq_moe_i8_workspace_size(T, static_cast<int>(k), static_cast<int>(E), H, I);
    own = empty({static_cast<int64_t>(nws < 256 ? 256 : nws)}, at::kByte, dev);
    wsp = own.data_ptr();
  }
  at::Tensor out = empty({T, H}, dt == CQ_DTYPE_F32 ? at::kFloat : at::kBFloat16, dev);
  const int st = cq_moe_i8(
      static_cast<const uint16_t*>(t[0]->data_ptr()), T,
      static_cast<const int32_t*>(t[1]->data_ptr()), static_cast<const float*>(t[2]->data_ptr()),
      static_cast<int>(k), static_cast<int>(E), static_cast<const int8_t*>(t[3]->data_ptr()),
      static_cast<const float*>(t[4]->data_ptr()), static_cast<const int8_t*>(t[5]->data_ptr()),
      static_cast<const float*>(t[6]->data_ptr()), H, I, static_cast<int>(dt), nullptr,
      out.data_ptr(), wsp, nws, at::cuda::getCurrentCUDAStream(dev).stream());
  return result(st, std::move(out));
  END_HANDLE_TH_ERRORS
}

// (logits, k, bias or None, scoring, renorm, scale)
PyObject* route(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 6) return none();
  const at::Tensor* l = tensor(args[0]);
  long k, scoring;
  if (!l || l->dim() != 2 || !l->is_cuda() || !integer(args[1], k) || !integer(args[3], scoring) ||
      !PyBool_Check(args[4]) || !PyFloat_CheckExact(args[5]))
    return none();
  const c10::DeviceIndex dev = l->get_device();
  const int64_t T = l->size(0), E = l->size(1);
  const bool f32 = l->scalar_type() == at::kFloat;
  if (dev != c10::cuda::current_device() || k < 0 || k > E || E > INT32_MAX ||
      !is(l, f32 ? at::kFloat : at::kBFloat16, {T, E}, dev))
    return none();
  const at::Tensor* b = nullptr;
  if (args[2] != Py_None) {
    b = tensor(args[2]);
    if (!is(b, at::kFloat, {E}, dev)) return none();
  }
  at::Tensor ids = empty({T, k}, at::kInt, dev), w = empty({T, k}, at::kFloat, dev);
  const int st = cq_moe_route(
      l->data_ptr(), f32 ? CQ_DTYPE_F32 : CQ_DTYPE_BF16, T, static_cast<int>(E),
      static_cast<int>(k), b ? static_cast<const float*>(b->data_ptr()) : nullptr,
      static_cast<int>(scoring), args[4] == Py_True, static_cast<float>(PyFloat_AS_DOUBLE(args[5])),
      static_cast<int32_t*>(ids.data_ptr()), static_cast<float*>(w.data_ptr()),
      at::cuda::getCurrentCUDAStream(dev).stream());
  if (st != CQ_OK) return PyLong_FromLong(st);
  PyObject* a = THPVariable_Wrap(std::move(ids));
  PyObject* c = THPVariable_Wrap(std::move(w));
  PyObject* both = a && c ? PyTuple_Pack(2, a, c) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(c);
  return both;
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"product", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(product)), METH_FASTCALL,
     "cq_gemm_i8 / cq_linear_i8 on checked tensors"},
    {"moe", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(moe)), METH_FASTCALL,
     "cq_moe_i8 on checked tensors"},
    {"route", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(route)), METH_FASTCALL,
     "cq_moe_route on checked tensors"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_cq_torch", "libcq calls on torch tensors", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cq_torch() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", CQ_BUILT_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
