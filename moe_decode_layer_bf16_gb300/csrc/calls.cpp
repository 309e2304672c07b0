// The attention operators' calls from Python, for steps whose kernels take a few
// microseconds: the checks of the tensors and the call of the C ABI without the
// Python attribute reads and ctypes conversions they would otherwise cost
// (kv_cache_append: 9 us of them for a 5 us kernel).
//
// Each function takes its arguments by position and returns the library's status,
// or -1 if an argument is not as the operator wants it; the Python function behind
// it then finds out which and raises.  Nothing is launched in that case.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <exception>

#include "../../include/moe_decode.h"

namespace {

struct Refused {};
struct PythonError {};  // the interpreter's error is set

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) throw Refused();
  return THPVariable_Unpack(o);
}

void want(bool ok) {
  if (!ok) throw Refused();
}

bool is_codes(const at::Tensor& t) {
  return t.scalar_type() == at::kByte || t.scalar_type() == at::kFloat8_e4m3fn;
}

bool dense(const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape) {
  return t.scalar_type() == type && t.sizes() == shape && t.is_contiguous();
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused();
  }
  want(v >= INT32_MIN && v <= INT32_MAX);
  return v;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused();
  }
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError();
  return v != 0;
}

// The stream's handle: an integer, or the current stream of the tensors' device,
// which is the current device.
void* stream_of(PyObject* o, int device) {
  want(device >= 0 && device == c10::cuda::current_device());
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused();
  }
  return p;
}

// Elements between rows of n dense ones; where there is only one row, its
// stride says nothing.
int64_t row_stride(const at::Tensor& t, int64_t n) { return t.size(0) > 1 ? t.stride(0) : (n + 7) / 8 * 8; }

bool dense_rows(const at::Tensor& t, int64_t inner) {  // [tokens, heads, dim], the last two dense
  return t.scalar_type() == at::kBFloat16 && t.dim() == 3 && t.size(2) == inner && (inner == 1 || t.stride(2) == 1) &&
         (t.size(1) == 1 || t.stride(1) == inner);
}

size_t room(const at::Tensor& ws, int device) {
  want(ws.is_contiguous() && ws.get_device() == device);
  return ws.nbytes();
}

// A C entry from Python: no C++ exception leaves it.
template <class F>
PyObject* call(Py_ssize_t got, Py_ssize_t wanted, F&& f) {
  if (got != wanted) {
    PyErr_Format(PyExc_TypeError, "%zd arguments are wanted, got %zd", wanted, got);
    return nullptr;
  }
  try {
    return PyLong_FromLong(f());
  } catch (const Refused&) {
    return PyLong_FromLong(-1);
  } catch (const PythonError&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

// x, w, w_s, out, workspace, e8m0, stream
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 7, [&]() -> int {
    const at::Tensor &x = tensor(a[0]), &w = tensor(a[1]), &ws = tensor(a[2]), &out = tensor(a[3]), &work = tensor(a[4]);
    want(x.dim() == 2 && w.dim() == 2);
    const int64_t M = x.size(0), K = x.size(1), N = w.size(0);
    const int dev = x.get_device();
    const bool f32 = out.scalar_type() == at::kFloat;
    want(x.scalar_type() == at::kBFloat16 && (K == 1 || x.stride(1) == 1) && is_codes(w) && w.size(1) == K &&
         w.is_contiguous() && dense(ws, at::kFloat, {(N + 127) / 128, (K + 127) / 128}) &&
         dense(out, f32 ? at::kFloat : at::kBFloat16, {M, N}) && M <= INT32_MAX && N <= INT32_MAX && K <= INT32_MAX);
    want(w.get_device() == dev && ws.get_device() == dev && out.get_device() == dev);
    const size_t bytes = room(work, dev);
    const bool e8m0 = truth(a[5]);
    void* s = stream_of(a[6], dev);
    return fp8_linear(x.data_ptr(), row_stride(x, K), static_cast<const uint8_t*>(w.data_ptr()),
                      static_cast<const float*>(ws.data_ptr()), (int)M, (int)N, (int)K, e8m0, out.data_ptr(), f32,
                      work.data_ptr(), bytes, s);
  });
}

struct Batch {
  moe_kv_cache c;
  const int32_t *table, *start, *lens;
  int width, B;
};

// k_cache, v_cache, k_scale, v_scale, page_table, q_start, lens
Batch batch(PyObject* const* a, int dev) {
  const at::Tensor &k = tensor(a[0]), &v = tensor(a[1]), &ks = tensor(a[2]), &vs = tensor(a[3]), &t = tensor(a[4]),
                   &q = tensor(a[5]), &l = tensor(a[6]);
  want(k.dim() == 4 && is_codes(k) && is_codes(v) && v.sizes() == k.sizes() && k.is_contiguous() && v.is_contiguous());
  want(l.dim() == 1 && t.dim() == 2);
  const int64_t B = l.size(0);
  want(dense(ks, at::kFloat, {k.size(0), k.size(1)}) && dense(vs, at::kFloat, {k.size(0), k.size(1)}) &&
       dense(l, at::kInt, {B}) && dense(q, at::kInt, {B + 1}) && dense(t, at::kInt, {B, t.size(1)}));
  for (const at::Tensor* x : {&k, &v, &ks, &vs, &t, &q, &l}) want(x->get_device() == dev);
  for (int i = 0; i < 4; ++i) want(k.size(i) <= INT32_MAX);
  want(B <= INT32_MAX && t.size(1) <= INT32_MAX);
  return {{static_cast<uint8_t*>(k.data_ptr()), static_cast<uint8_t*>(v.data_ptr()), static_cast<float*>(ks.data_ptr()),
           static_cast<float*>(vs.data_ptr()), (int)k.size(0), (int)k.size(1), (int)k.size(2), (int)k.size(3)},
          static_cast<const int32_t*>(t.data_ptr()), static_cast<const int32_t*>(q.data_ptr()),
          static_cast<const int32_t*>(l.data_ptr()), (int)t.size(1), (int)B};
}

// k, v, the batch's seven, max_new, workspace, stream
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 12, [&]() -> int {
    const at::Tensor &k = tensor(a[0]), &v = tensor(a[1]);
    const int dev = k.get_device();
    const Batch b = batch(a + 2, dev);
    const at::Tensor& work = tensor(a[10]);
    want(dense_rows(k, b.c.head_dim) && dense_rows(v, b.c.head_dim) && k.size(1) == b.c.kv_heads && v.sizes() == k.sizes() &&
         v.get_device() == dev && k.size(0) <= INT32_MAX);
    const int max_new = (int)integer(a[9]);
    const size_t bytes = room(work, dev);
    void* s = stream_of(a[11], dev);
    const int64_t row = (int64_t)b.c.kv_heads * b.c.head_dim;
    return kv_cache_append(&b.c, k.data_ptr(), row_stride(k, row), v.data_ptr(), row_stride(v, row), b.table, b.width,
                           b.start, b.lens, b.B, (int)k.size(0), max_new, work.data_ptr(), bytes, s);
  });
}

// q, the batch's seven, max_new, out, workspace, lse, sm_scale, softcap, window, slopes, stream
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 17, [&]() -> int {
    const at::Tensor& q = tensor(a[0]);
    const int dev = q.get_device();
    const Batch b = batch(a + 1, dev);
    const at::Tensor &out = tensor(a[9]), &work = tensor(a[10]);
    const int64_t d = b.c.head_dim;
    want(dense_rows(q, d));
    const int64_t total = q.size(0), heads = q.size(1);
    want(dense(out, at::kBFloat16, q.sizes()) && out.get_device() == dev && total <= INT32_MAX && heads <= INT32_MAX);
    float *lse = nullptr, *slopes = nullptr;
    if (a[11] != Py_None) {
      const at::Tensor& t = tensor(a[11]);
      want(dense(t, at::kFloat, {total, heads}) && t.get_device() == dev);
      lse = static_cast<float*>(t.data_ptr());
    }
    if (a[15] != Py_None) {
      const at::Tensor& t = tensor(a[15]);
      want(dense(t, at::kFloat, {heads}) && t.get_device() == dev);
      slopes = static_cast<float*>(t.data_ptr());
    }
    const int max_new = (int)integer(a[8]), window = (int)integer(a[14]);
    const double scale = a[12] == Py_None ? 1.0 / std::sqrt((double)d) : number(a[12]), cap = number(a[13]);
    const size_t bytes = room(work, dev);
    void* s = stream_of(a[16], dev);
    return decode_attention(&b.c, q.data_ptr(), row_stride(q, heads * d), (int)heads, b.table, b.width, b.start, b.lens,
                            b.B, (int)total, max_new, (float)scale, (float)cap, window, slopes, out.data_ptr(), lse,
                            work.data_ptr(), bytes, s);
  });
}

PyMethodDef methods[] = {{"fp8_linear", (PyCFunction)(void (*)(void))linear, METH_FASTCALL, nullptr},
                         {"kv_cache_append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, nullptr},
                         {"decode_attention", (PyCFunction)(void (*)(void))attention, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
