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

int32_t* ints(const at::Tensor& t, at::IntArrayRef shape, int dev) {
  want(dense(t, at::kInt, shape) && t.get_device() == dev);
  return static_cast<int32_t*>(t.data_ptr());
}

// Rows of [M, n] bf16 values, dense but for the step from row to row.
int64_t bf16_rows(const at::Tensor& t, int64_t M, int64_t n, int dev) {
  want(t.scalar_type() == at::kBFloat16 && t.dim() == 2 && t.size(0) == M && t.size(1) == n && (n == 1 || t.stride(1) == 1) &&
       t.get_device() == dev);
  return row_stride(t, n);
}

// residual, gain, codes, scales, residual_out, eps, x, out, e8m0, stream
PyObject* norm_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 10, [&]() -> int {
    const at::Tensor &res = tensor(a[0]), &gain = tensor(a[1]), &codes = tensor(a[2]), &scales = tensor(a[3]),
                     &res_out = tensor(a[4]);
    want(res.dim() == 2);
    const int64_t M = res.size(0), H = res.size(1);
    const int dev = res.get_device();
    want(M <= INT32_MAX && H <= INT32_MAX);
    const int64_t ldr = bf16_rows(res, M, H, dev);
    want(dense(gain, at::kBFloat16, {H}) && gain.get_device() == dev);
    want(is_codes(codes) && codes.is_contiguous() && codes.dim() == 2 && codes.size(0) == M && codes.size(1) == H &&
         codes.get_device() == dev);
    want(dense(scales, at::kFloat, {(H + 127) / 128, (M + 3) / 4 * 4}) && scales.get_device() == dev);
    want(dense(res_out, at::kBFloat16, {M, H}) && res_out.get_device() == dev);
    const double eps = number(a[5]);
    const void* x = nullptr;
    int64_t ldx = 0;
    if (a[6] != Py_None) {
      const at::Tensor& t = tensor(a[6]);
      ldx = bf16_rows(t, M, H, dev);
      x = t.data_ptr();
    }
    void* out = nullptr;
    if (a[7] != Py_None) {
      const at::Tensor& t = tensor(a[7]);
      want(dense(t, at::kBFloat16, {M, H}) && t.get_device() == dev);
      out = t.data_ptr();
    }
    const bool e8m0 = truth(a[8]);
    void* s = stream_of(a[9], dev);
    return rmsnorm_residual_fp8(x, ldx, res.data_ptr(), ldr, gain.data_ptr(), (int)M, (int)H, (float)eps, e8m0,
                                static_cast<uint8_t*>(codes.data_ptr()), static_cast<float*>(scales.data_ptr()), out,
                                res_out.data_ptr(), s);
  });
}

struct Pages {
  int32_t *table, *lens, *stack, *state;
  int width, B, capacity, page, pages, dev;
};

// page_table, lens, (new or done), free_pages, free_state, page_size, num_pages
Pages pages(PyObject* const* a) {
  const at::Tensor &table = tensor(a[0]), &lens = tensor(a[1]), &stack = tensor(a[3]);
  const int dev = table.get_device();
  want(table.dim() == 2 && stack.dim() == 1);
  const int64_t B = table.size(0), width = table.size(1), capacity = stack.size(0);
  want(B <= INT32_MAX && width <= INT32_MAX && capacity <= INT32_MAX);
  return {ints(table, {B, width}, dev), ints(lens, {B}, dev), ints(stack, {capacity}, dev), ints(tensor(a[4]), {2}, dev),
          (int)width, (int)B, (int)capacity, (int)integer(a[5]), (int)integer(a[6]), dev};
}

// page_table, lens, new, free_pages, free_state, page_size, num_pages, q_start, lens_out, free_out, positions, slots,
// workspace, stream
PyObject* extend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 14, [&]() -> int {
    const Pages p = pages(a);
    const int32_t* fresh = ints(tensor(a[2]), {p.B}, p.dev);
    int32_t *start = ints(tensor(a[7]), {(int64_t)p.B + 1}, p.dev), *lens_out = ints(tensor(a[8]), {p.B}, p.dev),
            *free_out = ints(tensor(a[9]), {2}, p.dev);
    const at::Tensor &pos = tensor(a[10]), &slots = tensor(a[11]);
    want(pos.dim() == 1 && pos.size(0) <= INT32_MAX && dense(slots, at::kLong, {pos.size(0)}) && slots.get_device() == p.dev);
    int32_t* positions = ints(pos, {pos.size(0)}, p.dev);
    const at::Tensor& work = tensor(a[12]);
    const size_t bytes = room(work, p.dev);
    void* s = stream_of(a[13], p.dev);
    return kv_pages_extend(p.table, p.width, p.lens, fresh, p.B, p.stack, p.capacity, p.state, p.page, p.pages, start, lens_out,
                           free_out, positions, static_cast<int64_t*>(slots.data_ptr()), (int)pos.size(0), work.data_ptr(),
                           bytes, s);
  });
}

// page_table, lens, done, free_pages, free_state, page_size, num_pages, lens_out, free_out, workspace, stream
PyObject* release(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 11, [&]() -> int {
    const Pages p = pages(a);
    const at::Tensor &done = tensor(a[2]), &work = tensor(a[9]);
    want((done.scalar_type() == at::kBool || done.scalar_type() == at::kByte) && done.dim() == 1 && done.size(0) == p.B &&
         done.is_contiguous() && done.get_device() == p.dev);
    int32_t *lens_out = ints(tensor(a[7]), {p.B}, p.dev), *free_out = ints(tensor(a[8]), {2}, p.dev);
    const size_t bytes = room(work, p.dev);
    void* s = stream_of(a[10], p.dev);
    return kv_pages_release(p.table, p.width, p.lens, static_cast<const uint8_t*>(done.data_ptr()), p.B, p.stack, p.capacity,
                            p.state, p.page, p.pages, lens_out, free_out, work.data_ptr(), bytes, s);
  });
}

// q, k, v, q_start, out, workspace, lse, sm_scale, softcap, window, slopes, stream, lens
PyObject* prompt(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 13, [&]() -> int {
    const at::Tensor &q = tensor(a[0]), &k = tensor(a[1]), &v = tensor(a[2]), &start = tensor(a[3]), &out = tensor(a[4]),
                     &work = tensor(a[5]);
    const int dev = q.get_device();
    want(q.dim() == 3 && k.dim() == 3 && start.dim() == 1 && start.size(0) >= 1);
    const int64_t total = q.size(0), heads = q.size(1), d = q.size(2), hk = k.size(1), B = start.size(0) - 1;
    want(dense_rows(q, d) && dense_rows(k, d) && dense_rows(v, d) && k.size(0) == total && v.sizes() == k.sizes() &&
         k.get_device() == dev && v.get_device() == dev);
    want(total <= INT32_MAX && heads <= INT32_MAX && hk <= INT32_MAX && d <= INT32_MAX && B <= INT32_MAX);
    const int32_t* starts = ints(start, {B + 1}, dev);
    want(dense(out, at::kBFloat16, q.sizes()) && out.get_device() == dev);
    float *lse = nullptr, *slopes = nullptr;
    if (a[6] != Py_None) {
      const at::Tensor& t = tensor(a[6]);
      want(dense(t, at::kFloat, {total, heads}) && t.get_device() == dev);
      lse = static_cast<float*>(t.data_ptr());
    }
    if (a[10] != Py_None) {
      const at::Tensor& t = tensor(a[10]);
      want(dense(t, at::kFloat, {heads}) && t.get_device() == dev);
      slopes = static_cast<float*>(t.data_ptr());
    }
    const double scale = a[7] == Py_None ? 1.0 / std::sqrt((double)d) : number(a[7]), cap = number(a[8]);
    const int window = (int)integer(a[9]);
    const size_t bytes = room(work, dev);
    void* s = stream_of(a[11], dev);
    const int32_t* lens = a[12] == Py_None ? nullptr : ints(tensor(a[12]), {B}, dev);
    return prompt_attention_checked(q.data_ptr(), row_stride(q, heads * d), k.data_ptr(), row_stride(k, hk * d), v.data_ptr(),
                                    row_stride(v, hk * d), (int)heads, (int)hk, (int)d, starts, lens, (int)B, (int)total,
                                    (float)scale, (float)cap, window, slopes, out.data_ptr(), lse, work.data_ptr(), bytes, s);
  });
}

PyMethodDef methods[] = {{"fp8_linear", (PyCFunction)(void (*)(void))linear, METH_FASTCALL, nullptr},
                         {"kv_cache_append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, nullptr},
                         {"decode_attention", (PyCFunction)(void (*)(void))attention, METH_FASTCALL, nullptr},
                         {"rmsnorm_residual_fp8", (PyCFunction)(void (*)(void))norm_fp8, METH_FASTCALL, nullptr},
                         {"kv_pages_extend", (PyCFunction)(void (*)(void))extend, METH_FASTCALL, nullptr},
                         {"kv_pages_release", (PyCFunction)(void (*)(void))release, METH_FASTCALL, nullptr},
                         {"prompt_attention", (PyCFunction)(void (*)(void))prompt, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
