// Argument marshalling of the paged calls from torch tensors, for Python.
//
// A step of a server makes these calls once per layer, and reading a dozen
// tensors' shapes, strides and addresses one attribute at a time from Python
// takes longer than the kernels (7 of 10 us for attn_decode_paged).  Each
// function here checks the common form of its arguments and makes the call
// through attn_paged_call; it returns the call's status, or -1 for anything
// else than that form, which the Python wrapper then looks into and reports.
// Nothing is computed here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <cstring>

namespace {

using Call = int (*)(int, const int64_t*, int);
Call g_call = nullptr;

enum { PLAN = 0, APPEND = 1, DECODE = 2, SELECT = 3, SPARSE = 4 };  // CATTN_CALL_*

struct Odd {};  // not the common form

// The tensor in `o`, a plain one on the current device.
struct Reader {
  c10::DeviceIndex dev = c10::cuda::current_device();
  const at::Tensor& operator()(PyObject* o) const {
    if (!THPVariable_CheckExact(o)) throw Odd{};
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != dev || t.layout() != at::kStrided) throw Odd{};
    return t;
  }
  // A bf16 view of `dim` axes with unit last stride.
  const at::Tensor& view(PyObject* o, int64_t dim) const {
    const at::Tensor& t = (*this)(o);
    if (t.scalar_type() != at::kBFloat16 || t.dim() != dim || t.stride(dim - 1) != 1) throw Odd{};
    return t;
  }
  // The address of a contiguous array of the given type and shape.
  int64_t array(PyObject* o, at::ScalarType type, at::IntArrayRef shape) const {
    const at::Tensor& t = (*this)(o);
    if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous()) throw Odd{};
    return address(t);
  }
  static int64_t address(const at::Tensor& t) {
    return static_cast<int64_t>(reinterpret_cast<uintptr_t>(t.data_ptr()));
  }
};

struct Words {
  int64_t w[40];
  int n = 0;
  void operator()(int64_t x) { w[n++] = x; }
  void real(double x) { std::memcpy(&w[n++], &x, 8); }
  void tensor(const at::Tensor& t) {  // address and (b, h, t) strides
    (*this)(Reader::address(t));
    for (int i = 0; i < 3; ++i) (*this)(t.stride(i));
  }
  // Rows (n, heads, D): the layout's b is not read.
  void rows(const at::Tensor& t) {
    (*this)(Reader::address(t));
    (*this)(0);
    (*this)(t.stride(1));
    (*this)(t.stride(0));
  }
};

int64_t number(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Odd{};
  }
  return x;
}

// Address, row stride and width of an int32 (B, width) table.
void table(const Reader& r, PyObject* o, int64_t B, int64_t* ptr, int64_t* stride,
           int64_t* width) {
  const at::Tensor& t = r(o);
  if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != B || t.stride(1) != 1)
    throw Odd{};
  *ptr = Reader::address(t);
  *width = t.size(1);
  *stride = B > 1 ? t.stride(0) : *width;
}

int64_t stream_of(const Reader& r) {
  return static_cast<int64_t>(
      reinterpret_cast<uintptr_t>(c10::cuda::getCurrentCUDAStream(r.dev).stream()));
}

// (address, bytes) of a workspace.
void scratch(const Reader& r, PyObject* o, Words& w) {
  const at::Tensor& t = r(o);
  if (!t.is_contiguous()) throw Odd{};
  w(Reader::address(t));
  w(static_cast<int64_t>(t.nbytes()));
}

template <typename F>
PyObject* run(int which, Py_ssize_t nargs, Py_ssize_t want, F fill) {
  int st = -1;
  if (nargs == want && g_call != nullptr) {
    try {
      Words w;
      const Reader r;
      fill(r, w);
      Py_BEGIN_ALLOW_THREADS
      st = g_call(which, w.w, w.n);
      Py_END_ALLOW_THREADS
    } catch (...) {  // Odd, or an error of torch's: the long way says which
      st = -1;
    }
  }
  return PyLong_FromLong(st);
}

// decode(q, k_cache, v_cache, block_table, lengths, pages or None, scale, o, lse, workspace)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const bool sparse = n == 10 && a[5] != Py_None;
  return run(sparse ? SPARSE : DECODE, n, 10, [&](const Reader& r, Words& w) {
    const at::Tensor &q = r.view(a[0], 4), &k = r.view(a[1], 4), &v = r.view(a[2], 4),
                     &o = r.view(a[7], 4);
    const int64_t B = q.size(0), H = q.size(1), Tq = q.size(2), D = q.size(3), Hkv = k.size(1);
    if (v.sizes() != k.sizes() || k.size(3) != D || o.sizes() != q.sizes()) throw Odd{};
    double scale = 1.0 / std::sqrt(static_cast<double>(D));
    if (a[6] != Py_None) {
      scale = PyFloat_AsDouble(a[6]);
      if (scale == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Odd{};
      }
    }
    w.tensor(q);
    w.tensor(k);
    w.tensor(v);
    w.real(scale);
    for (int64_t x : {B, H, Hkv, Tq, D, k.size(0), k.size(2)}) w(x);
    int64_t ptr, stride, width;
    table(r, a[3], B, &ptr, &stride, &width);
    w(ptr);
    w(stride);
    w(width);
    w(r.array(a[4], at::kInt, {B}));
    if (sparse) {
      const at::Tensor& pages = r(a[5]);
      if (pages.dim() != 3) throw Odd{};
      w(r.array(a[5], at::kInt, {B, Hkv, pages.size(2)}));
      w(pages.size(2));
    }
    w.tensor(o);
    w(r.array(a[8], at::kFloat, {B, H, Tq}));
    scratch(r, a[9], w);
    w(stream_of(r));
  });
}

// append(k_new, v_new, k_cache, v_cache, slots, bounds or None)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(APPEND, n, 6, [&](const Reader& r, Words& w) {
    const at::Tensor &kn = r.view(a[0], 3), &vn = r.view(a[1], 3), &k = r.view(a[2], 4),
                     &v = r.view(a[3], 4);
    const int64_t rows = kn.size(0), Hkv = k.size(1), D = k.size(3);
    if (kn.size(1) != Hkv || kn.size(2) != D || vn.sizes() != kn.sizes() ||
        v.sizes() != k.sizes())
      throw Odd{};
    w.rows(kn);
    w.rows(vn);
    for (int64_t x : {rows, Hkv, D, k.size(0), k.size(2)}) w(x);
    w(r.array(a[4], at::kLong, {rows}));
    w.tensor(k);
    w.tensor(v);
    w(a[5] == Py_None ? 0 : r.array(a[5], at::kBFloat16, {k.size(0), Hkv, 2, D}));
    w(stream_of(r));
  });
}

// plan(new_tokens, lengths, block_table, free_ring, ring_state, page_size, n_slots,
//      lengths_out, ring_state_out, cu_new, slots, positions, status)
PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(PLAN, n, 13, [&](const Reader& r, Words& w) {
    const int64_t B = r(a[0]).numel(), n_pages = r(a[3]).numel(), n_slots = number(a[6]);
    int64_t ptr, stride, width;
    table(r, a[2], B, &ptr, &stride, &width);
    w(r.array(a[0], at::kInt, {B}));
    w(r.array(a[1], at::kInt, {B}));
    w(ptr);
    w(stride);
    w(r.array(a[3], at::kInt, {n_pages}));
    w(r.array(a[4], at::kLong, {2}));
    for (int64_t x : {B, width, n_pages, number(a[5]), n_slots}) w(x);
    w(r.array(a[7], at::kInt, {B}));
    w(r.array(a[8], at::kLong, {2}));
    w(r.array(a[9], at::kInt, {B + 1}));
    w(r.array(a[10], at::kLong, {n_slots}));
    w(r.array(a[11], at::kInt, {n_slots}));
    w(r.array(a[12], at::kInt, {1}));
    w(stream_of(r));
  });
}

// select(q, bounds, block_table, lengths, page_size, n_select, n_first, n_last, pages, workspace)
PyObject* select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(SELECT, n, 10, [&](const Reader& r, Words& w) {
    const at::Tensor &q = r.view(a[0], 4), &bounds = r.view(a[1], 4);
    const int64_t B = q.size(0), H = q.size(1), Tq = q.size(2), D = q.size(3);
    const int64_t n_pages = bounds.size(0), Hkv = bounds.size(1), K = number(a[5]);
    w.tensor(q);
    w(r.array(a[1], at::kBFloat16, {n_pages, Hkv, 2, D}));
    for (int64_t x : {B, H, Hkv, Tq, D, n_pages, number(a[4])}) w(x);
    int64_t ptr, stride, width;
    table(r, a[2], B, &ptr, &stride, &width);
    w(ptr);
    w(stride);
    w(width);
    w(r.array(a[3], at::kInt, {B}));
    for (int64_t x : {K, number(a[6]), number(a[7])}) w(x);
    w(r.array(a[8], at::kInt, {B, Hkv, K}));
    scratch(r, a[9], w);
    w(stream_of(r));
  });
}

// use(address of attn_paged_call)
PyObject* use(PyObject*, PyObject* address) {
  const unsigned long long p = PyLong_AsUnsignedLongLong(address);
  if (PyErr_Occurred()) return nullptr;
  g_call = reinterpret_cast<Call>(static_cast<uintptr_t>(p));
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"use", use, METH_O, nullptr},
                         {"decode", fast(decode), METH_FASTCALL, nullptr},
                         {"append", fast(append), METH_FASTCALL, nullptr},
                         {"plan", fast(plan), METH_FASTCALL, nullptr},
                         {"select", fast(select), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods,
                      nullptr,               nullptr,        nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__torch_calls(void) {
  return PyModule_Create(&module);
}
