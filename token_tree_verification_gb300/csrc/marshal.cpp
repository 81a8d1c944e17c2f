// The binding's work on the host for the paged calls, in C++: the checks of the
// tensors, the output and the call of the C ABI, for arguments as they should
// be.  Anything else (a wrong type or shape, an error code, a stream of its own)
// returns None and is left to binding.py, which defines what happens then; so does
// a build without this module.  On a Grace core binding.py's checks take 4 to 7 us a
// call and ctypes 80 ns an argument, beside 2.5 us for the launch.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/Context.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>

#include "../../include/spec_tree.h"

namespace {

// Addresses of the C ABI in the library that binding.py has loaded.
decltype(&spec_rope) call_rope = nullptr;
decltype(&spec_rope_write_paged) call_write = nullptr;
decltype(&spec_tree_attn_paged) call_attn = nullptr;
decltype(&spec_kv_compact_paged) call_compact = nullptr;

constexpr int64_t kIntMax = 0x7FFFFFFF;

struct Unfit {};      // left to binding.py

inline void need(bool fits) {
  if (!fits) throw Unfit();
}

inline const at::Tensor &tensor(PyObject *o) {
  need(THPVariable_Check(o));
  return THPVariable_Unpack(o);
}

// A call's device (the current one), type and stream.
struct Call {
  c10::DeviceIndex device;
  at::ScalarType type;
  int dtype;

  explicit Call(const at::Tensor &t) : device(c10::cuda::current_device()), type(t.scalar_type()) {
    need(type == at::kBFloat16 || type == at::kFloat);
    dtype = type == at::kFloat ? SPEC_F32 : SPEC_BF16;
    need(at(t));
  }
  bool at(const at::Tensor &t) const { return t.is_cuda() && t.get_device() == device; }
  void *stream() const { return c10::cuda::getCurrentCUDAStream(device).stream(); }
  int32_t *i32(const at::Tensor &t, int64_t n) const {
    need(at(t) && t.scalar_type() == at::kInt && t.numel() == n && t.is_contiguous());
    return static_cast<int32_t *>(t.data_ptr());
  }
  int32_t *i32(PyObject *o, int64_t n) const { return i32(tensor(o), n); }
  int32_t *i32_or_null(PyObject *o, int64_t n) const { return o == Py_None ? nullptr : i32(o, n); }
  // Rows [T][heads][D] at any stride but in a head.
  const at::Tensor &rows(PyObject *o, int64_t T, int64_t heads, int64_t D) const {
    const at::Tensor &t = tensor(o);
    need(at(t) && t.scalar_type() == type && t.dim() == 3 && t.size(0) == T && t.size(1) == heads && t.size(2) == D &&
         t.stride(2) == 1 && T <= kIntMax && heads <= kIntMax);
    return t;
  }
  at::Tensor empty(at::IntArrayRef sizes, at::IntArrayRef strides, at::ScalarType as) const {
    need(!at::globalContext().deterministicAlgorithms());      // (torch then fills new tensors)
    return at::detail::empty_strided_cuda(sizes, strides, as, c10::Device(c10::kCUDA, device));
  }
};

struct Pool {
  void *k, *v;
  int32_t *table;
  int pages, heads, size, D, width;

  Pool(const Call &c, const at::Tensor &kp, PyObject *v_pages, PyObject *block_table, int64_t B) {
    const at::Tensor &vp = tensor(v_pages), &t = tensor(block_table);
    need(kp.dim() == 4 && c.at(vp) && vp.scalar_type() == c.type && vp.sizes() == kp.sizes() && kp.is_contiguous() &&
         vp.is_contiguous());
    need(t.dim() == 2 && t.size(0) == B && t.size(1) <= kIntMax && kp.size(0) <= kIntMax && kp.size(1) <= kIntMax &&
         kp.size(2) <= kIntMax && kp.size(3) <= kIntMax);
    table = c.i32(t, t.numel());
    k = kp.data_ptr();
    v = vp.data_ptr();
    pages = static_cast<int>(kp.size(0));
    heads = static_cast<int>(kp.size(1));
    size = static_cast<int>(kp.size(2));
    D = static_cast<int>(kp.size(3));
    width = static_cast<int>(t.size(1));
  }
};

// A rotation: the frequencies' tensor, the factor and the rotated dims; None rotates nothing.
struct Rotation {
  const uint64_t *freqs = nullptr;
  float scale = 1.f;
  int r = 0;

  Rotation(const Call &c, PyObject *table) {
    if (table == Py_None) return;
    need(PyTuple_Check(table) && PyTuple_GET_SIZE(table) == 3);
    const at::Tensor &f = tensor(PyTuple_GET_ITEM(table, 0));
    PyObject *s = PyTuple_GET_ITEM(table, 1), *n = PyTuple_GET_ITEM(table, 2);
    need(PyFloat_Check(s) && PyLong_Check(n));
    scale = static_cast<float>(PyFloat_AS_DOUBLE(s));
    const long dims = PyLong_AsLong(n);
    need(dims >= 0 && dims <= 512);
    r = static_cast<int>(dims);
    need(c.at(f) && f.scalar_type() == at::kLong && 2 * f.numel() == r && f.is_contiguous());
    freqs = static_cast<const uint64_t *>(f.data_ptr());
  }
};

int truth(PyObject *o) {
  const int t = PyObject_IsTrue(o);
  need(t >= 0);
  return t;
}

// Runs `work`, which returns the call's code; whatever does not fit becomes None.
template <typename Work>
PyObject *run(Work work) {
  try {
    return work();
  } catch (const Unfit &) {
  } catch (const std::exception &) {
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

template <typename Launch>
void launch(Launch call) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = call();
  Py_END_ALLOW_THREADS
  need(rc == SPEC_OK);
}

PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run([&]() -> PyObject * {      // x, table, start, offsets, status, depth, interleaved
    need(n == 7 && call_rope);
    const at::Tensor &x = tensor(a[0]), &status = tensor(a[4]);
    const Call c(x);
    need(x.dim() == 3);
    c.rows(a[0], x.size(0), x.size(1), x.size(2));
    const int64_t B = status.numel(), T = x.size(0), H = x.size(1), D = x.size(2);
    need(B >= 1 && B < kIntMax && D <= kIntMax);
    const Rotation rot(c, a[1]);
    int32_t *start = c.i32(a[2], B), *offsets = c.i32(a[3], B + 1), *codes = c.i32(status, B),
            *depth = c.i32_or_null(a[5], T);
    const int interleaved = truth(a[6]);
    at::Tensor y = c.empty({T, H, D}, {H * D, D, 1}, c.type);
    const void *xp = x.data_ptr();
    void *yp = y.data_ptr();
    const int64_t st = x.stride(0), sh = x.stride(1);
    void *stream = c.stream();
    launch([&] {
      return call_rope(xp, yp, c.dtype, static_cast<int>(B), static_cast<int>(T), static_cast<int>(H), static_cast<int>(D),
                       st, sh, H * D, D, rot.freqs, rot.r, rot.scale, interleaved, start, depth, offsets, codes, stream);
    });
    return THPVariable_Wrap(std::move(y));
  });
}

PyObject *rope_write_paged(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run([&]() -> PyObject * {      // q, k, v, k_pages, v_pages, block_table, prefix_lens, offsets, status, table,
                                        // depth, start, interleaved
    need(n == 13 && call_write);
    const at::Tensor &kp = tensor(a[3]), &status = tensor(a[8]), &q = tensor(a[0]);
    const Call c(kp);
    const int64_t B = status.numel();
    need(B >= 1 && B < kIntMax && q.dim() == 3);
    const Pool p(c, kp, a[4], a[5], B);
    const int64_t T = q.size(0), Hq = q.size(1), D = p.D;
    need(Hq >= 1);
    c.rows(a[0], T, Hq, D);
    const at::Tensor &k = c.rows(a[1], T, p.heads, D), &v = c.rows(a[2], T, p.heads, D);
    const Rotation rot(c, a[9]);
    int32_t *prefix = c.i32(a[6], B), *offsets = c.i32(a[7], B + 1), *codes = c.i32(status, B),
            *depth = c.i32_or_null(a[10], T), *start = c.i32_or_null(a[11], B);
    const int interleaved = truth(a[12]);
    at::Tensor y = c.empty({T, Hq, D}, {Hq * D, D, 1}, c.type);
    const void *qp = q.data_ptr(), *kr = k.data_ptr(), *vr = v.data_ptr();
    void *yp = y.data_ptr(), *stream = c.stream();
    launch([&] {
      return call_write(qp, yp, kr, vr, c.dtype, static_cast<int>(B), static_cast<int>(T), static_cast<int>(Hq), p.heads,
                        p.D, q.stride(0), q.stride(1), k.stride(0), k.stride(1), v.stride(0), v.stride(1), rot.freqs,
                        rot.r, rot.scale, interleaved, p.k, p.v, p.pages, p.size, p.table, p.width, prefix, start, depth,
                        offsets, codes, stream);
    });
    return THPVariable_Wrap(std::move(y));
  });
}

PyObject *tree_attn_paged(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run([&]() -> PyObject * {      // q, k_pages, v_pages, block_table, prefix_lens, offsets, mask, max_prefix, status,
                                        // softmax_scale, parents, causal
    need(n == 12 && call_attn);
    const at::Tensor &q = tensor(a[0]), &kp = tensor(a[1]), &status = tensor(a[8]);
    const Call c(kp);
    const int64_t B = status.numel();
    need(B >= 1 && B < kIntMax);
    const Pool p(c, kp, a[2], a[3], B);
    need(q.dim() == 3 && c.at(q) && q.scalar_type() == c.type && q.size(2) == p.D && q.is_contiguous() &&
         q.size(0) <= kIntMax && q.size(1) <= kIntMax);
    const int64_t T = q.size(0), Hq = q.size(1), D = p.D;
    const int causal = truth(a[11]);
    need(causal ? a[6] == Py_None && a[10] == Py_None : a[6] != Py_None || a[10] != Py_None);
    const int32_t *mask = a[6] == Py_None ? nullptr : c.i32(a[6], 4 * T),
                  *parents = mask ? nullptr : c.i32_or_null(a[10], T);
    int overflow = 0;
    need(PyLong_Check(a[7]));
    const long long bound = PyLong_AsLongLongAndOverflow(a[7], &overflow);
    need(overflow == 0);
    const double scale = PyFloat_AsDouble(a[9]);
    need(!(scale == -1.0 && PyErr_Occurred()));
    int32_t *prefix = c.i32(a[4], B), *offsets = c.i32(a[5], B + 1), *codes = c.i32(status, B);
    at::Tensor o = c.empty({T, Hq, D}, {Hq * D, D, 1}, c.type);
    const void *qp = q.data_ptr();
    void *op = o.data_ptr(), *stream = c.stream();
    const int max_prefix = static_cast<int>(bound < -1 ? -1 : bound < kIntMax ? bound : kIntMax);
    launch([&] {
      return call_attn(qp, p.k, p.v, op, c.dtype, static_cast<int>(B), static_cast<int>(T), static_cast<int>(Hq), p.heads,
                       p.D, p.pages, p.size, p.table, p.width, max_prefix, prefix, offsets,
                       reinterpret_cast<const uint32_t *>(mask), parents, causal, static_cast<float>(scale), codes,
                       stream);
    });
    return THPVariable_Wrap(std::move(o));
  });
}

PyObject *kv_compact_paged(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run([&]() -> PyObject * {      // k_pages, v_pages, block_table, prefix_lens, offsets, path_nodes, accept_len, status
    need(n == 8 && call_compact);
    const at::Tensor &kp = tensor(a[0]), &path = tensor(a[5]), &status = tensor(a[7]);
    const Call c(kp);
    const int64_t B = status.numel();
    need(B >= 1 && B < kIntMax && path.dim() >= 1);
    const Pool p(c, kp, a[1], a[2], B);
    const int64_t W = path.size(-1);
    need(W <= kIntMax);
    int32_t *prefix = c.i32(a[3], B), *offsets = c.i32(a[4], B + 1), *nodes = c.i32(path, B * W), *accept = c.i32(a[6], B),
            *codes = c.i32(status, B);
    at::Tensor lens = c.empty({B}, {1}, at::kInt);
    int32_t *out = static_cast<int32_t *>(lens.data_ptr());
    void *stream = c.stream();
    launch([&] {
      return call_compact(p.k, p.v, c.dtype, static_cast<int>(B), p.heads, p.D, p.pages, p.size, p.table, p.width, prefix,
                          offsets, nodes, accept, static_cast<int>(W), out, codes, stream);
    });
    return THPVariable_Wrap(std::move(lens));
  });
}

// bind(rope, write, attn, compact): the functions' addresses.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "four addresses");
    return nullptr;
  }
  void *f[4];
  for (int i = 0; i < 4; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (!f[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is null");
      return nullptr;
    }
  }
  std::memcpy(&call_rope, &f[0], sizeof(void *));
  std::memcpy(&call_write, &f[1], sizeof(void *));
  std::memcpy(&call_attn, &f[2], sizeof(void *));
  std::memcpy(&call_compact, &f[3], sizeof(void *));
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind), FAST(rope), FAST(rope_write_paged), FAST(tree_attn_paged), FAST(kv_compact_paged),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
