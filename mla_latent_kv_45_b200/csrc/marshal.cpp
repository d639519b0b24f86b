// The prompt calls' argument checks and pointers in C++, for _lib.py.
//
// A small call takes a few microseconds on the GPU, and looking at ten tensors from
// Python takes longer than that: a call of the attention, the append and the gather
// kept the host 13.4, 12.2 and 8.3 us from Python and keeps it 4.0, 4.0 and 3.2 us from
// here.  These functions look at the same things (type, shape, strides, device, address)
// in the tensors themselves and call the library on the given stream or the device's
// current one.  They decline whatever is not exactly as it should be by returning None;
// _lib.py then goes through its own checks, which say what is wrong.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cstring>
#include <initializer_list>

#include "mla.h"

namespace {

decltype(&mla_prompt_append) call_append = nullptr;
decltype(&mla_cache_gather) call_gather = nullptr;
decltype(&mla_prompt_attn) call_attn = nullptr;

// The tensor behind a Python object (borrowed), or nullptr.
const at::Tensor *tensor(PyObject *o) {
  return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}

// Strided, of this type and shape (-1: any size that an int holds), on CUDA device dev,
// the last axis (dense: all of it) contiguous.
bool is(const at::Tensor *t, at::ScalarType type, int dev, std::initializer_list<int64_t> shape,
        bool dense) {
  if (!t || !t->defined() || !t->is_cuda() || t->get_device() != dev ||
      t->layout() != at::kStrided || t->scalar_type() != type ||
      t->dim() != (int64_t)shape.size())
    return false;
  const auto sizes = t->sizes(), strides = t->strides();
  int i = 0;
  for (const int64_t want : shape) {
    if (sizes[i] > INT32_MAX || (want >= 0 && sizes[i] != want)) return false;
    ++i;
  }
  return dense ? t->is_contiguous() : sizes[i - 1] <= 1 || strides[i - 1] == 1;
}

mla_heads heads(const at::Tensor *t) { return {t->data_ptr(), t->stride(0), t->stride(1)}; }

const int32_t *ints(const at::Tensor *t) {
  return t ? static_cast<const int32_t *>(t->data_ptr()) : nullptr;
}

bool dims_of(PyObject *o, mla_dims *d) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE)) return false;
  const bool ok = b.len == (Py_ssize_t)sizeof(mla_dims);
  if (ok) std::memcpy(d, b.buf, sizeof(mla_dims));
  PyBuffer_Release(&b);
  return ok;
}

at::ScalarType type_of(const mla_dims &d) { return d.dtype == MLA_BF16 ? at::kBFloat16 : at::kFloat; }

bool cache_of(const mla_dims &d, PyObject *pool, PyObject *table, int dev, int64_t batch,
              mla_paged_cache *c) {
  const bool int8 = d.cache_format == MLA_CACHE_INT8;
  const at::Tensor *p = tensor(pool), *t = tensor(table);
  if (!is(p, int8 ? at::kByte : type_of(d), dev,
          {-1, d.page_size, int8 ? (int64_t)MLA_INT8_ROW_BYTES : (int64_t)d.d_c + d.d_rope}, true) ||
      !is(t, at::kInt, dev, {batch, -1}, true))
    return false;
  *c = {p->data_ptr(), (int)p->size(0), ints(t), (int)t->size(1), nullptr};
  return true;
}

// A workspace of any type.
bool ws_of(PyObject *o, int dev, void **ptr, size_t *bytes) {
  const at::Tensor *t = tensor(o);
  if (!t || !t->defined() || !t->is_cuda() || t->get_device() != dev || !t->is_contiguous())
    return false;
  *ptr = t->data_ptr();
  *bytes = t->nbytes();
  return true;
}

// The stream to launch on: `o` is None (the device's current one) or a CUDA stream's
// address, which _lib.py gives for a stream of device dev.  False where dev is not the
// current device.
bool stream_of(PyObject *o, int dev, mla_stream_t *s) {
  if (dev < 0 || c10::cuda::current_device() != dev) return false;
  if (o == Py_None) {
    *s = (mla_stream_t)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    return true;
  }
  const unsigned long long v = PyLong_AsUnsignedLongLong(o);
  if (PyErr_Occurred()) return false;
  *s = (mla_stream_t)(uintptr_t)v;
  return true;
}

PyObject *decline() {
  PyErr_Clear();
  Py_RETURN_NONE;
}

// The interpreter's lock is given up while this lives, and is back before an exception of the
// library is caught.
class Unlocked {
 public:
  Unlocked() : state_(PyEval_SaveThread()) {}
  ~Unlocked() { PyEval_RestoreThread(state_); }
  Unlocked(const Unlocked &) = delete;
  Unlocked &operator=(const Unlocked &) = delete;

 private:
  PyThreadState *state_;
};

// No C++ exception leaves a call from Python.
template <class F>
PyObject *guarded(F &&f) {
  try {
    return f();
  } catch (...) {
    return decline();
  }
}

// append(dims, pool, table, x, gamma, cu, ctx, q, q_out, ws, stream)
PyObject *py_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    mla_dims d;
    if (n != 11 || !call_append || !dims_of(a[0], &d)) return decline();
    const at::Tensor *x = tensor(a[3]), *gamma = tensor(a[4]), *cu = tensor(a[5]);
    const at::Tensor *ctx = a[6] == Py_None ? nullptr : tensor(a[6]);
    if (!x || !x->defined() || !x->is_cuda() || !cu || !cu->defined() || cu->dim() != 1)
      return decline();
    const int dev = x->get_device();
    const int64_t batch = cu->size(0) - 1;
    const auto dt = type_of(d), xt = x->scalar_type();
    if ((xt != at::kFloat && xt != dt) || !is(x, xt, dev, {-1, (int64_t)d.d_c + d.d_rope}, false) ||
        !is(gamma, dt, dev, {d.d_c}, true) || !is(cu, at::kInt, dev, {-1}, true) ||
        (a[6] != Py_None && !is(ctx, at::kInt, dev, {batch}, true)))
      return decline();
    const int64_t tokens = x->size(0);
    const bool with_q = a[7] != Py_None;
    mla_heads q{}, qo{};
    if (with_q != (a[8] != Py_None)) return decline();
    if (with_q) {
      const at::Tensor *t = tensor(a[7]), *o = tensor(a[8]);
      if (!is(t, dt, dev, {tokens, d.n_heads, d.d_rope}, false) ||
          !is(o, dt, dev, {tokens, d.n_heads, d.d_rope}, false))
        return decline();
      q = heads(t);
      qo = heads(o);
    }
    mla_paged_cache c;
    void *ws;
    size_t bytes;
    mla_stream_t s;
    if (!cache_of(d, a[1], a[2], dev, batch, &c) || !ws_of(a[9], dev, &ws, &bytes) ||
        !stream_of(a[10], dev, &s))
      return decline();
    const int xd = xt == at::kFloat ? MLA_FP32 : MLA_BF16;
    const void *xp = x->data_ptr(), *gp = gamma->data_ptr();
    const int64_t xs = x->stride(0);
    const int32_t *cup = ints(cu), *ctxp = ints(ctx);
    mla_status st;
    {
      Unlocked unlocked;
      st = call_append(&d, &c, (int)batch, (int)tokens, xp, xd, xs, gp, cup, ctxp,
                       with_q ? &q : nullptr, with_q ? &qo : nullptr, ws, bytes, s);
    }
    return PyLong_FromLong(st);
  });
}

// gather(dims, pool, table, cu, first, rows, ws, stream)
PyObject *py_gather(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    mla_dims d;
    if (n != 8 || !call_gather || !dims_of(a[0], &d)) return decline();
    const at::Tensor *cu = tensor(a[3]), *rows = tensor(a[5]);
    const at::Tensor *first = a[4] == Py_None ? nullptr : tensor(a[4]);
    if (!rows || !rows->defined() || !rows->is_cuda() || !cu || !cu->defined() || cu->dim() != 1)
      return decline();
    const int dev = rows->get_device();
    const int64_t batch = cu->size(0) - 1;
    mla_paged_cache c;
    void *ws;
    size_t bytes;
    mla_stream_t s;
    if (!is(rows, type_of(d), dev, {-1, (int64_t)d.d_c + d.d_rope}, true) ||
        !is(cu, at::kInt, dev, {-1}, true) ||
        (a[4] != Py_None && !is(first, at::kInt, dev, {batch}, true)) ||
        !cache_of(d, a[1], a[2], dev, batch, &c) || !ws_of(a[6], dev, &ws, &bytes) ||
        !stream_of(a[7], dev, &s))
      return decline();
    const int n_rows = (int)rows->size(0);
    const int32_t *cup = ints(cu), *fp = ints(first);
    void *rp = rows->data_ptr();
    mla_status st;
    {
      Unlocked unlocked;
      st = call_gather(&d, &c, (int)batch, n_rows, cup, fp, rp, ws, bytes, s);
    }
    return PyLong_FromLong(st);
  });
}

// attn(dims, q_nope, q_rope, k_nope, k_rope, v, cu_q, cu_k, out, lse, ws, stream)
PyObject *py_attn(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    mla_dims d;
    if (n != 12 || !call_attn || !dims_of(a[0], &d)) return decline();
    const at::Tensor *qn = tensor(a[1]), *qr = tensor(a[2]), *kn = tensor(a[3]),
                     *kr = tensor(a[4]), *v = tensor(a[5]), *cu_q = tensor(a[6]),
                     *cu_k = tensor(a[7]), *out = tensor(a[8]);
    const at::Tensor *lse = a[9] == Py_None ? nullptr : tensor(a[9]);
    if (!qn || !qn->defined() || !qn->is_cuda() || !cu_q || !cu_q->defined() || cu_q->dim() != 1)
      return decline();
    const int dev = qn->get_device();
    const auto dt = type_of(d);
    if (!is(qn, dt, dev, {-1, d.n_heads, d.d_nope}, false) ||
        !is(kn, dt, dev, {-1, -1, d.d_nope}, false))
      return decline();
    const int64_t n_q = qn->size(0), n_k = kn->size(0), kv = kn->size(1), off = cu_q->size(0);
    void *ws;
    size_t bytes;
    mla_stream_t s;
    if (!is(qr, dt, dev, {n_q, d.n_heads, d.d_rope}, false) ||
        !is(kr, dt, dev, {n_k, d.d_rope}, false) || !is(v, dt, dev, {n_k, kv, d.d_v}, false) ||
        !is(cu_q, at::kInt, dev, {-1}, true) || !is(cu_k, at::kInt, dev, {off}, true) ||
        !is(out, dt, dev, {n_q, d.n_heads, d.d_v}, true) ||
        (a[9] != Py_None && !is(lse, at::kFloat, dev, {n_q, d.n_heads}, true)) ||
        !ws_of(a[10], dev, &ws, &bytes) || !stream_of(a[11], dev, &s))
      return decline();
    const mla_heads hq = heads(qn), hr = heads(qr), hk = heads(kn), hv = heads(v);
    const void *krp = kr->data_ptr();
    const int64_t krs = kr->stride(0);
    const int32_t *cqp = ints(cu_q), *ckp = ints(cu_k);
    void *op = out->data_ptr();
    float *lp = lse ? static_cast<float *>(lse->data_ptr()) : nullptr;
    mla_status st;
    {
      Unlocked unlocked;
      st = call_attn(&d, (int)(off - 1), (int)n_q, (int)n_k, (int)kv, &hq, &hr, &hk, krp, krs, &hv,
                     cqp, ckp, op, lp, ws, bytes, s);
    }
    return PyLong_FromLong(st);
  });
}

// bind(append, gather, attn): addresses of the library's functions
PyObject *py_bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  unsigned long long p[3];
  if (n != 3) {
    PyErr_SetString(PyExc_TypeError, "bind takes three addresses");
    return nullptr;
  }
  for (int i = 0; i < 3; ++i) {
    p[i] = PyLong_AsUnsignedLongLong(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  call_append = reinterpret_cast<decltype(call_append)>((uintptr_t)p[0]);
  call_gather = reinterpret_cast<decltype(call_gather)>((uintptr_t)p[1]);
  call_attn = reinterpret_cast<decltype(call_attn)>((uintptr_t)p[2]);
  Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef methods[] = {{"append", fast<py_append>(), METH_FASTCALL, nullptr},
                         {"gather", fast<py_gather>(), METH_FASTCALL, nullptr},
                         {"attn", fast<py_attn>(), METH_FASTCALL, nullptr},
                         {"bind", fast<py_bind>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// The module reads tensors through the headers of the torch it was compiled against and is
// used with no other: BUILT_FOR (_lib.torch_build) is compared before bind is called.
PyMODINIT_FUNC PyInit__marshal() {
  PyObject *m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "BUILT_FOR", MLA_BUILT_FOR)) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
