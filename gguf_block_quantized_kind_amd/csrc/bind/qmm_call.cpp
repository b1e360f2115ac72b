// qmm_call.cpp -- the operators that a decode step calls once per layer, on torch
// tensors: checks of the operands, sizes from their shapes, allocation of
// outputs, and the C entry point on the operands' device and its current
// stream.  In C++ because the host's time is what a small step waits for: the
// same in Python, with the C call made through ctypes, took 2 to 4 us more a
// call (one token's rotation 6.3 us, of which the kernel's launch takes 2.7).
//
// setup(addresses, check, cache_kind_id, layout_id) sets the library's functions
// and what raises for a status or an unknown name.  Every function takes its
// arguments by position (the package's functions of the same names carry the
// defaults).  The interpreter lock is released during the C call.
#define PY_SSIZE_T_CLEAN
#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <sstream>

#include "../../../include/qmm.h"

namespace {

// The library's functions, by their header's types.
#define EACH_FUNCTION(X) \
  X(qmm_rope) X(qmm_kv_write) X(qmm_kv_append) X(qmm_kv_read) X(qmm_attn_decode) X(qmm_attn_decode_workspace_bytes) \
  X(qmm_kv_page_bytes)
#define DECLARE(fn) decltype(&::fn) p_##fn = nullptr;
EACH_FUNCTION(DECLARE)
#undef DECLARE
PyObject *g_check, *g_cache_kind_id, *g_layout_id;

struct Raised {};  // a Python exception is set

template <typename... A>
[[noreturn]] void raise(PyObject *type, const A &...a) {
  std::ostringstream s;
  (s << ... << a);
  PyErr_SetString(type, s.str().c_str());
  throw Raised{};
}

const at::Tensor &tensor(PyObject *o, const char *what) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, what, " must be a torch tensor, got ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}
int64_t integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}
int call_id(PyObject *fn, PyObject *o) {
  PyObject *r = PyObject_CallOneArg(fn, o);
  if (!r) throw Raised{};
  const long v = PyLong_AsLong(r);
  Py_DECREF(r);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return (int)v;
}
bool is(PyObject *o, const char *name) { return PyUnicode_Check(o) && PyUnicode_CompareWithASCIIString(o, name) == 0; }
int cache_kind(PyObject *o) {
  return is(o, "Q8_0") ? QMM_Q8_0 : is(o, "Q4_0") ? QMM_Q4_0 : is(o, "F16") ? QMM_CACHE_F16 : call_id(g_cache_kind_id, o);
}
int layout_of(PyObject *o) {
  return is(o, "half") ? QMM_ROPE_HALF : is(o, "interleaved") ? QMM_ROPE_INTERLEAVED : call_id(g_layout_id, o);
}
at::ScalarType type_of(PyObject *o) {
  if (!THPDtype_Check(o)) raise(PyExc_TypeError, "a torch dtype is needed, got ", Py_TYPE(o)->tp_name);
  return reinterpret_cast<THPDtype *>(o)->scalar_type;
}
int code(at::ScalarType t) {
  return t == at::kFloat ? QMM_F32 : t == at::kHalf ? QMM_F16 : 99;  // 99: refused by the library as a bad dtype
}

// T, heads, head_dim and row stride of [T, heads, head_dim] rows.
struct Rows {
  int64_t T, H, D, stride;
};
Rows rows_of(const at::Tensor &x, const char *what) {
  if (x.dim() != 3) raise(PyExc_ValueError, what, " must be [rows, heads, head_dim], got ", x.sizes());
  const int64_t T = x.size(0), H = x.size(1), D = x.size(2);
  if ((D > 1 && x.stride(2) != 1) || (H > 1 && x.stride(1) != D))
    raise(PyExc_ValueError, "the heads of a row of ", what, " must be packed, got strides ", x.strides());
  return Rows{T, H, D, T > 1 ? x.stride(0) : H * D};
}
const int32_t *ints_of(const at::Tensor &t, int64_t count, const char *what) {
  if (t.scalar_type() != at::kInt) raise(PyExc_TypeError, what, " must be int32, got ", t.scalar_type());
  if (t.numel() != count || !t.is_contiguous())
    raise(PyExc_ValueError, what, " must hold ", count, " contiguous elements, got ", t.sizes());
  return (const int32_t *)t.data_ptr();
}
int64_t check_pages(const at::Tensor &p, int kind, int64_t page_size, int64_t n_kv, int64_t D, const char *what) {
  if (p.dim() != 2 || p.element_size() != 1 || !p.is_contiguous())
    raise(PyExc_TypeError, what, " must be a contiguous byte tensor [n_pages, page_bytes]");
  const int64_t bytes = p_qmm_kv_page_bytes(kind, page_size, n_kv, D);
  if (bytes > 0 && p.size(1) != bytes)
    raise(PyExc_ValueError, what, " has pages of ", p.size(1), " bytes, page_size=", page_size, ", n_kv=", n_kv,
          " and head_dim=", D, " need ", bytes);
  return p.size(0);
}
struct Cache {
  int k_kind, v_kind;
  void *k, *v;
  int64_t n, page_size, n_kv, D;
};
Cache cache_of(const at::Tensor &kp, const at::Tensor &vp, PyObject *k_kind, PyObject *v_kind, PyObject *page, int64_t n_kv,
               int64_t D) {
  Cache c{cache_kind(k_kind), cache_kind(v_kind), nullptr, nullptr, 0, integer(page), n_kv, D};
  c.n = check_pages(kp, c.k_kind, c.page_size, n_kv, D, "k_pages");
  if (check_pages(vp, c.v_kind, c.page_size, n_kv, D, "v_pages") != c.n)
    raise(PyExc_ValueError, "k_pages holds ", c.n, " pages, v_pages ", vp.size(0));
  c.k = kp.data_ptr(), c.v = vp.data_ptr();
  return c;
}
const double *freqs_of(const at::Tensor &f, int64_t &n_rot) {
  if (f.scalar_type() != at::kDouble || f.dim() != 1 || !f.is_contiguous())
    raise(PyExc_TypeError, "freqs must be a contiguous float64 vector, got ", f.scalar_type(), " ", f.sizes());
  n_rot = 2 * f.numel();
  return (const double *)f.data_ptr();
}
// The operands' device: one GPU.
at::Device one_gpu(std::initializer_list<const at::Tensor *> ts) {
  const at::Device d = (*ts.begin())->device();
  for (const at::Tensor *t : ts)
    if (!t->is_cuda() || t->device() != d)
      raise(PyExc_ValueError, "operands must be on one GPU, got ", t->device(), " with ", d);
  return d;
}
// A type asked for beside a tensor to write into has to be that tensor's.
void check_out_type(PyObject *out, PyObject *dtype, const char *what) {
  if (out != Py_None && dtype != Py_None && tensor(out, what).scalar_type() != type_of(dtype))
    raise(PyExc_TypeError, what, " is ", tensor(out, what).scalar_type(), ", the type asked for is ", type_of(dtype));
}
at::Tensor make(const at::Tensor &like, at::IntArrayRef shape, at::ScalarType t) {
  return at::empty(shape, at::TensorOptions().dtype(t).device(like.device()));
}

// Calls fn(args..., the device's current stream) with that device current.
template <typename F, typename... A>
void call(at::Device d, F fn, A... args) {
  int status;
  {
    const c10::DeviceGuard guard(d);
    void *s = (void *)c10::hip::getCurrentHIPStream(d.index()).stream();
    Py_BEGIN_ALLOW_THREADS;
    status = fn(args..., s);
    Py_END_ALLOW_THREADS;
  }
  if (status == QMM_OK) return;
  PyObject *r = PyObject_CallFunction(g_check, "i", status);  // raises
  Py_XDECREF(r);
  if (r) PyErr_Format(PyExc_RuntimeError, "status %d", status);
  throw Raised{};
}

// q_out or y: `o` (its object returned again) or a tensor made for the call.
struct Out {
  at::Tensor t;
  PyObject *given;
  int64_t stride;
  Out(PyObject *o, PyObject *dtype, const at::Tensor &like, const Rows &r) : given(o == Py_None ? nullptr : o) {
    if (given) {
      t = tensor(o, "out");
      const Rows w = rows_of(t, "out");
      if (w.T != r.T || w.H != r.H || w.D != r.D) raise(PyExc_ValueError, "out is ", t.sizes(), ", needs ", like.sizes());
      one_gpu({&like, &t});
      stride = w.stride;
    } else {
      t = make(like, {r.T, r.H, r.D}, dtype == Py_None ? like.scalar_type() : type_of(dtype));
      stride = r.H * r.D;
    }
  }
  PyObject *result() { return given ? Py_NewRef(given) : THPVariable_Wrap(std::move(t)); }
};

// x, positions, freqs, layout, mscale, out, out_dtype
PyObject *rope(PyObject *const *a) {
  const at::Tensor &x = tensor(a[0], "x"), &pos = tensor(a[1], "positions"), &freqs = tensor(a[2], "freqs");
  const Rows r = rows_of(x, "x");
  const int32_t *p = ints_of(pos, r.T, "positions");
  int64_t n_rot;
  const double *f = freqs_of(freqs, n_rot);
  const int layout = layout_of(a[3]);
  const float mscale = (float)number(a[4]);
  check_out_type(a[5], a[6], "out");
  const at::Device d = one_gpu({&x, &pos, &freqs});
  Out out(a[5], a[6], x, r);
  call(d, p_qmm_rope, f, n_rot, layout, mscale, p, (const void *)x.data_ptr(), code(x.scalar_type()), r.stride,
       out.t.data_ptr(), code(out.t.scalar_type()), out.stride, r.T, r.H, r.D);
  return out.result();
}

struct Tokens {
  Rows k, v;
  const int32_t *slots;
};
Tokens tokens_of(const at::Tensor &k, const at::Tensor &v, const at::Tensor &slots) {
  const Rows kr = rows_of(k, "k"), vr = rows_of(v, "v");
  if (kr.T != vr.T || kr.H != vr.H || kr.D != vr.D) raise(PyExc_ValueError, "k is ", k.sizes(), ", v is ", v.sizes());
  if (k.scalar_type() != v.scalar_type()) raise(PyExc_TypeError, "k is ", k.scalar_type(), ", v is ", v.scalar_type());
  return Tokens{kr, vr, ints_of(slots, kr.T, "slots")};
}

// k, v, slots, k_pages, v_pages, k_kind, v_kind, page_size
PyObject *kv_write(PyObject *const *a) {
  const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &slots = tensor(a[2], "slots"),
                   &kp = tensor(a[3], "k_pages"), &vp = tensor(a[4], "v_pages");
  const Tokens t = tokens_of(k, v, slots);
  const Cache c = cache_of(kp, vp, a[5], a[6], a[7], t.k.H, t.k.D);
  call(one_gpu({&k, &v, &slots, &kp, &vp}), p_qmm_kv_write, c.k_kind, c.v_kind, c.k, c.v, c.n, c.page_size, c.n_kv, c.D,
       (const void *)k.data_ptr(), t.k.stride, (const void *)v.data_ptr(), t.v.stride, code(k.scalar_type()), t.slots,
       t.k.T);
  Py_RETURN_NONE;
}

// q, k, v, positions, slots, k_pages, v_pages, k_kind, v_kind, page_size, freqs, layout, mscale, out, out_dtype
PyObject *kv_append(PyObject *const *a) {
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &pos = tensor(a[3], "positions"),
                   &slots = tensor(a[4], "slots"), &kp = tensor(a[5], "k_pages"), &vp = tensor(a[6], "v_pages"),
                   &freqs = tensor(a[10], "freqs");
  const Tokens t = tokens_of(k, v, slots);
  const Rows r = rows_of(q, "q");
  if (r.T != t.k.T || r.D != t.k.D) raise(PyExc_ValueError, "q is ", q.sizes(), ", k is ", k.sizes());
  if (q.scalar_type() != k.scalar_type()) raise(PyExc_TypeError, "q is ", q.scalar_type(), ", k is ", k.scalar_type());
  const int32_t *p = ints_of(pos, r.T, "positions");
  const Cache c = cache_of(kp, vp, a[7], a[8], a[9], t.k.H, t.k.D);
  int64_t n_rot;
  const double *f = freqs_of(freqs, n_rot);
  const int layout = layout_of(a[11]);
  const float mscale = (float)number(a[12]);
  check_out_type(a[13], a[14], "out");
  const at::Device d = one_gpu({&q, &k, &v, &pos, &slots, &kp, &vp, &freqs});
  Out out(a[13], a[14], q, r);
  call(d, p_qmm_kv_append, f, n_rot, layout, mscale, p, (const void *)q.data_ptr(), r.stride, r.H, out.t.data_ptr(),
       code(out.t.scalar_type()), out.stride, c.k_kind, c.v_kind, c.k, c.v, c.n, c.page_size, c.n_kv, c.D,
       (const void *)k.data_ptr(), t.k.stride, (const void *)v.data_ptr(), t.v.stride, code(k.scalar_type()), t.slots, r.T);
  return out.result();
}

// slots, k_pages, v_pages, k_kind, v_kind, page_size, n_kv, head_dim, dtype, k_out, v_out
PyObject *kv_read(PyObject *const *a) {
  const at::Tensor &slots = tensor(a[0], "slots"), &kp = tensor(a[1], "k_pages"), &vp = tensor(a[2], "v_pages");
  const int64_t T = slots.numel(), H = integer(a[6]), D = integer(a[7]);
  const int32_t *s = ints_of(slots, T, "slots");
  const Cache c = cache_of(kp, vp, a[3], a[4], a[5], H, D);
  check_out_type(a[9], a[8], "k_out");
  const at::Device d = one_gpu({&slots, &kp, &vp});
  const bool given = a[9] != Py_None;
  if (given != (a[10] != Py_None)) raise(PyExc_ValueError, "k_out and v_out go together");
  at::Tensor k, v;
  const int64_t shape[3] = {T, H, D};
  if (given) {
    k = tensor(a[9], "k_out"), v = tensor(a[10], "v_out");
    for (const at::Tensor *t : {&k, &v})
      if (t->sizes() != at::IntArrayRef(shape) || !t->is_contiguous() || t->scalar_type() != k.scalar_type())
        raise(PyExc_ValueError, "k_out and v_out must be contiguous ", at::IntArrayRef(shape), " of one type");
    one_gpu({&slots, &k, &v});
  } else {
    if (H < 0 || D < 0) raise(PyExc_ValueError, "n_kv=", H, " and head_dim=", D, " are not sizes");
    const at::ScalarType type = a[8] == Py_None ? at::kHalf : type_of(a[8]);
    k = make(slots, shape, type), v = make(slots, shape, type);
  }
  call(d, p_qmm_kv_read, c.k_kind, c.v_kind, (const void *)c.k, (const void *)c.v, c.n, c.page_size, c.n_kv, c.D, s, T,
       k.data_ptr(), v.data_ptr(), code(k.scalar_type()));
  if (given) return PyTuple_Pack(2, a[9], a[10]);
  PyObject *ko = THPVariable_Wrap(std::move(k)), *vo = THPVariable_Wrap(std::move(v));
  PyObject *both = ko && vo ? PyTuple_Pack(2, ko, vo) : nullptr;
  Py_XDECREF(ko);
  Py_XDECREF(vo);
  return both;
}

// q, k_pages, v_pages, block_table, seq_lens, k_kind, v_kind, page_size, n_kv, scale, window, sinks, out, workspace
PyObject *attn_decode(PyObject *const *a) {
  const at::Tensor &q = tensor(a[0], "q"), &kp = tensor(a[1], "k_pages"), &vp = tensor(a[2], "v_pages"),
                   &table = tensor(a[3], "block_table"), &lens = tensor(a[4], "seq_lens");
  const Rows r = rows_of(q, "q");
  const int32_t *l = ints_of(lens, r.T, "seq_lens");
  if (table.dim() != 2 || table.size(0) != r.T)
    raise(PyExc_ValueError, "block_table must be [", r.T, ", max_pages], got ", table.sizes());
  const int64_t max_pages = table.size(1);
  const int32_t *pages = ints_of(table, r.T * max_pages, "block_table");
  const Cache c = cache_of(kp, vp, a[5], a[6], a[7], integer(a[8]), r.D);
  const float scale = (float)(a[9] == Py_None ? std::pow((double)r.D, -0.5) : number(a[9]));
  const int64_t window = integer(a[10]);
  const at::Device d = one_gpu({&q, &kp, &vp, &table, &lens});
  const float *sinks = nullptr;
  if (a[11] != Py_None) {
    const at::Tensor &s = tensor(a[11], "sinks");
    if (s.scalar_type() != at::kFloat || !s.is_contiguous() || s.numel() != r.H)
      raise(PyExc_ValueError, "sinks must be ", r.H, " contiguous float32 values");
    one_gpu({&q, &s});
    sinks = (const float *)s.data_ptr();
  }
  at::Tensor out, work;
  const int64_t shape[3] = {r.T, r.H, r.D};
  if (a[12] != Py_None) {
    out = tensor(a[12], "out");
    if (out.sizes() != at::IntArrayRef(shape) || !out.is_contiguous() || out.scalar_type() != q.scalar_type())
      raise(PyExc_ValueError, "out must be contiguous ", at::IntArrayRef(shape), " of q's type");
    one_gpu({&q, &out});
  } else {
    out = make(q, shape, q.scalar_type());
  }
  size_t bytes;
  if (a[13] != Py_None) {
    work = tensor(a[13], "workspace");
    if (!work.is_contiguous()) raise(PyExc_ValueError, "workspace must be contiguous");
    one_gpu({&q, &work});
    bytes = work.nbytes();
  } else {
    bytes = p_qmm_attn_decode_workspace_bytes(r.T, r.H, c.n_kv, r.D);
    work = make(q, {(int64_t)std::max(bytes, (size_t)1)}, at::kByte);
  }
  call(d, p_qmm_attn_decode, c.k_kind, c.v_kind, (const void *)c.k, (const void *)c.v, c.n, c.page_size, c.n_kv, c.D,
       (const void *)q.data_ptr(), code(q.scalar_type()), r.stride, r.H, pages, max_pages, l, r.T, scale, window, sinks,
       out.data_ptr(), work.data_ptr(), bytes);
  return a[12] != Py_None ? Py_NewRef(a[12]) : THPVariable_Wrap(std::move(out));
}

template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) return PyErr_Format(PyExc_TypeError, "%d arguments are needed, got %zd", N, n);
  if (!g_check) return PyErr_Format(PyExc_RuntimeError, "setup() has not been called");
  try {
    return F(a);
  } catch (const Raised &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject *setup(PyObject *, PyObject *args) {
  PyObject *addresses, *check, *kind, *layout;
  if (!PyArg_ParseTuple(args, "O!OOO", &PyDict_Type, &addresses, &check, &kind, &layout)) return nullptr;
#define SET(fn)                                                                             \
  {                                                                                         \
    PyObject *o = PyDict_GetItemString(addresses, #fn);                                     \
    if (!o) return PyErr_Format(PyExc_ValueError, "no address of " #fn);                    \
    p_##fn = (decltype(p_##fn))PyLong_AsVoidPtr(o);                                         \
    if (!p_##fn) return PyErr_Format(PyExc_ValueError, "the address of " #fn " is no address"); \
  }
  EACH_FUNCTION(SET)
#undef SET
  g_check = Py_NewRef(check), g_cache_kind_id = Py_NewRef(kind), g_layout_id = Py_NewRef(layout);
  Py_RETURN_NONE;
}

#define METHOD(fn, n) {#fn, (PyCFunction)(void (*)(void))entry<fn, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(rope, 7),     METHOD(kv_write, 8),     METHOD(kv_append, 15),
                         METHOD(kv_read, 11), METHOD(attn_decode, 14), {"setup", setup, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qmm_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qmm_call(void) { return PyModule_Create(&module); }
