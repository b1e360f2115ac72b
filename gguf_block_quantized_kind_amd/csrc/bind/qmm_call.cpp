// qmm_call.cpp -- the operators that a decode step calls once per layer, on torch
// tensors: checks of the operands, sizes from their shapes, allocation of
// outputs, and the C entry point on the operands' device and its current
// stream.  In C++ because the host's time is what a small step waits for: the
// same in Python, with the C call made through ctypes, took 2 to 4 us more a
// call (one token's rotation 6.3 us, of which the kernel's launch takes 2.7).
//
// setup(addresses, check, cache_kind_id, layout_id, kind_id, act_id, score_id) sets
// the library's functions and what raises for a status or an unknown name.  Every
// function takes its arguments by position (the package's functions of the same
// names carry the defaults).  The interpreter lock is released during the C call.
#define PY_SSIZE_T_CLEAN
#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
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
  X(qmm_kv_page_bytes) X(qmm_rmsnorm) X(qmm_rmsnorm_q8) X(qmm_gemv_q8) X(qmm_moe_route) X(qmm_matmul_ep)             \
  X(qmm_matmul_packed_ep) X(qmm_matmul_ep_workspace_bytes) X(qmm_kind_from_name) X(qmm_row_bytes) X(qmm_packed_bytes)
#define DECLARE(fn) decltype(&::fn) p_##fn = nullptr;
EACH_FUNCTION(DECLARE)
#undef DECLARE
PyObject *g_check, *g_cache_kind_id, *g_layout_id, *g_kind_id, *g_act_id, *g_score_id;

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
// Whether someone looks at new tensors: a mode that watches or replaces torch's
// operators, or torch's filling of new memory.
bool watched() {
  return c10::impl::dispatch_mode_enabled() ||
         (at::globalContext().deterministicAlgorithms() && at::globalContext().deterministicFillUninitializedMemory());
}
// A tensor beside `like`, which is on a GPU (0.13 us less each than through the dispatcher,
// where nobody looks).
at::Tensor make(const at::Tensor &like, at::IntArrayRef shape, at::ScalarType t) {
  if (watched()) {
    at::Tensor made = at::empty(shape, at::TensorOptions().dtype(t).device(like.device()));
    if (made.device() != like.device() || made.scalar_type() != t || made.sizes() != shape || !made.is_contiguous())
      raise(PyExc_TypeError, "a new tensor of ", shape, " ", t, " on ", like.device(), " came back as ", made.sizes(), " ",
            made.scalar_type(), " on ", made.device());
    return made;
  }
  return at::Tensor(at::detail::empty_cuda(shape, t, like.device(), std::nullopt));
}

// Tensors that are used together in one allocation, each at a multiple of 256 bytes
// (0.2 us less a tensor than one each; one each where someone looks).
template <int N>
void make_together(at::Tensor (&t)[N], const at::Tensor &like, const at::IntArrayRef (&shapes)[N],
                   const at::ScalarType (&types)[N]) {
  int64_t at_byte[N], bytes = 0;
  for (int i = 0; i < N; ++i) {
    int64_t n = (int64_t)c10::elementSize(types[i]);
    for (const int64_t size : shapes[i]) {
      if (size < 0 || (size > 0 && n > INT64_MAX / 4 / size)) raise(PyExc_ValueError, "no tensor is of ", shapes[i]);
      n *= size;
    }
    at_byte[i] = bytes;
    bytes += (n + 255) / 256 * 256;
  }
  if (watched()) {
    for (int i = 0; i < N; ++i) t[i] = make(like, shapes[i], types[i]);
    return;
  }
  const at::Tensor all = make(like, {bytes}, at::kByte);
  for (int i = 0; i < N; ++i) {
    t[i] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(),
                                                    c10::scalarTypeToTypeMeta(types[i]));
    c10::TensorImpl *const impl = t[i].unsafeGetTensorImpl();
    impl->set_storage_offset(at_byte[i] / (int64_t)c10::elementSize(types[i]));
    impl->set_sizes_contiguous(shapes[i]);
  }
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

int weight_kind(PyObject *o) {
  if (PyUnicode_Check(o)) {
    const char *name = PyUnicode_AsUTF8(o);
    if (!name) throw Raised{};
    const int id = p_qmm_kind_from_name(name);
    if (id >= 0) return id;
  }
  return call_id(g_kind_id, o);
}
int act_of(PyObject *o) {
  return o == Py_None || is(o, "none") ? QMM_ACT_NONE
         : is(o, "silu")               ? QMM_ACT_SILU
         : is(o, "gelu")               ? QMM_ACT_GELU
         : is(o, "gelu_tanh")          ? QMM_ACT_GELU_TANH
         : is(o, "relu")               ? QMM_ACT_RELU
                                       : call_id(g_act_id, o);
}

// [T, D] rows, or [T, heads, D] as rows_of.
Rows any_rows_of(const at::Tensor &x, const char *what) {
  if (x.dim() != 2) return rows_of(x, what);
  const int64_t T = x.size(0), D = x.size(1);
  if (D > 1 && x.stride(1) != 1) raise(PyExc_ValueError, "the rows of ", what, " must be packed, got strides ", x.strides());
  return Rows{T, 1, D, T > 1 ? x.stride(0) : D};
}
const float *floats_of(const at::Tensor &t, int64_t count, const char *what) {
  if (t.scalar_type() != at::kFloat) raise(PyExc_TypeError, what, " must be float32, got ", t.scalar_type());
  if (t.numel() != count || !t.is_contiguous())
    raise(PyExc_ValueError, what, " must hold ", count, " contiguous elements, got ", t.sizes());
  return (const float *)t.data_ptr();
}
void same_shape(const at::Tensor &t, const at::Tensor &like, const char *what) {
  if (t.sizes() != like.sizes()) raise(PyExc_ValueError, what, " is ", t.sizes(), ", needs ", like.sizes());
}

// A norm's operands besides its result: x, weight, residual, sum_out.
struct NormIn {
  const at::Tensor &x;
  Rows r;
  const float *weight = nullptr;
  float eps;
  at::Tensor residual, sum;  // undefined without a residual
  int64_t residual_stride = 0, sum_stride = 0;
  PyObject *sum_given = nullptr;
  at::Device device;
  NormIn(PyObject *px, PyObject *pw, PyObject *pe, PyObject *pr, PyObject *ps)
      : x(tensor(px, "x")), r(any_rows_of(x, "x")), eps((float)number(pe)), device(one_gpu({&x})) {
    if (pw != Py_None) {
      const at::Tensor &w = tensor(pw, "weight");
      weight = floats_of(w, r.D, "weight");
      one_gpu({&x, &w});
    }
    if (pr == Py_None) {
      if (ps != Py_None) raise(PyExc_ValueError, "sum_out without a residual");
      return;
    }
    residual = tensor(pr, "residual");
    same_shape(residual, x, "residual");
    residual_stride = any_rows_of(residual, "residual").stride;
    one_gpu({&x, &residual});
    if (ps != Py_None) {
      sum_given = ps;
      sum = tensor(ps, "sum_out");
      same_shape(sum, x, "sum_out");
      if (sum.scalar_type() != residual.scalar_type())
        raise(PyExc_TypeError, "sum_out is ", sum.scalar_type(), ", the residual is ", residual.scalar_type());
      sum_stride = any_rows_of(sum, "sum_out").stride;
      one_gpu({&x, &sum});
    } else {
      sum = make(x, x.sizes(), residual.scalar_type());
      sum_stride = r.H * r.D;
    }
  }
  const void *res() const { return residual.defined() ? residual.data_ptr() : nullptr; }
  int res_code() const { return residual.defined() ? code(residual.scalar_type()) : QMM_F32; }
  void *sum_ptr() const { return sum.defined() ? sum.data_ptr() : nullptr; }
  // `y` (a new reference), and the sum with it where there is a residual.
  PyObject *with_sum(PyObject *y) {
    if (!y || !sum.defined()) return y;
    PyObject *s = sum_given ? Py_NewRef(sum_given) : THPVariable_Wrap(std::move(sum));
    PyObject *both = s ? PyTuple_Pack(2, y, s) : nullptr;
    Py_DECREF(y);
    Py_XDECREF(s);
    return both;
  }
};

// x, weight, eps, residual, out, out_dtype, sum_out
PyObject *rmsnorm(PyObject *const *a) {
  check_out_type(a[4], a[5], "out");
  NormIn in(a[0], a[1], a[2], a[3], a[6]);
  at::Tensor y;
  int64_t stride = in.r.H * in.r.D;
  if (a[4] != Py_None) {
    y = tensor(a[4], "out");
    same_shape(y, in.x, "out");
    stride = any_rows_of(y, "out").stride;
    one_gpu({&in.x, &y});
  } else {
    y = make(in.x, in.x.sizes(), a[5] == Py_None ? in.x.scalar_type() : type_of(a[5]));
  }
  call(in.device, p_qmm_rmsnorm, (const void *)in.x.data_ptr(), code(in.x.scalar_type()), in.r.stride, in.res(),
       in.res_code(), in.residual_stride, in.weight, in.eps, in.sum_ptr(), in.sum_stride, y.data_ptr(),
       code(y.scalar_type()), stride, in.r.T, in.r.H, in.r.D);
  return in.with_sum(a[4] != Py_None ? Py_NewRef(a[4]) : THPVariable_Wrap(std::move(y)));
}

// kind, x, weight, eps, residual, codes, scales, code_sums, sum_out
PyObject *rmsnorm_q8(PyObject *const *a) {
  const int kind = weight_kind(a[0]);
  NormIn in(a[1], a[2], a[3], a[4], a[8]);
  if (in.x.dim() != 2) raise(PyExc_ValueError, "x must be [rows, elements], got ", in.x.sizes());
  const int64_t T = in.r.T, D = in.r.D, shape[2] = {T, D}, blocks[2] = {T, D / 32};
  at::Tensor t[3];
  const char *names[3] = {"codes", "scales", "code_sums"};
  const at::ScalarType types[3] = {at::kChar, at::kFloat, at::kInt};
  const bool given = a[5] != Py_None;
  const at::IntArrayRef want[3] = {shape, blocks, blocks};
  if (!given) make_together(t, in.x, want, types);
  for (int i = 0; given && i < 3; ++i) {
    t[i] = tensor(a[5 + i], names[i]);
    if (t[i].scalar_type() != types[i] || t[i].sizes() != want[i] || !t[i].is_contiguous())
      raise(PyExc_ValueError, names[i], " must be contiguous ", types[i], " ", want[i], ", got ", t[i].scalar_type(), " ",
            t[i].sizes());
    one_gpu({&in.x, &t[i]});
  }
  call(in.device, p_qmm_rmsnorm_q8, kind, (const void *)in.x.data_ptr(), code(in.x.scalar_type()), in.r.stride, in.res(),
       in.res_code(), in.residual_stride, in.weight, in.eps, in.sum_ptr(), in.sum_stride, (int8_t *)t[0].data_ptr(),
       (float *)t[1].data_ptr(), (int32_t *)t[2].data_ptr(), T, D);
  PyObject *o[3], *acts = nullptr;
  for (int i = 0; i < 3; ++i) o[i] = given ? Py_NewRef(a[5 + i]) : THPVariable_Wrap(std::move(t[i]));
  if (o[0] && o[1] && o[2]) acts = PyTuple_Pack(3, o[0], o[1], o[2]);
  for (int i = 0; i < 3; ++i) Py_XDECREF(o[i]);
  return in.with_sum(acts);
}

// A product's epilogue and result: bias, act, mul, residual, out, out_dtype.
struct Ep {
  qmm_epilogue e{};
  at::Tensor out;
  PyObject *given;
  int64_t stride;
  Ep(PyObject *const *a, const at::Tensor &x, int64_t M, int64_t N) : given(a[4] == Py_None ? nullptr : a[4]), stride(N) {
    const int64_t shape[2] = {M, N};
    e.act = act_of(a[1]);
    if (a[0] != Py_None) {
      const at::Tensor &b = tensor(a[0], "bias");
      e.bias = floats_of(b, N, "bias");
      one_gpu({&x, &b});
    }
    auto rows = [&](PyObject *o, const char *what, int &type, int64_t &stride) -> const at::Tensor & {
      const at::Tensor &t = tensor(o, what);
      if (t.sizes() != at::IntArrayRef(shape)) raise(PyExc_ValueError, what, " is ", t.sizes(), ", needs ", at::IntArrayRef(shape));
      one_gpu({&x, &t});
      type = code(t.scalar_type());
      stride = any_rows_of(t, what).stride;
      return t;
    };
    if (a[2] != Py_None) e.mul = rows(a[2], "mul", e.mul_dtype, e.mul_stride).data_ptr();
    if (a[3] != Py_None) e.residual = rows(a[3], "residual", e.residual_dtype, e.residual_stride).data_ptr();
    check_out_type(a[4], a[5], "out");
    int type;
    if (given) {
      out = rows(given, "out", type, stride);
    } else {
      if (N < 0) raise(PyExc_ValueError, "N=", N, " is not a size");
      out = make(x, shape, a[5] == Py_None ? at::kFloat : type_of(a[5]));
    }
  }
  PyObject *result() { return given ? Py_NewRef(given) : THPVariable_Wrap(std::move(out)); }
};
void bytes_of(const at::Tensor &t, int64_t need, const char *what) {
  if (t.element_size() != 1) raise(PyExc_TypeError, what, " must be a byte tensor, got ", t.scalar_type());
  if (!t.is_contiguous() || t.numel() < need)
    raise(PyExc_ValueError, what, " holds ", t.numel(), " bytes (contiguous: ", t.is_contiguous(), "), needs ", need);
}

// A workspace of `bytes` (0: none is used): `o`, or one made for the call.
struct Workspace {
  at::Tensor t;
  size_t bytes = 0;
  Workspace(PyObject *o, const at::Tensor &like, size_t need) {
    if (o != Py_None) {
      t = tensor(o, "workspace");
      if (!t.is_contiguous()) raise(PyExc_ValueError, "workspace must be contiguous");
      one_gpu({&like, &t});
      bytes = t.nbytes();
    } else if (need) {
      t = make(like, {(int64_t)need}, at::kByte);
      bytes = need;
    }
  }
  void *ptr() const { return t.defined() ? t.data_ptr() : nullptr; }
};

// kind, W, A, N, bias, act, mul, residual, out, out_dtype, workspace
template <bool PACKED>
PyObject *matmul_with(PyObject *const *a) {
  const int kind = weight_kind(a[0]);
  const at::Tensor &W = tensor(a[1], PACKED ? "P" : "W"), &A = tensor(a[2], "A");
  if ((A.dim() != 1 && A.dim() != 2) || !A.is_contiguous())
    raise(PyExc_ValueError, "A must be contiguous [M, K] or [K], got ", A.sizes());
  const int64_t K = A.size(A.dim() - 1), M = A.dim() == 1 ? 1 : A.size(0);
  const int64_t rb = PACKED ? 0 : p_qmm_row_bytes(kind, K);
  // (Without N, rows of a kind or length that the library refuses count as one.)
  const int64_t N = a[3] != Py_None ? integer(a[3]) : rb > 0 ? W.numel() / rb : 1;
  const int64_t need = PACKED ? p_qmm_packed_bytes(kind, N, K) : rb > 0 && N > 0 && N <= INT32_MAX ? rb * N : 0;
  bytes_of(W, need, PACKED ? "P" : "W");
  const at::Device d = one_gpu({&A, &W});
  Ep ep(a + 4, A, M, N);
  const int type = code(A.scalar_type());
  size_t bytes = 0;
  if (a[10] == Py_None && M > QMM_GEMV_MAX_M) {
    const c10::DeviceGuard guard(d);
    bytes = p_qmm_matmul_ep_workspace_bytes(kind, PACKED, M, N, K, type);
  }
  const Workspace work(a[10], A, bytes);
  call(d, PACKED ? p_qmm_matmul_packed_ep : p_qmm_matmul_ep, kind, (const void *)W.data_ptr(), (const void *)A.data_ptr(),
       type, (const qmm_epilogue *)&ep.e, ep.out.data_ptr(), code(ep.out.scalar_type()), ep.stride, M, N, K, work.ptr(),
       work.bytes);
  return ep.result();
}
PyObject *matmul_ep(PyObject *const *a) { return matmul_with<false>(a); }
PyObject *matmul_packed_ep(PyObject *const *a) { return matmul_with<true>(a); }

// kind, P, codes, scales, code_sums, N, bias, act, mul, residual, out, out_dtype
PyObject *gemv_q8(PyObject *const *a) {
  const int kind = weight_kind(a[0]);
  const at::Tensor &P = tensor(a[1], "P"), &q = tensor(a[2], "codes"), &d = tensor(a[3], "scales"), &s = tensor(a[4], "code_sums");
  if (q.dim() != 2 || !q.is_contiguous() || q.scalar_type() != at::kChar)
    raise(PyExc_ValueError, "codes must be contiguous int8 [M, K], got ", q.scalar_type(), " ", q.sizes());
  const int64_t M = q.size(0), K = q.size(1), N = integer(a[5]);
  const float *scales = floats_of(d, M * (K / 32), "scales");
  const int32_t *sums = ints_of(s, M * (K / 32), "code_sums");
  bytes_of(P, p_qmm_packed_bytes(kind, N, K), "P");
  const at::Device dev = one_gpu({&q, &P, &d, &s});
  Ep ep(a + 6, q, M, N);
  call(dev, p_qmm_gemv_q8, kind, (const void *)P.data_ptr(), (const int8_t *)q.data_ptr(), scales, sums,
       (const qmm_epilogue *)&ep.e, ep.out.data_ptr(), code(ep.out.scalar_type()), ep.stride, M, N, K);
  return ep.result();
}

// logits, topk, score, bias, n_group, topk_group, group_top, normalize, scale, slots, ids, weights
PyObject *moe_route(PyObject *const *a) {
  const at::Tensor &x = tensor(a[0], "logits");
  if (x.dim() != 2) raise(PyExc_ValueError, "logits must be [tokens, experts], got ", x.sizes());
  const Rows r = any_rows_of(x, "logits");
  const int64_t M = r.T, E = r.D, k = integer(a[1]);
  const int score = is(a[2], "softmax")   ? QMM_ROUTE_SOFTMAX
                    : is(a[2], "sigmoid") ? QMM_ROUTE_SIGMOID
                                          : call_id(g_score_id, a[2]);
  const int64_t n_group = integer(a[4]), topk_group = integer(a[5]), top = integer(a[6]);
  const int normalize = PyObject_IsTrue(a[7]);
  if (normalize < 0) throw Raised{};
  const float scale = (float)number(a[8]);
  const at::Device d = one_gpu({&x});
  const float *bias = nullptr;
  if (a[3] != Py_None) {
    const at::Tensor &b = tensor(a[3], "bias");
    bias = floats_of(b, E, "bias");
    one_gpu({&x, &b});
  }
  const int32_t *slots = nullptr;
  if (a[9] != Py_None) {
    const at::Tensor &s = tensor(a[9], "slots");
    slots = ints_of(s, M, "slots");
    one_gpu({&x, &s});
  }
  const bool given = a[10] != Py_None;
  if (given != (a[11] != Py_None)) raise(PyExc_ValueError, "ids and weights go together");
  const int64_t shape[2] = {M, k};
  at::Tensor ids, w;
  if (given) {
    ids = tensor(a[10], "ids"), w = tensor(a[11], "weights");
    for (const at::Tensor *t : {&ids, &w})
      if (t->sizes() != at::IntArrayRef(shape)) raise(PyExc_ValueError, "ids and weights must be ", at::IntArrayRef(shape));
    ints_of(ids, M * k, "ids");
    floats_of(w, M * k, "weights");
    one_gpu({&x, &ids, &w});
  } else {
    if (k < 0) raise(PyExc_ValueError, "topk=", k, " is not a size");
    at::Tensor t[2];
    make_together(t, x, {at::IntArrayRef(shape), at::IntArrayRef(shape)}, {at::kInt, at::kFloat});
    ids = std::move(t[0]), w = std::move(t[1]);
  }
  call(d, p_qmm_moe_route, (const void *)x.data_ptr(), code(x.scalar_type()), r.stride, bias, M, E, k, score, n_group,
       topk_group, (int)std::max<int64_t>(std::min<int64_t>(top, 3), 0), normalize, scale, slots, (int32_t *)ids.data_ptr(),
       (float *)w.data_ptr());
  if (given) return PyTuple_Pack(2, a[10], a[11]);
  PyObject *io = THPVariable_Wrap(std::move(ids)), *wo = THPVariable_Wrap(std::move(w));
  PyObject *both = io && wo ? PyTuple_Pack(2, io, wo) : nullptr;
  Py_XDECREF(io);
  Py_XDECREF(wo);
  return both;
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
  PyObject *addresses, *check, *cache_kind, *layout, *kind, *act, *score;
  if (!PyArg_ParseTuple(args, "O!OOOOOO", &PyDict_Type, &addresses, &check, &cache_kind, &layout, &kind, &act, &score))
    return nullptr;
#define SET(fn)                                                                             \
  {                                                                                         \
    PyObject *o = PyDict_GetItemString(addresses, #fn);                                     \
    if (!o) return PyErr_Format(PyExc_ValueError, "no address of " #fn);                    \
    p_##fn = (decltype(p_##fn))PyLong_AsVoidPtr(o);                                         \
    if (!p_##fn) return PyErr_Format(PyExc_ValueError, "the address of " #fn " is no address"); \
  }
  EACH_FUNCTION(SET)
#undef SET
  g_check = Py_NewRef(check), g_cache_kind_id = Py_NewRef(cache_kind), g_layout_id = Py_NewRef(layout);
  g_kind_id = Py_NewRef(kind), g_act_id = Py_NewRef(act), g_score_id = Py_NewRef(score);
  Py_RETURN_NONE;
}

#define METHOD(fn, n) {#fn, (PyCFunction)(void (*)(void))entry<fn, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(rope, 7),     METHOD(kv_write, 8),     METHOD(kv_append, 15),
                         METHOD(kv_read, 11), METHOD(attn_decode, 14), METHOD(rmsnorm, 7),
                         METHOD(rmsnorm_q8, 9), METHOD(gemv_q8, 12),   METHOD(moe_route, 12),
                         METHOD(matmul_ep, 11), METHOD(matmul_packed_ep, 11), {"setup", setup, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qmm_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qmm_call(void) { return PyModule_Create(&module); }
