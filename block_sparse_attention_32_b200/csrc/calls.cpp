// Python calls of the operators around the sparse path: argument checks and
// marshalling of torch tensors into the C ABI, in C++ because a decode step is
// shorter on the GPU than the same checks written in Python (about 30 us a call;
// 5 here).  Every function returns the msa_status and raises ValueError for
// tensors that do not fit together; nothing is kept between calls.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "../../include/msa.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Bad : std::runtime_error {
  using std::runtime_error::runtime_error;
};

const Tensor* arg(PyObject* o, const char* name, bool optional) {
  if (o == Py_None) {
    if (optional) return nullptr;
    throw Bad(std::string(name) + " is missing");
  }
  if (!THPVariable_Check(o)) throw Bad(std::string(name) + ": must be a tensor");
  return &THPVariable_Unpack(o);
}
int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Bad(std::string(name) + ": must be an integer");
  }
  return v;
}
double number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Bad(std::string(name) + ": must be a number");
  }
  return v;
}
int truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    throw Bad(std::string(name) + ": must be true or false");
  }
  return v;
}
std::string shape_of(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}
void need_shape(const char* name, const Tensor& t, at::IntArrayRef shape) {
  if (t.sizes() != shape)
    throw Bad(std::string(name) + ": shape " + shape_of(t.sizes()) + ", expected " +
              shape_of(shape));
}
void need_type(const char* name, const Tensor& t, ScalarType dt) {
  if (t.scalar_type() != dt)
    throw Bad(std::string(name) + ": " + c10::toString(t.scalar_type()) + ", expected " +
              c10::toString(dt));
}

// Collects a call's tensors: types, shapes and, at the end, that all of them live
// on the current device, whose current stream the call is enqueued on.
struct Call {
  const Tensor* seen[20];
  int n = 0;
  const Tensor* add(const Tensor* t) {
    if (t != nullptr) seen[n++] = t;
    return t;
  }
  // [B, T, H, D] rows (heads_first: the tensor itself is [B, H, T, D])
  msa_tensor rows(const char* name, PyObject* o, int64_t B, int64_t T, int64_t H, int64_t D,
                  bool heads_first = false, ScalarType dt = ScalarType::BFloat16) {
    const Tensor& t = *add(arg(o, name, false));
    const int64_t s0[4] = {B, T, H, D}, s1[4] = {B, H, T, D};
    need_shape(name, t, at::IntArrayRef(heads_first ? s1 : s0, 4));
    need_type(name, t, dt);
    if (t.stride(3) != 1)
      throw Bad(std::string(name) + ": the last dimension must be contiguous");
    return {t.const_data_ptr(), t.stride(0), t.stride(heads_first ? 2 : 1),
            t.stride(heads_first ? 1 : 2)};
  }
  // a contiguous tensor (null for None where it is optional)
  void* flat(const char* name, PyObject* o, at::IntArrayRef shape, ScalarType dt, bool optional) {
    const Tensor* t = add(arg(o, name, optional));
    if (t == nullptr) return nullptr;
    need_shape(name, *t, shape);
    need_type(name, *t, dt);
    if (!t->is_contiguous()) throw Bad(std::string(name) + ": must be contiguous");
    return t->data_ptr();
  }
  int32_t* dev_err(PyObject* o) {
    const Tensor* t = add(arg(o, "dev_err", true));
    if (t == nullptr) return nullptr;
    need_type("dev_err", *t, ScalarType::Int);
    if (t->numel() < 1) throw Bad("dev_err: must have an element");
    return static_cast<int32_t*>(t->data_ptr());
  }
  void* workspace(PyObject* o, size_t* bytes) {
    const Tensor* t = add(arg(o, "ws", false));
    if (!t->is_contiguous()) throw Bad("ws: must be contiguous");
    *bytes = t->nbytes();
    return t->data_ptr();
  }
  void* stream() const {
    for (int i = 0; i < n; ++i)
      if (!seen[i]->is_cuda()) throw Bad("every tensor must be on a CUDA device");
    const auto dev = c10::cuda::current_device();
    for (int i = 0; i < n; ++i)
      if (seen[i]->get_device() != dev)
        throw Bad("every tensor must be on the current device cuda:" + std::to_string((int)dev));
    return c10::cuda::getCurrentCUDAStream(dev).stream();
  }
};

void need_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) throw Bad("expected " + std::to_string(want) + " arguments");
}

// what the dense, paged and backward forms share
struct NormRope {
  msa_norm_rope_dims d{};
  msa_tensor q{}, k{};
  const float *w_q, *w_k, *table;
  int64_t n_pos;
  const int64_t* positions;

  NormRope(Call& c, PyObject* oq, PyObject* ok, PyObject* owq, PyObject* owk, PyObject* otab,
           PyObject* opos, PyObject* opos0, PyObject* oeps, PyObject* ointer) {
    const Tensor* tq = arg(oq, "q", true);
    const Tensor* tk = arg(ok, "k", true);
    const Tensor* some = tq != nullptr ? tq : tk;
    if (some == nullptr || some->dim() != 4) throw Bad("q or k must be given, [B, T, H, D]");
    const Tensor* tab = c.add(arg(otab, "table", true));
    if (tab != nullptr) {
      if (tab->dim() != 2 || !tab->is_contiguous())
        throw Bad("table: must be contiguous [positions, rot]");
      need_type("table", *tab, ScalarType::Float);
    }
    d.batch = some->size(0);
    d.n_tok = some->size(1);
    d.d = (int32_t)some->size(3);
    d.pos0 = integer(opos0, "pos0");
    d.eps = (float)number(oeps, "eps");
    d.interleaved = truth(ointer, "interleaved");
    d.rot = tab == nullptr ? 0 : (int32_t)tab->size(1);
    if (tq != nullptr) {
      d.h_q = (int32_t)(tq->dim() == 4 ? tq->size(2) : 0);
      q = c.rows("q", oq, d.batch, d.n_tok, d.h_q, d.d);
    }
    if (tk != nullptr) {
      d.h_k = (int32_t)(tk->dim() == 4 ? tk->size(2) : 0);
      k = c.rows("k", ok, d.batch, d.n_tok, d.h_k, d.d);
    }
    const int64_t row[1] = {d.d}, bt[2] = {d.batch, d.n_tok};
    w_q = static_cast<float*>(c.flat("w_q", owq, row, ScalarType::Float, true));
    w_k = static_cast<float*>(c.flat("w_k", owk, row, ScalarType::Float, true));
    positions =
        static_cast<int64_t*>(c.flat("positions", opos, bt, ScalarType::Long, true));
    // no rotation: every position is in range
    n_pos = tab == nullptr ? INT64_MAX : tab->size(0);
    table = tab == nullptr ? nullptr : tab->const_data_ptr<float>();
  }
};

msa_paged_kv paged(Call& c, PyObject* ok, PyObject* ov, PyObject* otable, PyObject* olens,
                   int64_t batch) {
  const Tensor& k = *c.add(arg(ok, "k_pages", false));
  const Tensor& v = *c.add(arg(ov, "v_pages", false));
  const Tensor& t = *c.add(arg(otable, "block_table", false));
  for (const Tensor* x : {&k, &v}) {
    const char* name = x == &k ? "k_pages" : "v_pages";
    if (x->dim() != 4 || x->size(3) != MSA_HEAD_DIM || x->stride(3) != 1)
      throw Bad(std::string(name) +
                ": must be [n_pages, h_kv, page_size, 128] with a contiguous last dimension");
    need_type(name, *x, ScalarType::BFloat16);
  }
  if (k.sizes() != v.sizes() || k.strides() != v.strides())
    throw Bad("k_pages and v_pages must have the same shape and strides");
  if (t.dim() != 2 || t.size(0) != batch)
    throw Bad("block_table: must be [B, pages per sequence], a row for each of the " +
              std::to_string(batch) + " sequences");
  need_type("block_table", t, ScalarType::Int);
  if (!t.is_contiguous()) throw Bad("block_table: must be contiguous");
  const int64_t b[1] = {batch};
  msa_paged_kv p{};
  p.k = k.data_ptr();
  p.v = v.data_ptr();
  p.n_pages = k.size(0);
  p.s_page = k.stride(0);
  p.s_head = k.stride(1);
  p.s_tok = k.stride(2);
  p.block_table = t.const_data_ptr<int32_t>();
  p.table_stride = t.size(1);
  p.seq_lens = olens == nullptr ? nullptr
                                : static_cast<int32_t*>(
                                      c.flat("seq_lens", olens, b, ScalarType::Int, false));
  p.page_size = (int32_t)k.size(2);
  p.h_kv = (int32_t)k.size(1);
  return p;
}

// the dims structure of capi.make_dims, read through the buffer protocol
msa_dims dims_of(PyObject* o) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) {
    PyErr_Clear();
    throw Bad("dims: must be a Dims structure");
  }
  msa_dims d;
  const bool fits = b.len == (Py_ssize_t)sizeof(d);
  if (fits) d = *static_cast<const msa_dims*>(b.buf);
  PyBuffer_Release(&b);
  if (!fits) throw Bad("dims: must be a Dims structure");
  return d;
}

template <typename F>
PyObject* guarded(F&& f) {
  try {
    return PyLong_FromLong(f());
  } catch (const Bad& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

template <typename F>
long enqueue(F&& f) {
  msa_status s;
  Py_BEGIN_ALLOW_THREADS
  s = f();
  Py_END_ALLOW_THREADS
  return s;
}

// q, k, w_q, w_k, table, q_out, k_out, positions, pos0, eps, interleaved, dev_err
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    need_args(n, 12);
    Call c;
    NormRope r(c, a[0], a[1], a[2], a[3], a[4], a[7], a[8], a[9], a[10]);
    msa_tensor qo{}, ko{};
    if (a[0] != Py_None) qo = c.rows("q_out", a[5], r.d.batch, r.d.n_tok, r.d.h_q, r.d.d);
    if (a[1] != Py_None) ko = c.rows("k_out", a[6], r.d.batch, r.d.n_tok, r.d.h_k, r.d.d, true);
    int32_t* err = c.dev_err(a[11]);
    void* st = c.stream();
    return enqueue([&] {
      return msa_qk_norm_rope(&r.d, r.q, r.k, r.w_q, r.w_k, r.table, r.n_pos, r.positions, qo, ko,
                              err, st);
    });
  });
}

// q, k, v, w_q, w_k, table, q_out, k_pages, v_pages, block_table, positions, pos0, eps,
// interleaved, dev_err
PyObject* norm_rope_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    need_args(n, 15);
    Call c;
    if (a[1] == Py_None) throw Bad("k is missing");
    NormRope r(c, a[0], a[1], a[3], a[4], a[5], a[10], a[11], a[12], a[13]);
    const msa_tensor v = c.rows("v", a[2], r.d.batch, r.d.n_tok, r.d.h_k, r.d.d);
    msa_tensor qo{};
    if (a[0] != Py_None) qo = c.rows("q_out", a[6], r.d.batch, r.d.n_tok, r.d.h_q, r.d.d);
    const msa_paged_kv cache = paged(c, a[7], a[8], a[9], nullptr, r.d.batch);
    int32_t* err = c.dev_err(a[14]);
    void* st = c.stream();
    return enqueue([&] {
      return msa_qk_norm_rope_paged(&r.d, r.q, r.k, v, r.w_q, r.w_k, r.table, r.n_pos,
                                    r.positions, qo, &cache, err, st);
    });
  });
}

// q, k, w_q, w_k, table, d_q, d_k, dx_q, dx_k, dw_q, dw_k, ws, positions, pos0, eps,
// interleaved, dev_err
PyObject* norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    need_args(n, 17);
    Call c;
    NormRope r(c, a[0], a[1], a[2], a[3], a[4], a[12], a[13], a[14], a[15]);
    const msa_norm_rope_dims& d = r.d;
    const Tensor* dy = arg(a[0] != Py_None ? a[5] : a[6], a[0] != Py_None ? "d_q" : "d_k", false);
    const ScalarType t = dy->scalar_type();
    if (t != ScalarType::BFloat16 && t != ScalarType::Float)
      throw Bad("gradients must be bf16 or fp32");
    msa_tensor dq{}, dk{}, xq{}, xk{};
    if (a[0] != Py_None) {
      dq = c.rows("d_q", a[5], d.batch, d.n_tok, d.h_q, d.d, false, t);
      xq = c.rows("dx_q", a[7], d.batch, d.n_tok, d.h_q, d.d);
    }
    if (a[1] != Py_None) {
      dk = c.rows("d_k", a[6], d.batch, d.n_tok, d.h_k, d.d, true, t);
      xk = c.rows("dx_k", a[8], d.batch, d.n_tok, d.h_k, d.d);
    }
    const int64_t row[1] = {d.d};
    float* wq = static_cast<float*>(c.flat("dw_q", a[9], row, ScalarType::Float, true));
    float* wk = static_cast<float*>(c.flat("dw_k", a[10], row, ScalarType::Float, true));
    size_t bytes;
    void* ws = c.workspace(a[11], &bytes);
    int32_t* err = c.dev_err(a[16]);
    void* st = c.stream();
    return enqueue([&] {
      return msa_qk_norm_rope_bwd(&d, r.q, r.k, r.w_q, r.w_k, r.table, r.n_pos, r.positions, dq,
                                  dk, t == ScalarType::Float ? 1 : 0, xq, xk, wq, wk, ws, bytes,
                                  err, st);
    });
  });
}

// dims, window, n_sink, q, k_pages, v_pages, block_table, seq_lens, out, lse, ws, dev_err
PyObject* paged_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    need_args(n, 12);
    Call c;
    const msa_dims d = dims_of(a[0]);
    const int64_t window = integer(a[1], "window"), sink = integer(a[2], "n_sink");
    const msa_tensor q = c.rows("q", a[3], d.batch, 1, d.h_q, MSA_HEAD_DIM);
    const msa_paged_kv cache = paged(c, a[4], a[5], a[6], a[7], d.batch);
    const int64_t qs[4] = {d.batch, 1, d.h_q, MSA_HEAD_DIM};
    void* out = c.flat("out", a[8], qs, ScalarType::BFloat16, false);
    void* lse = c.flat("lse", a[9], at::IntArrayRef(qs, 3), ScalarType::Float, false);
    size_t bytes;
    void* ws = c.workspace(a[10], &bytes);
    int32_t* err = c.dev_err(a[11]);
    void* st = c.stream();
    return enqueue([&] {
      return msa_paged_decode_attn(&d, window, sink, q, &cache, out, static_cast<float*>(lse), ws,
                                   bytes, err, st);
    });
  });
}

struct Window {
  msa_dims d;
  int64_t window, sink, qs[4], ks[4];
  msa_tensor q, k, v;
  Window(Call& c, PyObject* const* a) : d(dims_of(a[0])) {
    window = integer(a[1], "window");
    sink = integer(a[2], "n_sink");
    qs[0] = ks[0] = d.batch;
    qs[1] = d.n_q;
    qs[2] = d.h_q;
    ks[1] = d.h_kv;
    ks[2] = d.n_kv;
    qs[3] = ks[3] = MSA_HEAD_DIM;
    q = c.rows("q", a[3], d.batch, d.n_q, d.h_q, MSA_HEAD_DIM);
    k = c.rows("k", a[4], d.batch, d.n_kv, d.h_kv, MSA_HEAD_DIM, true);
    v = c.rows("v", a[5], d.batch, d.n_kv, d.h_kv, MSA_HEAD_DIM, true);
  }
  int32_t* lens(Call& c, PyObject* o) const {
    return static_cast<int32_t*>(
        c.flat("kv_len", o, at::IntArrayRef(qs, 1), ScalarType::Int, true));
  }
  float* lse(Call& c, PyObject* o) const {
    return static_cast<float*>(
        c.flat("lse", o, at::IntArrayRef(qs, 3), ScalarType::Float, false));
  }
};

// dims, window, n_sink, q, k, v, out, out_rest, lse, kv_len, dev_err
PyObject* window_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    need_args(n, 11);
    Call c;
    const Window w(c, a);
    void* out = c.flat("out", a[6], w.qs, ScalarType::BFloat16, false);
    void* rest = c.flat("out_rest", a[7], w.qs, ScalarType::Char, true);
    float* lse = w.lse(c, a[8]);
    int32_t* lens = w.lens(c, a[9]);
    int32_t* err = c.dev_err(a[10]);
    void* st = c.stream();
    return enqueue([&] {
      return msa_window_attn_fwd(&w.d, w.window, w.sink, w.q, w.k, w.v, lens, out, rest, lse, err,
                                 st);
    });
  });
}

// dims, window, n_sink, q, k, v, o, o_rest, d_o, lse, dq, dk, dv, ws, kv_len, dev_err
PyObject* window_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    need_args(n, 16);
    Call c;
    const Window w(c, a);
    const msa_tensor o = c.rows("o", a[6], w.d.batch, w.d.n_q, w.d.h_q, MSA_HEAD_DIM);
    const void* rest = c.flat("o_rest", a[7], w.qs, ScalarType::Char, true);
    const msa_tensor d_o = c.rows("d_o", a[8], w.d.batch, w.d.n_q, w.d.h_q, MSA_HEAD_DIM);
    const float* lse = w.lse(c, a[9]);
    void* dq = c.flat("dq", a[10], w.qs, ScalarType::BFloat16, false);
    void* dk = c.flat("dk", a[11], w.ks, ScalarType::BFloat16, false);
    void* dv = c.flat("dv", a[12], w.ks, ScalarType::BFloat16, false);
    size_t bytes;
    void* ws = c.workspace(a[13], &bytes);
    int32_t* lens = w.lens(c, a[14]);
    int32_t* err = c.dev_err(a[15]);
    void* st = c.stream();
    return enqueue([&] {
      return msa_window_attn_bwd(&w.d, w.window, w.sink, w.q, w.k, w.v, o, rest, d_o, lse, lens, dq,
                                 dk, dv, ws, bytes, err, st);
    });
  });
}

#define MSA_CALL(f) {#f, reinterpret_cast<PyCFunction>(f), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MSA_CALL(norm_rope),    MSA_CALL(norm_rope_paged),
                         MSA_CALL(norm_rope_bwd), MSA_CALL(paged_decode),
                         MSA_CALL(window_fwd),    MSA_CALL(window_bwd),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "msa_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch that the module was compiled for; it serves no other
PyMODINIT_FUNC PyInit_msa_calls() {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", MSA_TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
