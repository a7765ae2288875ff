// fm_python.cpp -- the Python binding's fast half: checks torch tensors and calls
// the C interface for the operators that a decode step makes one token at a time,
// where a check of ten tensors in Python takes longer than the kernel.  Holds no
// state and launches nothing itself; the Python functions of the package supply
// names, defaults and documentation.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "fluxmi.h"

namespace {

// One call: its name for messages, the current device, and whether an argument
// was refused (then a Python exception is set).
struct Call {
  const char* fn;
  int device;
  bool bad = false;

  void refuse(PyObject* type, const std::string& what) {
    if (!bad) PyErr_SetString(type, (std::string(fn) + ": " + what).c_str());
    bad = true;
  }

  // The tensor behind o, or nullptr for None.
  const at::Tensor* tensor(const char* name, PyObject* o) {
    if (o == Py_None || bad) return nullptr;
    if (!THPVariable_Check(o)) {
      refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
      return nullptr;
    }
    return &THPVariable_Unpack(o);
  }

  // Its address, if it has this type and shape, is contiguous and on the device.
  void* at(const char* name, PyObject* o, at::ScalarType type,
           std::initializer_list<int64_t> shape) {
    const at::Tensor* t = tensor(name, o);
    if (!t) return nullptr;
    if (t->scalar_type() != type || t->sizes() != at::IntArrayRef(shape)) {
      std::string want = std::string(c10::toString(type)) + " (";
      for (int64_t d : shape) want += std::to_string(d) + ",";
      std::string got = std::string(c10::toString(t->scalar_type())) + " (";
      for (int64_t d : t->sizes()) got += std::to_string(d) + ",";
      refuse(PyExc_ValueError, std::string(name) + " must be " + want + "), got " + got + ")");
      return nullptr;
    }
    if (!t->is_cuda() || t->get_device() != device) {
      refuse(PyExc_ValueError, std::string(name) + " must live on the current GPU");
      return nullptr;
    }
    if (!t->is_contiguous()) {
      refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
      return nullptr;
    }
    return t->data_ptr();
  }

  // A token mask: uint8, or bool, which holds the same bytes.
  void* mask(PyObject* o, int64_t T) {
    const at::Tensor* t = tensor("token_mask", o);
    return at("token_mask", o, t && t->scalar_type() == at::kBool ? at::kBool : at::kByte, {T});
  }

  // A workspace of any type.
  void* workspace(PyObject* o, size_t& bytes) {
    bytes = 0;
    const at::Tensor* t = tensor("ws", o);
    if (!t) return nullptr;
    if (!t->is_cuda() || t->get_device() != device || !t->is_contiguous()) {
      refuse(PyExc_ValueError, "ws must be contiguous and live on the current GPU");
      return nullptr;
    }
    bytes = t->nbytes();
    return t->data_ptr();
  }

  // The type code of a floating tensor type.
  fm_dtype_t code(at::ScalarType t) {
    if (t == at::kHalf) return FM_F16;
    if (t == at::kBFloat16) return FM_BF16;
    if (t != at::kFloat)
      refuse(PyExc_TypeError, std::string("unsupported dtype ") + c10::toString(t));
    return FM_F32;
  }

  // A scalar that the C interface takes in 32 bits.
  int32_t i32(const char* name, PyObject* o) {
    if (bad) return 0;
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) bad = true;
    else if (v != (int32_t)v)
      refuse(PyExc_ValueError, std::string(name) + " does not fit in 32 bits");
    return (int32_t)v;
  }

  // Sizes of a two-dimensional tensor that has to be there.
  const at::Tensor* matrix(const char* name, PyObject* o) {
    const at::Tensor* t = tensor(name, o);
    if (bad) return nullptr;
    if (!t || t->dim() != 2) {
      refuse(PyExc_ValueError, std::string(name) + " must be a matrix");
      return nullptr;
    }
    return t;
  }
};

// Reads the scalars among the arguments.
struct Args {
  PyObject* const* a;
  int64_t i(int k) const { return PyLong_AsLongLong(a[k]); }
  float f(int k) const { return (float)PyFloat_AsDouble(a[k]); }
  hipStream_t stream(int k) const { return (hipStream_t)PyLong_AsVoidPtr(a[k]); }
};

PyObject* done(const Call& c, fm_status_t st) {
  if (c.bad || PyErr_Occurred()) return nullptr;
  return PyLong_FromLong((long)st);
}

bool count(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  return false;
}

constexpr at::ScalarType kInt = at::kInt, kFloat = at::kFloat, kByte = at::kByte;

// device, stream, logits, topk_ids, topk_weights, score, renormalize, scale, bias,
// token_mask, counts, prob_sums, loss, ws
PyObject* moe_gate(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count(n, 14)) return nullptr;
  const Args a{v};
  Call c{"fm_moe_gate", (int)a.i(0)};
  const at::Tensor *x = c.matrix("logits", v[2]), *id = c.matrix("topk_ids", v[3]);
  if (c.bad) return nullptr;
  const int64_t T = x->size(0), E = x->size(1), topk = id->size(1);
  const at::ScalarType dt = x->scalar_type();
  const fm_dtype_t code = c.code(dt);
  const int32_t score = c.i32("score", v[5]), renorm = c.i32("renormalize", v[6]);
  size_t bytes;
  void* ws = c.workspace(v[13], bytes);
  void *px = c.at("logits", v[2], dt, {T, E}), *pid = c.at("topk_ids", v[3], kInt, {T, topk}),
       *pw = c.at("topk_weights", v[4], kFloat, {T, topk}), *pb = c.at("bias", v[8], kFloat, {E}),
       *pm = c.mask(v[9], T), *pc = c.at("counts", v[10], kInt, {E + 1}),
       *ps = c.at("prob_sums", v[11], kFloat, {E}), *pl = c.at("loss", v[12], kFloat, {1});
  const float scale = a.f(7);
  const hipStream_t stream = a.stream(1);
  if (c.bad || PyErr_Occurred()) return nullptr;
  return done(c, fm_moe_gate(code, T, (int32_t)E, (int32_t)topk, (fm_gate_score_t)score,
                             renorm, scale, px, (const float*)pb, (const uint8_t*)pm,
                             (int32_t*)pid, (float*)pw, (int32_t*)pc, (float*)ps, (float*)pl, ws,
                             bytes, stream));
}

// device, stream, logits, topk_ids, d_logits, score, renormalize, scale, token_mask,
// d_weights, counts, d_loss
PyObject* moe_gate_bwd(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count(n, 12)) return nullptr;
  const Args a{v};
  Call c{"fm_moe_gate_bwd", (int)a.i(0)};
  const at::Tensor *x = c.matrix("logits", v[2]), *id = c.matrix("topk_ids", v[3]);
  if (c.bad) return nullptr;
  const int64_t T = x->size(0), E = x->size(1), topk = id->size(1);
  const at::ScalarType dt = x->scalar_type();
  const fm_dtype_t code = c.code(dt);
  const int32_t score = c.i32("score", v[5]), renorm = c.i32("renormalize", v[6]);
  void *px = c.at("logits", v[2], dt, {T, E}), *pid = c.at("topk_ids", v[3], kInt, {T, topk}),
       *pd = c.at("d_logits", v[4], dt, {T, E}), *pm = c.mask(v[8], T),
       *pw = c.at("d_weights", v[9], kFloat, {T, topk}), *pc = c.at("counts", v[10], kInt, {E + 1}),
       *pl = c.at("d_loss", v[11], kFloat, {1});
  const float scale = a.f(7);
  const hipStream_t stream = a.stream(1);
  if (c.bad || PyErr_Occurred()) return nullptr;
  return done(c, fm_moe_gate_bwd(code, T, (int32_t)E, (int32_t)topk, (fm_gate_score_t)score,
                                 renorm, scale, px, (const uint8_t*)pm,
                                 (const int32_t*)pid, (const float*)pw, (const int32_t*)pc,
                                 (const float*)pl, pd, stream));
}

// Types of the norm's operands: dt from the 16-bit ones, the residual stream's and
// the block's from their own, each from the others where it has none.
struct NormTypes {
  at::ScalarType dt, sd, bd;
  NormTypes(Call& c, PyObject* const* v, std::initializer_list<int> small,
            std::initializer_list<int> streams, std::initializer_list<int> blocks) {
    auto first = [&](std::initializer_list<int> l, at::ScalarType& t) {
      for (int k : l)
        if (const at::Tensor* x = c.tensor("operand", v[k])) {
          t = x->scalar_type();
          return true;
        }
      return false;
    };
    const bool s = first(streams, sd), b = first(blocks, bd);
    if (!first(small, dt))
      dt = s && sd != kFloat ? sd : b && bd != kFloat ? bd : at::kBFloat16;
    if (!s) sd = dt;
    if (!b) bd = dt;
  }
};

// device, stream, out, y, block, resid, w_post, w_pre, gate, scale, eps, rstd_post,
// rstd_pre
PyObject* norm_residual(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count(n, 13)) return nullptr;
  const Args a{v};
  Call c{"fm_norm_residual", (int)a.i(0)};
  const at::Tensor* like = c.matrix("block or resid", v[4] != Py_None ? v[4] : v[5]);
  if (c.bad) return nullptr;
  const int64_t M = like->size(0), N = like->size(1);
  const NormTypes t(c, v, {3, 7, 6, 8}, {5, 2}, {4});
  const at::Tensor* gate = c.tensor("gate", v[8]);
  const int64_t G = gate && gate->dim() == 2 ? gate->size(0) : 0;
  void *pb = c.at("block", v[4], t.bd, {M, N}), *pr = c.at("resid", v[5], t.sd, {M, N}),
       *wq = c.at("w_post", v[6], t.dt, {N}), *wp = c.at("w_pre", v[7], t.dt, {N}),
       *pg = c.at("gate", v[8], t.dt, {G, N}), *po = c.at("out", v[2], t.sd, {M, N}),
       *py = c.at("y", v[3], t.dt, {M, N}), *rq = c.at("rstd_post", v[11], kFloat, {M}),
       *rp = c.at("rstd_pre", v[12], kFloat, {M});
  const fm_dtype_t dt = c.code(t.dt), sd = c.code(t.sd), bd = c.code(t.bd);
  const float scale = a.f(9), eps = a.f(10);
  const hipStream_t stream = a.stream(1);
  if (c.bad || PyErr_Occurred()) return nullptr;
  return done(c, fm_norm_residual(dt, sd, bd, M, N, pb, pr, wq, wp, pg, G, scale, eps, po, py,
                                  (float*)rq, (float*)rp, stream));
}

// device, stream, d_resid, d_block, out, block, d_y, d_out, w_post, w_pre, gate,
// scale, rstd_post, rstd_pre, d_w_post, d_w_pre, d_gate, ws
PyObject* norm_residual_bwd(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count(n, 18)) return nullptr;
  const Args a{v};
  Call c{"fm_norm_residual_bwd", (int)a.i(0)};
  const at::Tensor* like = c.matrix("d_y or d_out", v[6] != Py_None ? v[6] : v[7]);
  if (c.bad) return nullptr;
  const int64_t M = like->size(0), N = like->size(1);
  const NormTypes t(c, v, {6, 9, 8, 10}, {7, 4, 2}, {5, 3});
  const at::Tensor* gate = c.tensor("gate", v[10]);
  const int64_t G = gate && gate->dim() == 2 ? gate->size(0) : 0;
  size_t bytes;
  void* ws = c.workspace(v[17], bytes);
  void *dr = c.at("d_resid", v[2], t.sd, {M, N}), *db = c.at("d_block", v[3], t.bd, {M, N}),
       *po = c.at("out", v[4], t.sd, {M, N}), *pb = c.at("block", v[5], t.bd, {M, N}),
       *dy = c.at("d_y", v[6], t.dt, {M, N}), *dz = c.at("d_out", v[7], t.sd, {M, N}),
       *wq = c.at("w_post", v[8], t.dt, {N}), *wp = c.at("w_pre", v[9], t.dt, {N}),
       *pg = c.at("gate", v[10], t.dt, {G, N}), *rq = c.at("rstd_post", v[12], kFloat, {M}),
       *rp = c.at("rstd_pre", v[13], kFloat, {M}), *dq = c.at("d_w_post", v[14], kFloat, {N}),
       *dp = c.at("d_w_pre", v[15], kFloat, {N}), *dg = c.at("d_gate", v[16], kFloat, {G, N});
  const fm_dtype_t dt = c.code(t.dt), sd = c.code(t.sd), bd = c.code(t.bd);
  const float scale = a.f(11);
  const hipStream_t stream = a.stream(1);
  if (c.bad || PyErr_Occurred()) return nullptr;
  return done(c, fm_norm_residual_bwd(dt, sd, bd, M, N, dy, dz, po, pb, wq, wp, pg, G, scale,
                                      (const float*)rq, (const float*)rp, dr, db, (float*)dq,
                                      (float*)dp, (float*)dg, ws, bytes, stream));
}

int64_t row_bytes(int64_t K) { return (K + 127) / 128 * 64; }

int64_t groups_of(Call& c, int64_t K, int64_t group) {
  if (group != 32 && group != 64 && group != 128) {
    c.refuse(PyExc_ValueError, "group must be 32, 64 or 128");
    return 0;
  }
  return (K + group - 1) / group;
}

// device, stream, A, packed, scales, C, group, zeros
PyObject* gemm_w4(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count(n, 8)) return nullptr;
  const Args a{v};
  Call c{"fm_gemm_w4", (int)a.i(0)};
  const at::Tensor *x = c.matrix("A", v[2]), *y = c.matrix("C", v[5]);
  if (c.bad) return nullptr;
  const int64_t M = x->size(0), K = x->size(1), N = y->size(1), group = a.i(6);
  const int64_t G = groups_of(c, K, group);
  const at::ScalarType dt = x->scalar_type(), ct = y->scalar_type();
  void *px = c.at("A", v[2], dt, {M, K}), *pp = c.at("packed", v[3], kByte, {N, row_bytes(K)}),
       *ps = c.at("scales", v[4], dt, {G, N}), *py = c.at("C", v[5], ct, {M, N}),
       *pz = c.at("zeros", v[7], kByte, {G, N});
  const fm_dtype_t da = c.code(dt), dc = c.code(ct);
  const hipStream_t stream = a.stream(1);
  if (c.bad || PyErr_Occurred()) return nullptr;
  return done(c, fm_gemm_w4(da, dc, M, N, K, (int32_t)group, px, pp, ps, (const uint8_t*)pz, py,
                            stream));
}

// sorted_pairs and the rows of H: at least `pairs` of each
void check_pairs(Call& c, const at::Tensor* h, PyObject* sorted, int64_t pairs, int64_t& sp) {
  const at::Tensor* s = c.tensor("sorted_pairs", sorted);
  if (c.bad) return;
  if (!s || s->dim() != 1 || s->size(0) < pairs || h->size(0) < pairs)
    return c.refuse(PyExc_ValueError, "H or sorted_pairs is too short");
  sp = s->size(0);
}

// device, stream, X, topk_ids, packed, scales, H, sorted_pairs, expert_offsets,
// expert_begin, group, ws, zeros, act
PyObject* moe_gather_gemm_w4(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count(n, 14)) return nullptr;
  const Args a{v};
  Call c{"fm_moe_gather_gemm_w4", (int)a.i(0)};
  const at::Tensor *x = c.matrix("X", v[2]), *id = c.matrix("topk_ids", v[3]),
                   *h = c.matrix("H", v[6]), *p = c.tensor("packed", v[4]);
  if (!c.bad && (!p || p->dim() != 3)) c.refuse(PyExc_ValueError, "packed must have three dimensions");
  if (c.bad) return nullptr;
  const int64_t T = x->size(0), K = x->size(1), N = h->size(1), topk = id->size(1),
                nl = p->size(0), group = a.i(10), G = groups_of(c, K, group);
  const int32_t e0 = c.i32("expert_begin", v[9]), act = c.i32("act", v[13]);
  int64_t sp = 0;
  check_pairs(c, h, v[7], T * topk, sp);
  const at::ScalarType dt = x->scalar_type();
  const fm_dtype_t code = c.code(dt);
  size_t bytes;
  void* ws = c.workspace(v[11], bytes);
  void *px = c.at("X", v[2], dt, {T, K}), *pid = c.at("topk_ids", v[3], kInt, {T, topk}),
       *pp = c.at("packed", v[4], kByte, {nl, N, row_bytes(K)}),
       *ps = c.at("scales", v[5], dt, {nl, G, N}), *ph = c.at("H", v[6], dt, {h->size(0), N}),
       *po = c.at("sorted_pairs", v[7], kInt, {sp}),
       *pf = c.at("expert_offsets", v[8], kInt, {nl + 1}),
       *pz = c.at("zeros", v[12], kByte, {nl, G, N});
  const hipStream_t stream = a.stream(1);
  if (c.bad || PyErr_Occurred()) return nullptr;
  return done(c, fm_moe_gather_gemm_w4(code, T, K, N, (int32_t)topk, e0, (int32_t)nl,
                                       (int32_t)group, px, (const int32_t*)pid, pp, ps,
                                       (const uint8_t*)pz, ph, (int32_t*)po, (int32_t*)pf,
                                       (fm_act_t)act, ws, bytes, stream));
}

// device, stream, H, packed, scales, topk_ids, sorted_pairs, expert_offsets,
// topk_weights, out, expert_begin, group, ws, zeros, add
PyObject* moe_gemm_scatter_w4(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count(n, 15)) return nullptr;
  const Args a{v};
  Call c{"fm_moe_gemm_scatter_w4", (int)a.i(0)};
  const at::Tensor *h = c.matrix("H", v[2]), *w = c.matrix("topk_weights", v[8]),
                   *o = c.matrix("out", v[9]), *p = c.tensor("packed", v[3]);
  if (!c.bad && (!p || p->dim() != 3)) c.refuse(PyExc_ValueError, "packed must have three dimensions");
  if (c.bad) return nullptr;
  const int64_t T = w->size(0), topk = w->size(1), K = h->size(1), N = o->size(1),
                nl = p->size(0), group = a.i(11), G = groups_of(c, K, group);
  const int32_t e0 = c.i32("expert_begin", v[10]);
  int64_t sp = 0;
  check_pairs(c, h, v[6], T * topk, sp);
  const at::ScalarType dt = h->scalar_type();
  const fm_dtype_t code = c.code(dt);
  size_t bytes;
  void* ws = c.workspace(v[12], bytes);
  void *ph = c.at("H", v[2], dt, {h->size(0), K}),
       *pp = c.at("packed", v[3], kByte, {nl, N, row_bytes(K)}),
       *ps = c.at("scales", v[4], dt, {nl, G, N}),
       *pid = c.at("topk_ids", v[5], kInt, {T, topk}),
       *pq = c.at("sorted_pairs", v[6], kInt, {sp}),
       *pf = c.at("expert_offsets", v[7], kInt, {nl + 1}),
       *pw = c.at("topk_weights", v[8], kFloat, {T, topk}),
       *po = c.at("out", v[9], kFloat, {T, N}), *pz = c.at("zeros", v[13], kByte, {nl, G, N}),
       *pa = c.at("add", v[14], kFloat, {T, N});
  const hipStream_t stream = a.stream(1);
  if (c.bad || PyErr_Occurred()) return nullptr;
  return done(c, fm_moe_gemm_scatter_w4(code, T, N, K, (int32_t)topk, e0, (int32_t)nl,
                                        (int32_t)group, ph, pp, ps, (const uint8_t*)pz,
                                        (const int32_t*)pid, (const int32_t*)pq,
                                        (const int32_t*)pf, (const float*)pw, (const float*)pa,
                                        (float*)po, ws, bytes, stream));
}

// The random state of a call that drops: seed and offset.
const uint64_t* rng_of(Call& c, PyObject* o) { return (const uint64_t*)c.at("rng", o, at::kLong, {2}); }

// device, stream, x, y, p, rng, draw, row_begin, col_begin
PyObject* dropout(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count(n, 9)) return nullptr;
  const Args a{v};
  Call c{"fm_dropout", (int)a.i(0)};
  const at::Tensor* x = c.matrix("x", v[2]);
  if (c.bad) return nullptr;
  const int64_t M = x->size(0), N = x->size(1);
  const at::ScalarType dt = x->scalar_type();
  const fm_dtype_t code = c.code(dt);
  void *px = c.at("x", v[2], dt, {M, N}), *py = c.at("y", v[3], dt, {M, N});
  const uint64_t* rng = rng_of(c, v[5]);
  const float p = a.f(4);
  const int64_t draw = a.i(6), row = a.i(7), col = a.i(8);
  const hipStream_t stream = a.stream(1);
  if (c.bad || PyErr_Occurred()) return nullptr;
  return done(c, fm_dropout(code, M, N, px, p, rng, draw, row, col, py, stream));
}

// device, stream, out, y, block, resid, bias, w, b, p, rng, draw, row_begin, eps,
// y_scale, mean, rstd
PyObject* layer_norm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count(n, 17)) return nullptr;
  const Args a{v};
  Call c{"fm_layer_norm", (int)a.i(0)};
  const at::Tensor* like = c.matrix("block or resid", v[4] != Py_None ? v[4] : v[5]);
  if (c.bad) return nullptr;
  const int64_t M = like->size(0), N = like->size(1);
  const NormTypes t(c, v, {7, 6, 8}, {5, 2}, {4});
  void *pb = c.at("block", v[4], t.bd, {M, N}), *pr = c.at("resid", v[5], t.sd, {M, N}),
       *pi = c.at("bias", v[6], t.dt, {N}), *pw = c.at("w", v[7], t.dt, {N}),
       *pc = c.at("b", v[8], t.dt, {N}), *po = c.at("out", v[2], t.sd, {M, N}),
       *py = c.at("y", v[3], v[14] == Py_None ? t.dt : at::kChar, {M, N}),
       *ps = c.at("y_scale", v[14], kFloat, {M}), *pm = c.at("mean", v[15], kFloat, {M}),
       *pq = c.at("rstd", v[16], kFloat, {M});
  const uint64_t* rng = rng_of(c, v[10]);
  const fm_dtype_t dt = c.code(t.dt), sd = c.code(t.sd), bd = c.code(t.bd);
  const float p = a.f(9), eps = a.f(13);
  const int64_t draw = a.i(11), row = a.i(12);
  const hipStream_t stream = a.stream(1);
  if (c.bad || PyErr_Occurred()) return nullptr;
  return done(c, fm_layer_norm(dt, sd, bd, M, N, pb, pr, pi, pw, pc, p, rng, draw, row, eps, po, py,
                               (float*)ps, (float*)pm, (float*)pq, stream));
}

// device, stream, d_resid, d_block, out, d_y, d_out, w, p, rng, draw, row_begin, mean,
// rstd, d_bias, d_w, d_b, ws
PyObject* layer_norm_bwd(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count(n, 18)) return nullptr;
  const Args a{v};
  Call c{"fm_layer_norm_bwd", (int)a.i(0)};
  const at::Tensor* like = c.matrix("d_y or d_out", v[5] != Py_None ? v[5] : v[6]);
  if (c.bad) return nullptr;
  const int64_t M = like->size(0), N = like->size(1);
  const NormTypes t(c, v, {5, 7}, {6, 4, 2}, {3});
  size_t bytes;
  void* ws = c.workspace(v[17], bytes);
  void *dr = c.at("d_resid", v[2], t.sd, {M, N}), *db = c.at("d_block", v[3], t.bd, {M, N}),
       *po = c.at("out", v[4], t.sd, {M, N}), *dy = c.at("d_y", v[5], t.dt, {M, N}),
       *dz = c.at("d_out", v[6], t.sd, {M, N}), *pw = c.at("w", v[7], t.dt, {N}),
       *pm = c.at("mean", v[12], kFloat, {M}), *pq = c.at("rstd", v[13], kFloat, {M}),
       *di = c.at("d_bias", v[14], kFloat, {N}), *dw = c.at("d_w", v[15], kFloat, {N}),
       *dc = c.at("d_b", v[16], kFloat, {N});
  const uint64_t* rng = rng_of(c, v[9]);
  const fm_dtype_t dt = c.code(t.dt), sd = c.code(t.sd), bd = c.code(t.bd);
  const float p = a.f(8);
  const int64_t draw = a.i(10), row = a.i(11);
  const hipStream_t stream = a.stream(1);
  if (c.bad || PyErr_Occurred()) return nullptr;
  return done(c, fm_layer_norm_bwd(dt, sd, bd, M, N, dy, dz, po, (const float*)pm,
                                   (const float*)pq, pw, p, rng, draw, row, dr, db, (float*)di,
                                   (float*)dw, (float*)dc, ws, bytes, stream));
}

// device, stream, x, q, scale
PyObject* quant_i8(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count(n, 5)) return nullptr;
  const Args a{v};
  Call c{"fm_quant_i8", (int)a.i(0)};
  const at::Tensor* x = c.matrix("x", v[2]);
  if (c.bad) return nullptr;
  const int64_t M = x->size(0), N = x->size(1);
  const at::ScalarType dt = x->scalar_type();
  const fm_dtype_t code = c.code(dt);
  void *px = c.at("x", v[2], dt, {M, N}), *pq = c.at("q", v[3], at::kChar, {M, N}),
       *ps = c.at("scale", v[4], kFloat, {M});
  const hipStream_t stream = a.stream(1);
  if (c.bad || PyErr_Occurred()) return nullptr;
  return done(c, fm_quant_i8(code, M, N, px, (int8_t*)pq, (float*)ps, stream));
}

// device, stream, A, a_scale, W, w_scale, C, bias, act
PyObject* gemm_i8(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count(n, 9)) return nullptr;
  const Args a{v};
  Call c{"fm_gemm_i8", (int)a.i(0)};
  const at::Tensor *x = c.matrix("A", v[2]), *y = c.matrix("C", v[6]), *b = c.tensor("bias", v[7]);
  if (c.bad) return nullptr;
  const int64_t M = x->size(0), K = x->size(1), N = y->size(1);
  const at::ScalarType ct = y->scalar_type(),
                       dt = b ? b->scalar_type() : ct == kFloat ? at::kBFloat16 : ct;
  const fm_dtype_t code = c.code(dt), cc = c.code(ct);
  const int32_t act = c.i32("act", v[8]);
  void *pa = c.at("A", v[2], at::kChar, {M, K}), *ps = c.at("a_scale", v[3], kFloat, {M}),
       *pw = c.at("W", v[4], at::kChar, {N, K}), *pt = c.at("w_scale", v[5], kFloat, {N}),
       *pc = c.at("C", v[6], ct, {M, N}), *pb = c.at("bias", v[7], dt, {N});
  const hipStream_t stream = a.stream(1);
  if (c.bad || PyErr_Occurred()) return nullptr;
  return done(c, fm_gemm_i8(code, cc, M, N, K, (const int8_t*)pa, (const float*)ps,
                            (const int8_t*)pw, (const float*)pt, pb, (fm_act_t)act, pc, stream));
}

// device, stream, X, W, w_scale, C, bias, act, ws
PyObject* linear_i8(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count(n, 9)) return nullptr;
  const Args a{v};
  Call c{"fm_linear_i8", (int)a.i(0)};
  const at::Tensor *x = c.matrix("X", v[2]), *y = c.matrix("C", v[5]);
  if (c.bad) return nullptr;
  const int64_t M = x->size(0), K = x->size(1), N = y->size(1);
  const at::ScalarType dt = x->scalar_type(), ct = y->scalar_type();
  const fm_dtype_t code = c.code(dt), cc = c.code(ct);
  const int32_t act = c.i32("act", v[7]);
  size_t bytes;
  void* ws = c.workspace(v[8], bytes);
  void *px = c.at("X", v[2], dt, {M, K}), *pw = c.at("W", v[3], at::kChar, {N, K}),
       *pt = c.at("w_scale", v[4], kFloat, {N}), *pc = c.at("C", v[5], ct, {M, N}),
       *pb = c.at("bias", v[6], dt, {N});
  const hipStream_t stream = a.stream(1);
  if (c.bad || PyErr_Occurred()) return nullptr;
  return done(c, fm_linear_i8(code, cc, M, N, K, px, (const int8_t*)pw, (const float*)pt, pb,
                              (fm_act_t)act, pc, ws, bytes, stream));
}

// No C++ exception leaves the module.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* v, Py_ssize_t n) {
  try {
    return F(self, v, n);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

#define FM_METHOD(F) {#F, (PyCFunction)(void (*)(void))guarded<F>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FM_METHOD(moe_gate),
                         FM_METHOD(moe_gate_bwd),
                         FM_METHOD(norm_residual),
                         FM_METHOD(norm_residual_bwd),
                         FM_METHOD(gemm_w4),
                         FM_METHOD(moe_gather_gemm_w4),
                         FM_METHOD(moe_gemm_scatter_w4),
                         FM_METHOD(dropout),
                         FM_METHOD(layer_norm),
                         FM_METHOD(layer_norm_bwd),
                         FM_METHOD(quant_i8),
                         FM_METHOD(gemm_i8),
                         FM_METHOD(linear_i8),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fluxmi", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__fluxmi(void) { return PyModule_Create(&module); }
