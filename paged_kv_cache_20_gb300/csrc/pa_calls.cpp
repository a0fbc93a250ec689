// pa_calls.cpp -- the Python binding's short way into the calls that a decode step makes
// on few tokens, where the GPU needs 2-7 us and checking a dozen tensors from Python took
// 6-7 us a call (rotary append of 8 tokens back to back: 11.3 us through Python and ctypes,
// 3.1 this way).
//
// Each function takes the binding's arguments in order, checks them as the binding does
// (types, shapes, layout, device) and makes the C call on the current stream.  It returns
// the pa_status, or None where any check fails or an argument is one that only the
// binding's own code handles: that code then makes the call or says what is wrong.  So
// nothing here refuses anything, and every message has one place.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/pagedattn.h"

namespace {

using at::ScalarType;
using at::Tensor;

// The arguments of one call; `ok` turns false at the first that does not fit.
struct Call {
  PyObject *const *args;
  int dev = -1;
  bool ok = true;

  const Tensor *tensor(int i) {
    PyObject *o = args[i];
    if (!THPVariable_Check(o)) {
      ok = false;
      return nullptr;
    }
    const Tensor *t = &THPVariable_Unpack(o);
    if (!t->is_cuda() || (dev >= 0 && t->get_device() != dev)) {
      ok = false;
      return nullptr;
    }
    return t;
  }
  bool none(int i) const { return args[i] == Py_None; }
  // the call's device is its first tensor's, which has to be the current one
  const Tensor *first(int i) {
    const Tensor *t = tensor(i);
    if (!ok) return nullptr;
    dev = t->get_device();
    ok = dev == c10::cuda::current_device();
    return ok ? t : nullptr;
  }
  // contiguous, of this type and shape
  void *dense(int i, ScalarType type, at::IntArrayRef shape) {
    const Tensor *t = ok ? tensor(i) : nullptr;
    ok = ok && t->scalar_type() == type && t->sizes() == shape && t->is_contiguous();
    return ok ? t->data_ptr() : nullptr;
  }
  void *maybe(int i, ScalarType type, at::IntArrayRef shape) {
    return ok && !none(i) ? dense(i, type, shape) : nullptr;
  }
  long integer(int i) {
    const long v = PyLong_Check(args[i]) ? PyLong_AsLong(args[i]) : -1;
    if (!PyLong_Check(args[i]) || v < 0 || v > INT32_MAX) {  // (-1 also stands for an overflow)
      PyErr_Clear();
      ok = false;
    }
    return v;
  }
  void *stream() const { return c10::cuda::getCurrentCUDAStream(dev).stream(); }
};

// The C call itself, without the interpreter's lock: a launch waits where the driver's queue
// is full, and other threads (or a host function in that queue) may need the interpreter to
// go on.  (0.03 to 0.13 us a call.)
template <typename F>
pa_status unlocked(F call) {
  struct Lock {
    PyThreadState *state = PyEval_SaveThread();
    ~Lock() { PyEval_RestoreThread(state); }
  } lock;
  return call();
}

bool element(const Tensor &t, pa_dtype *dt) {
  if (t.scalar_type() == at::kHalf)
    *dt = PA_FP16;
  else if (t.scalar_type() == at::kBFloat16)
    *dt = PA_BF16;
  else
    return false;
  return true;
}

bool codes(ScalarType t) { return t == at::kByte || t == at::kFloat8_e4m3fn; }

// A pair of caches and their scales: 16-bit of type `type` without, e4m3 codes with.
struct Caches {
  void *k = nullptr, *v = nullptr;
  const float *ks = nullptr, *vs = nullptr;
  int64_t blocks = 0, heads = 0, block = 0, dim = 0;
  Caches(Call &c, int k_at, int v_at, int ks_at, int vs_at, ScalarType type) {
    const Tensor *t = c.ok ? c.tensor(k_at) : nullptr;
    c.ok = c.ok && t->dim() == 4 && c.none(ks_at) == c.none(vs_at);
    if (!c.ok) return;
    const at::IntArrayRef shape = t->sizes();
    blocks = shape[0], heads = shape[1], block = shape[2], dim = shape[3];
    if (!c.none(ks_at)) {
      type = t->scalar_type();
      c.ok = codes(type);
      ks = static_cast<const float *>(c.maybe(ks_at, at::kFloat, {heads}));
      vs = static_cast<const float *>(c.maybe(vs_at, at::kFloat, {heads}));
    }
    if (!c.ok) return;
    k = c.dense(k_at, type, shape);
    v = c.dense(v_at, type, shape);
  }
};

// [tokens][heads][dim] with dense heads: pointer, and elements between tokens.
void *tokens3(Call &c, int i, ScalarType type, at::IntArrayRef shape, int64_t *stride) {
  const Tensor *t = c.ok ? c.tensor(i) : nullptr;
  c.ok = c.ok && t->scalar_type() == type && t->sizes() == shape;
  if (!c.ok) return nullptr;
  if (t->is_contiguous()) {
    *stride = shape[1] * shape[2];
  } else {
    c.ok = t->stride(2) == 1 && t->stride(1) == shape[2] && shape[0] > 1;
    *stride = t->stride(0);
  }
  return c.ok ? t->data_ptr() : nullptr;
}

bool fits(std::initializer_list<int64_t> sizes) {
  for (const int64_t s : sizes)
    if (s > INT32_MAX) return false;
  return true;
}

PyObject *answer(const Call &c, pa_status st) {
  if (!c.ok) Py_RETURN_NONE;
  return PyLong_FromLong(st);
}

// q_out, q, k, v, k_cache, v_cache, positions, slot_mapping, turns, pair_axis, interleaved,
// k_scale, v_scale
pa_status rope_append(Call &c) {
  const Tensor *q = c.first(1);
  pa_dtype dt = PA_FP16;
  c.ok = c.ok && q->dim() == 3 && element(*q, &dt) && PyBool_Check(c.args[10]);
  if (!c.ok) return PA_OK;
  const ScalarType type = q->scalar_type();
  const Caches kv(c, 4, 5, 11, 12, type);
  const int64_t n = q->size(0), hq = q->size(1);
  c.ok = c.ok && q->size(2) == kv.dim && n > 0;
  int64_t sq = 0, so = 0, sk = 0, sv = 0;
  void *qp = tokens3(c, 1, type, {n, hq, kv.dim}, &sq), *qo = tokens3(c, 0, type, {n, hq, kv.dim}, &so);
  void *kp = tokens3(c, 2, type, {n, kv.heads, kv.dim}, &sk);
  void *vp = tokens3(c, 3, type, {n, kv.heads, kv.dim}, &sv);
  const Tensor *pos = c.ok ? c.tensor(6) : nullptr, *turns = c.ok ? c.tensor(8) : nullptr;
  c.ok = c.ok && (pos->dim() == 2 || pos->dim() == 1) && turns->dim() == 1;
  if (!c.ok) return PA_OK;
  const int64_t axes = pos->dim() == 2 ? pos->size(0) : 1, half = turns->size(0);
  void *pp = pos->dim() == 2 ? c.dense(6, at::kInt, {axes, n}) : c.dense(6, at::kInt, {n});
  void *sm = c.dense(7, at::kLong, {n}), *tp = c.dense(8, at::kLong, {half}), *ap = c.dense(9, at::kInt, {half});
  c.ok = c.ok && fits({n, hq, kv.heads, kv.blocks, axes, 2 * half});
  if (!c.ok) return PA_OK;
  const int adjacent = c.args[10] == Py_True;
  void *s = c.stream();
  return unlocked([&] {
    return pa_rope_append(qo, qp, kp, vp, kv.k, kv.v, static_cast<const int32_t *>(pp),
                          static_cast<const int64_t *>(sm), static_cast<const int64_t *>(tp),
                          static_cast<const int32_t *>(ap), (int)n, (int)hq, (int)kv.heads, (int)kv.dim,
                          (int)(2 * half), (int)axes, adjacent, so, sq, sk, sv, (int)kv.block, (int)kv.blocks, dt,
                          kv.ks, kv.vs, s);
  });
}

// out, scores, q, k_cache, v_cache, block_tables, context_lens, scale, q_len, num_splits,
// workspace, row_pos, seq_lens, k_scale, v_scale
pa_status decode_scored(Call &c) {
  const Tensor *q = c.first(2);
  pa_dtype dt = PA_FP16;
  c.ok = c.ok && element(*q, &dt) && PyFloat_Check(c.args[7]) && c.none(11) == c.none(12);
  if (!c.ok) return PA_OK;
  const ScalarType type = q->scalar_type();
  const Caches kv(c, 3, 4, 13, 14, type);
  const long u = c.integer(8), splits = c.integer(9);
  const Tensor *bt = c.ok ? c.tensor(5) : nullptr, *ws = c.ok ? c.tensor(10) : nullptr;
  c.ok = c.ok && bt->dim() == 2 && ws->is_contiguous() && q->dim() >= 3;
  if (!c.ok) return PA_OK;
  const int64_t n = bt->size(0), width = bt->size(1), hq = q->size(-2), rows = width * kv.block;
  void *tables = c.dense(5, at::kInt, {n, width}), *lens = c.dense(6, at::kInt, {n});
  void *qp, *op;
  if (q->dim() == 4) {
    qp = c.dense(2, type, {n, u, hq, kv.dim});
    op = c.dense(0, type, {n, u, hq, kv.dim});
  } else {
    c.ok = c.ok && u == 1;
    qp = c.dense(2, type, {n, hq, kv.dim});
    op = c.dense(0, type, {n, hq, kv.dim});
  }
  void *sc = c.dense(1, at::kFloat, {n, kv.heads, rows});
  void *rp = c.maybe(11, at::kInt, {n, kv.heads, rows}), *sl = c.maybe(12, at::kInt, {n});
  c.ok = c.ok && fits({n, hq, kv.heads, kv.blocks, rows});
  if (!c.ok) return PA_OK;
  const float scale = (float)PyFloat_AS_DOUBLE(c.args[7]);
  void *room = ws->data_ptr(), *s = c.stream();
  const size_t room_bytes = ws->nbytes();
  return unlocked([&] {
    return pa_decode_scored(op, static_cast<float *>(sc), static_cast<int32_t *>(rp), qp, kv.k, kv.v, kv.ks, kv.vs,
                            static_cast<const int32_t *>(tables), static_cast<const int32_t *>(lens),
                            static_cast<const int32_t *>(sl), (int)n, (int)hq, (int)kv.heads, (int)kv.dim,
                            (int)kv.block, scale, (int)width, (int)kv.blocks, (int)u, dt, (int)splits, room,
                            room_bytes, s);
  });
}

// k_cache, v_cache, scores, row_pos, block_tables, context_lens, seq_lens, budget, sinks,
// recent, scores_out, row_pos_out, new_lens, workspace
pa_status evict(Call &c) {
  const Tensor *k = c.first(0);
  c.ok = c.ok && k->dim() == 4 && c.none(10) == c.none(11);
  if (!c.ok) return PA_OK;
  const ScalarType type = k->scalar_type();
  const int bytes = type == at::kHalf || type == at::kBFloat16 ? 2 : codes(type) ? 1 : 0;
  const at::IntArrayRef shape = k->sizes();
  void *kp = c.dense(0, type, shape), *vp = c.dense(1, type, shape);
  const Tensor *bt = c.ok ? c.tensor(4) : nullptr, *ws = c.ok ? c.tensor(13) : nullptr;
  c.ok = c.ok && bytes && bt->dim() == 2 && ws->is_contiguous();
  if (!c.ok) return PA_OK;
  const int64_t n = bt->size(0), width = bt->size(1), h = shape[1], rows = width * shape[2];
  const long budget = c.integer(7), sinks = c.integer(8), recent = c.integer(9);
  void *sc = c.dense(2, at::kFloat, {n, h, rows}), *rp = c.dense(3, at::kInt, {n, h, rows});
  void *so = c.none(10) ? sc : c.dense(10, at::kFloat, {n, h, rows});
  void *po = c.none(11) ? rp : c.dense(11, at::kInt, {n, h, rows});
  void *tables = c.dense(4, at::kInt, {n, width}), *lens = c.dense(5, at::kInt, {n});
  void *seen = c.dense(6, at::kInt, {n}), *nl = c.dense(12, at::kInt, {n});
  c.ok = c.ok && fits({n, h, shape[0], rows});
  if (!c.ok) return PA_OK;
  const int blocks = (int)shape[0], block = (int)shape[2], dim = (int)shape[3];
  void *room = ws->data_ptr(), *s = c.stream();
  const size_t room_bytes = ws->nbytes();
  return unlocked([&] {
    return pa_evict(kp, vp, static_cast<float *>(so), static_cast<int32_t *>(po), static_cast<int32_t *>(nl),
                    static_cast<const float *>(sc), static_cast<const int32_t *>(rp),
                    static_cast<const int32_t *>(tables), static_cast<const int32_t *>(lens),
                    static_cast<const int32_t *>(seen), (int)n, (int)h, dim, block, (int)width, blocks, (int)budget,
                    (int)sinks, (int)recent, bytes, room, room_bytes, s);
  });
}

// fp32 [n][r][vocab], rows dense and evenly spaced
const float *prob_rows(Call &c, int i, int64_t n, int64_t r, int64_t vocab, int64_t *row) {
  const Tensor *t = c.ok ? c.tensor(i) : nullptr;
  c.ok = c.ok && t->scalar_type() == at::kFloat && t->dim() == 3 && t->size(0) == n && t->size(1) == r &&
         t->size(2) == vocab && t->is_contiguous();
  *row = vocab;
  return c.ok ? static_cast<const float *>(t->data_ptr()) : nullptr;
}

// target_probs, draft_probs, draft_tokens, accept_u, sample_u, draft_lens, context_lens,
// out_tokens, num_accepted, new_lens
pa_status verify_drafts(Call &c) {
  const Tensor *p = c.first(0), *x = c.ok ? c.tensor(2) : nullptr;
  c.ok = c.ok && p->dim() == 3 && x->dim() == 2 && c.none(9) == c.none(6);
  if (!c.ok) return PA_OK;
  const int64_t n = x->size(0), k = x->size(1), vocab = p->size(2);
  int64_t ps = 0, qs = 0;
  const float *pp = prob_rows(c, 0, n, k + 1, vocab, &ps);
  const float *qp = c.none(1) ? nullptr : prob_rows(c, 1, n, k, vocab, &qs);
  void *xp = c.dense(2, at::kInt, {n, k}), *au = c.dense(3, at::kFloat, {n, k}), *su = c.dense(4, at::kFloat, {n});
  void *dl = c.maybe(5, at::kInt, {n}), *cl = c.maybe(6, at::kInt, {n}), *nl = c.maybe(9, at::kInt, {n});
  void *out = c.dense(7, at::kInt, {n, k + 1}), *acc = c.dense(8, at::kInt, {n});
  c.ok = c.ok && fits({n, k, vocab});
  if (!c.ok) return PA_OK;
  void *s = c.stream();
  return unlocked([&] {
    return pa_verify_drafts(static_cast<int32_t *>(out), static_cast<int32_t *>(acc), static_cast<int32_t *>(nl),
                            static_cast<const int32_t *>(cl), pp, qp, static_cast<const int32_t *>(xp),
                            static_cast<const int32_t *>(dl), static_cast<const float *>(au),
                            static_cast<const float *>(su), (int)n, (int)k, (int)vocab, ps, qs, s);
  });
}

// (no exception leaves: a tensor that has no plain storage, say, is the binding's business)
template <pa_status (*F)(Call &), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  Call c{args};
  try {
    const pa_status st = F(c);
    return answer(c, st);
  } catch (...) {
    Py_RETURN_NONE;
  }
}

PyMethodDef kMethods[] = {
    {"rope_append", (PyCFunction)(void (*)(void))entry<rope_append, 13>, METH_FASTCALL, nullptr},
    {"decode_scored", (PyCFunction)(void (*)(void))entry<decode_scored, 15>, METH_FASTCALL, nullptr},
    {"evict", (PyCFunction)(void (*)(void))entry<evict, 14>, METH_FASTCALL, nullptr},
    {"verify_drafts", (PyCFunction)(void (*)(void))entry<verify_drafts, 10>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", "Checked calls of libpagedattn.so.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch whose headers this was built with; with another one nothing here
// may be called.
PyMODINIT_FUNC PyInit__calls(void) {
  PyObject *m = PyModule_Create(&kModule);
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", PA_TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
