// Tensor calls of the operators in front of the scores: checks of the tensors (types, shapes,
// strides, devices) and the C ABI call, natively.  A step of a few tokens runs in 4 to 6 us on the
// GPU; the same checks in Python took 6 to 11 us a call.  No arithmetic of the operators lives here:
// the functions of libecho.so are called through the addresses that binding.py hands over.
#include <Python.h>

#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <string>

#include "../../include/echo.h"

namespace {

PyObject *g_error = nullptr;        // binding.EchoError(function, code, text)
PyObject *g_raw_stream = nullptr;   // device index -> handle of torch's current stream
const char *(*g_last_error)() = nullptr;
int (*g_page_step)(const echo_page_args *, void *, size_t, void *) = nullptr;
decltype(&echo_quant_fp8) g_quant = nullptr;
decltype(&echo_matmul_fp8) g_matmul = nullptr;
decltype(&echo_qk_norm_rope) g_rope = nullptr;
decltype(&echo_indexer_qk) g_indexer = nullptr;
decltype(&echo_newest_queries) g_newest = nullptr;

struct Refused {};                  // a Python error is set

[[noreturn]] void raise(const char *fn, int code, const std::string &text) {
  PyObject *e = PyObject_CallFunction(g_error, "sis", fn, code, text.c_str());
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Refused{};
}
[[noreturn]] void refuse(const char *fn, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  raise(fn, ECHO_EINVAL, buf);
}

const at::Tensor *tensor(const char *fn, const char *name, PyObject *o, bool may_be_none = false) {
  if (o == Py_None && may_be_none) return nullptr;
  if (!THPVariable_Check(o)) refuse(fn, "%s is not a tensor", name);
  return &THPVariable_Unpack(o);
}
int64_t integer(PyObject *o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}
int32_t integer32(const char *fn, const char *name, PyObject *o) {
  const int64_t v = integer(o);
  if (v != static_cast<int32_t>(v)) refuse(fn, "%s does not fit 32 bits", name);
  return static_cast<int32_t>(v);
}
double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return v;
}

int32_t float_type(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return ECHO_BF16;
    case at::kHalf: return ECHO_FP16;
    case at::kFloat: return ECHO_FP32;
    default: return -1;
  }
}
bool is_codes(at::ScalarType t) { return t == at::kByte || t == at::kFloat8_e4m3fn; }
int32_t count32(const char *fn, int64_t n) {
  if (n > INT32_MAX) refuse(fn, "a size above 2^31 - 1");
  return static_cast<int32_t>(n);
}
void *address(const at::Tensor *t) { return t ? t->data_ptr() : nullptr; }

// The call's device and stream.  `any`: tensors of any device go (a library whose kernels run on
// the host); otherwise they are on torch's current GPU.
struct Where {
  const char *fn;
  c10::Device dev;
  Where(const char *f, const at::Tensor *first) : fn(f), dev(first->device()) {}
  void same(const char *name, const at::Tensor *t) const {
    if (t && t->device() != dev) refuse(fn, "%s is on another device than the first tensor", name);
  }
  void *stream(PyObject *given, bool any) const {
    if (!any) {
      if (dev.type() != c10::DeviceType::CUDA) refuse(fn, "tensors on %s, not on a GPU", dev.str().c_str());
      const c10::Device cur = c10::impl::VirtualGuardImpl(c10::DeviceType::CUDA).getDevice();
      if (cur != dev) refuse(fn, "tensors on %s; the current device is %s", dev.str().c_str(), cur.str().c_str());
    }
    if (given != Py_None) return reinterpret_cast<void *>(PyLong_AsUnsignedLongLong(given));
    PyObject *i = PyLong_FromLong(dev.index());
    PyObject *s = i ? PyObject_CallOneArg(g_raw_stream, i) : nullptr;
    Py_XDECREF(i);
    if (!s) throw Refused{};
    void *h = reinterpret_cast<void *>(PyLong_AsUnsignedLongLong(s));
    Py_DECREF(s);
    return h;
  }
};

// t is contiguous, of type `type`, on the call's device and holds n elements (n < 0: any number).
void want(const Where &w, const char *name, const at::Tensor *t, at::ScalarType type, int64_t n) {
  if (!t) return;
  if (t->scalar_type() != type) refuse(w.fn, "%s is %s, not %s", name, c10::toString(t->scalar_type()), c10::toString(type));
  if (!t->is_contiguous()) refuse(w.fn, "%s is not contiguous", name);
  if (n >= 0 && t->numel() != n) refuse(w.fn, "%s has %lld elements, not %lld", name, static_cast<long long>(t->numel()), static_cast<long long>(n));
  w.same(name, t);
}

void check(const char *fn, int code) {
  if (code != ECHO_OK) raise(fn, code, g_last_error());
}

int64_t row_stride(const char *fn, const char *name, const at::Tensor &t) {
  const int64_t rows = t.size(0), cols = t.size(1);
  if (cols > 1 && t.stride(1) != 1) refuse(fn, "the rows of %s are not contiguous", name);
  return rows > 1 ? t.stride(0) : cols;
}
// The stride of a dimension of one means nothing.
int64_t stride(const at::Tensor &t, int d) { return t.size(d) > 1 ? t.stride(d) : 0; }

template <typename F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t need, F f) {
  if (got != need) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", got, need);
    return nullptr;
  }
  try {
    f();
  } catch (const Refused &) {
    return nullptr;
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
  Py_RETURN_NONE;
}

PyObject *page_step(PyObject *, PyObject *const *o, Py_ssize_t n_args) {
  return guarded(n_args, 17, [&] {
    const char *fn = "echo_page_step";
    const at::Tensor *len_in = tensor(fn, "len_in", o[0]), *new_len = tensor(fn, "new_len", o[1]),
                     *table = tensor(fn, "page_table", o[2]), *free_list = tensor(fn, "free_list", o[4]),
                     *count_in = tensor(fn, "count_in", o[5]), *len_out = tensor(fn, "len_out", o[6]),
                     *count_out = tensor(fn, "count_out", o[7]), *row_begin = tensor(fn, "row_begin", o[8]),
                     *slot = tensor(fn, "slot", o[9]), *row = tensor(fn, "row", o[10], true),
                     *pos = tensor(fn, "pos", o[11]), *status = tensor(fn, "status", o[12]),
                     *ws = tensor(fn, "ws", o[13], true), *done = tensor(fn, "done", o[14], true);
    const Where w(fn, len_in);
    const int64_t n = len_in->numel(), cap = slot->numel();
    want(w, "len_in", len_in, at::kInt, n);
    want(w, "new_len", new_len, at::kInt, n);
    if (table->dim() != 2 || table->size(0) != n) refuse(fn, "page_table has no row for each request");
    want(w, "page_table", table, at::kInt, -1);
    want(w, "free_list", free_list, at::kInt, -1);
    want(w, "count_in", count_in, at::kInt, 1);
    want(w, "len_out", len_out, at::kInt, n);
    want(w, "count_out", count_out, at::kInt, 1);
    want(w, "row_begin", row_begin, at::kInt, n + 1);
    want(w, "slot", slot, at::kLong, cap);
    want(w, "row", row, at::kInt, cap);
    want(w, "pos", pos, at::kInt, cap);
    want(w, "status", status, at::kInt, 1);
    if (done) want(w, "done", done, done->scalar_type() == at::kBool ? at::kBool : at::kByte, n);
    if (ws) want(w, "ws", ws, ws->scalar_type(), -1);
    void *st = w.stream(o[15], o[16] == Py_True);
    const echo_page_args a = {
        count32(fn, n), integer32(fn, "page_size", o[3]), count32(fn, table->size(1)), count32(fn, free_list->numel()), count32(fn, cap),
        static_cast<const int32_t *>(address(len_in)), static_cast<const int32_t *>(address(new_len)),
        static_cast<const uint8_t *>(address(done)), static_cast<int32_t *>(address(table)),
        static_cast<int32_t *>(address(free_list)), static_cast<const int32_t *>(address(count_in)),
        static_cast<int32_t *>(address(len_out)), static_cast<int32_t *>(address(count_out)),
        static_cast<int32_t *>(address(row_begin)), static_cast<int64_t *>(address(slot)),
        static_cast<int32_t *>(address(row)), static_cast<int32_t *>(address(pos)), static_cast<int32_t *>(address(status))};
    check(fn, g_page_step(&a, address(ws), ws ? ws->nbytes() : 0, st));
  });
}

PyObject *quant_fp8(PyObject *, PyObject *const *o, Py_ssize_t n_args) {
  return guarded(n_args, 5, [&] {
    const char *fn = "echo_quant_fp8";
    const at::Tensor *x = tensor(fn, "x", o[0]), *y = tensor(fn, "y", o[1]), *scale = tensor(fn, "scale", o[2]);
    const int32_t kind = float_type(x->scalar_type());
    if (kind < 0 || x->dim() != 2) refuse(fn, "x is not a matrix of bf16, fp16 or fp32");
    const int64_t rows = x->size(0), cols = x->size(1);
    if (y->sizes() != x->sizes() || scale->dim() != 2 || scale->size(0) != rows || scale->size(1) != (cols + 127) / 128)
      refuse(fn, "shapes of y or scale do not go with x [%lld, %lld]", static_cast<long long>(rows), static_cast<long long>(cols));
    if (!is_codes(y->scalar_type()) || scale->scalar_type() != at::kFloat) refuse(fn, "y is not FP8 codes or scale not fp32");
    const Where w(fn, x);
    w.same("y", y);
    w.same("scale", scale);
    const int64_t ldx = row_stride(fn, "x", *x), ldy = row_stride(fn, "y", *y);
    check(fn, g_quant(address(x), kind, rows, count32(fn, cols), ldx, static_cast<uint8_t *>(address(y)), ldy,
                      static_cast<float *>(address(scale)), stride(*scale, 0), stride(*scale, 1), w.stream(o[3], o[4] == Py_True)));
  });
}

// Row stride of a matrix of codes whose rows are read in 16-byte pieces.
int64_t codes_stride(const char *fn, const char *name, const at::Tensor &t) {
  if (!is_codes(t.scalar_type())) refuse(fn, "%s is not FP8 codes", name);
  const int64_t rows = t.size(0), k = t.size(1);
  int64_t ld = row_stride(fn, name, t);
  if (rows < 2) ld = (ld + 15) / 16 * 16;                  // of no row's distance from another
  if (k % 16 && rows && static_cast<int64_t>(t.storage().nbytes()) - t.storage_offset() < (rows - 1) * ld + (k + 15) / 16 * 16)
    refuse(fn, "the last row of %s ends inside a 16-byte piece", name);
  return ld;
}

PyObject *matmul_fp8(PyObject *, PyObject *const *o, Py_ssize_t n_args) {
  return guarded(n_args, 7, [&] {
    const char *fn = "echo_matmul_fp8";
    const at::Tensor *a = tensor(fn, "a", o[0]), *as = tensor(fn, "a_scale", o[1]), *b = tensor(fn, "b", o[2]),
                     *bs = tensor(fn, "b_scale", o[3]), *c = tensor(fn, "c", o[4]);
    if (a->dim() != 2 || b->dim() != 2 || c->dim() != 2) refuse(fn, "a, b and c are matrices");
    const int64_t m = a->size(0), k = a->size(1), n = b->size(0), nb = (k + 127) / 128;
    if (b->size(1) != k || c->size(0) != m || c->size(1) != n || as->dim() != 2 || as->size(0) != m || as->size(1) != nb ||
        bs->dim() != 2 || bs->size(0) != (n + 127) / 128 || bs->size(1) != nb)
      refuse(fn, "shapes do not go together for a [%lld, %lld] and b [%lld, %lld]", static_cast<long long>(m),
             static_cast<long long>(k), static_cast<long long>(n), static_cast<long long>(b->size(1)));
    const int32_t kind = float_type(c->scalar_type());
    if (kind < 0 || as->scalar_type() != at::kFloat || bs->scalar_type() != at::kFloat)
      refuse(fn, "c is not bf16, fp16 or fp32, or a scale not fp32");
    const Where w(fn, a);
    w.same("a_scale", as);
    w.same("b", b);
    w.same("b_scale", bs);
    w.same("c", c);
    const int64_t lda = codes_stride(fn, "a", *a), ldb = codes_stride(fn, "b", *b), ldc = row_stride(fn, "c", *c);
    check(fn, g_matmul(static_cast<const uint8_t *>(address(a)), lda, static_cast<const float *>(address(as)), stride(*as, 0), stride(*as, 1),
                       static_cast<const uint8_t *>(address(b)), ldb, static_cast<const float *>(address(bs)), stride(*bs, 0),
                       stride(*bs, 1), count32(fn, m), count32(fn, n), count32(fn, k), address(c), ldc, kind, w.stream(o[5], o[6] == Py_True)));
  });
}

// Strides of tokens and heads.
void head_strides(const char *fn, const char *name, const at::Tensor &t, int64_t &tok, int64_t &head) {
  if (t.numel() && t.size(2) > 1 && t.stride(2) != 1) refuse(fn, "the heads of %s are not contiguous", name);
  tok = stride(t, 0);
  head = stride(t, 1);
}

constexpr int QK = 15;              // arguments of qk_args: q, k, pos, cos_sin, rot_begin, ..., k_bias
echo_qk_args qk_args(const Where &w, const at::Tensor &q, const at::Tensor &k, PyObject *const *o) {
  const char *fn = w.fn;
  const at::Tensor *pos = tensor(fn, "pos", o[2]), *cs = tensor(fn, "cos_sin", o[3], true);
  const int32_t kind = float_type(q.scalar_type());
  if (kind < 0 || k.scalar_type() != q.scalar_type() || q.dim() != 3 || k.dim() != 3)
    refuse(fn, "q and k are not [tokens, heads, head_dim] of one type, bf16, fp16 or fp32");
  const int64_t n = q.size(0), dim = q.size(2);
  if (k.size(0) != n || k.size(2) != dim) refuse(fn, "q and k have other numbers of tokens or other head sizes");
  w.same("k", &k);
  want(w, "pos", pos, at::kInt, n);
  echo_qk_args a = {};
  a.n_pos = ECHO_INF;
  if (cs) {
    want(w, "cos_sin", cs, at::kFloat, -1);
    if (cs->dim() != 2) refuse(fn, "cos_sin is not [positions, rotated values]");
    a.n_pos = count32(fn, cs->size(0));
    a.rot_dim = count32(fn, cs->size(1));
  }
  const char *names[4] = {"q_weight", "q_bias", "k_weight", "k_bias"};
  const int at_arg[4] = {8, 9, 11, 12};
  const float *vec[4];
  for (int i = 0; i < 4; ++i) {
    const at::Tensor *t = tensor(fn, names[i], o[at_arg[i]], true);
    want(w, names[i], t, at::kFloat, dim);
    vec[i] = static_cast<const float *>(address(t));
  }
  a.n_tok = count32(fn, n);
  a.n_q_heads = count32(fn, q.size(1));
  a.n_k_heads = count32(fn, k.size(1));
  a.head_dim = count32(fn, dim);
  a.type = kind;
  a.rot_begin = integer32(fn, "rot_begin", o[4]);
  a.interleaved = PyObject_IsTrue(o[5]);
  a.eps = static_cast<float>(number(o[6]));
  a.q_norm = integer32(fn, "q_norm", o[7]);
  a.k_norm = integer32(fn, "k_norm", o[10]);
  a.q = address(&q);
  a.k = address(&k);
  head_strides(fn, "q", q, a.q_tok_stride, a.q_head_stride);
  head_strides(fn, "k", k, a.k_tok_stride, a.k_head_stride);
  a.q_weight = vec[0];
  a.q_bias = vec[1];
  a.k_weight = vec[2];
  a.k_bias = vec[3];
  a.pos = static_cast<const int32_t *>(address(pos));
  a.cos_sin = static_cast<const float *>(address(cs));
  return a;
}

// o: the QK arguments (the last two are the stream and any), then q_out, k_out
PyObject *qk_norm_rope(PyObject *, PyObject *const *o, Py_ssize_t n_args) {
  return guarded(n_args, QK + 2, [&] {
    const char *fn = "echo_qk_norm_rope";
    const at::Tensor *q = tensor(fn, "q", o[0]), *k = tensor(fn, "k", o[1]), *qo = tensor(fn, "q_out", o[QK]),
                     *ko = tensor(fn, "k_out", o[QK + 1]);
    const Where w(fn, q);
    const echo_qk_args a = qk_args(w, *q, *k, o);
    if (qo->sizes() != q->sizes() || ko->sizes() != k->sizes() || qo->scalar_type() != q->scalar_type() ||
        ko->scalar_type() != q->scalar_type())
      refuse(fn, "q_out or k_out does not match its input");
    w.same("q_out", qo);
    w.same("k_out", ko);
    int64_t qt, qh, kt, kh;
    head_strides(fn, "q_out", *qo, qt, qh);
    head_strides(fn, "k_out", *ko, kt, kh);
    check(fn, g_rope(&a, address(qo), qt, qh, address(ko), kt, kh, w.stream(o[QK - 2], o[QK - 1] == Py_True)));
  });
}

// o: the QK arguments, then w, q8, w_out, k_cache, k_scale, slot, w_mul
PyObject *indexer_qk(PyObject *, PyObject *const *o, Py_ssize_t n_args) {
  return guarded(n_args, QK + 7, [&] {
    const char *fn = "echo_indexer_qk";
    const at::Tensor *q = tensor(fn, "q", o[0]), *k = tensor(fn, "k", o[1]), *hw = tensor(fn, "w", o[QK]),
                     *q8 = tensor(fn, "q8", o[QK + 1]), *w_out = tensor(fn, "w_out", o[QK + 2]),
                     *cache = tensor(fn, "k_cache", o[QK + 3]), *scale = tensor(fn, "k_scale", o[QK + 4]),
                     *slot = tensor(fn, "slot", o[QK + 5]);
    const Where w(fn, q);
    const echo_qk_args a = qk_args(w, *q, *k, o);
    const int64_t n = q->size(0), heads = q->size(1), slots = scale->numel();
    if (hw->scalar_type() != at::kFloat || hw->dim() != 2 || hw->size(0) != n || hw->size(1) != heads)
      refuse(fn, "w is not fp32 [tokens, heads]");
    if (heads > 1 && n && hw->stride(1) != 1) refuse(fn, "the rows of w are not contiguous");
    w.same("w", hw);
    if (!is_codes(q8->scalar_type()) || q8->sizes() != q->sizes()) refuse(fn, "q8 is not FP8 codes of q's shape");
    want(w, "q8", q8, q8->scalar_type(), -1);
    want(w, "w_out", w_out, at::kFloat, n * heads);
    if (!is_codes(cache->scalar_type())) refuse(fn, "k_cache is not FP8 codes");
    if (cache->numel() != slots * q->size(2)) refuse(fn, "k_cache and k_scale hold different numbers of keys");
    want(w, "k_cache", cache, cache->scalar_type(), -1);
    want(w, "k_scale", scale, at::kFloat, -1);
    want(w, "slot", slot, at::kLong, n);
    check(fn, g_indexer(&a, static_cast<const float *>(address(hw)), n > 1 ? hw->stride(0) : heads, static_cast<float>(number(o[QK + 6])),
                        static_cast<uint8_t *>(address(q8)), static_cast<float *>(address(w_out)),
                        static_cast<uint8_t *>(address(cache)), static_cast<float *>(address(scale)),
                        static_cast<const int64_t *>(address(slot)), slots, w.stream(o[QK - 2], o[QK - 1] == Py_True)));
  });
}

PyObject *newest_queries(PyObject *, PyObject *const *o, Py_ssize_t n_args) {
  return guarded(n_args, 9, [&] {
    const char *fn = "echo_newest_queries";
    const at::Tensor *q8 = tensor(fn, "q8", o[0]), *hw = tensor(fn, "w", o[1]), *begin = tensor(fn, "row_begin", o[2]),
                     *len = tensor(fn, "key_len", o[3]), *q_out = tensor(fn, "q_out", o[4]),
                     *w_out = tensor(fn, "w_out", o[5]), *len_out = tensor(fn, "len_out", o[6]);
    const Where w(fn, q8);
    if (!is_codes(q8->scalar_type()) || q8->dim() != 3 || q8->size(2) != ECHO_D_INDEX)
      refuse(fn, "q8 is not FP8 codes [tokens, heads, %d]", ECHO_D_INDEX);
    const int64_t n_tok = q8->size(0), heads = q8->size(1), n = len->numel();
    want(w, "q8", q8, q8->scalar_type(), -1);
    want(w, "w", hw, at::kFloat, n_tok * heads);
    want(w, "row_begin", begin, at::kInt, n + 1);
    want(w, "key_len", len, at::kInt, n);
    if (!is_codes(q_out->scalar_type())) refuse(fn, "q_out is not FP8 codes");
    want(w, "q_out", q_out, q_out->scalar_type(), n * heads * ECHO_D_INDEX);
    want(w, "w_out", w_out, at::kFloat, n * heads);
    want(w, "len_out", len_out, at::kInt, n);
    check(fn, g_newest(static_cast<const uint8_t *>(address(q8)), static_cast<const float *>(address(hw)),
                       static_cast<const int32_t *>(address(begin)), static_cast<const int32_t *>(address(len)),
                       count32(fn, n), count32(fn, n_tok), count32(fn, heads), static_cast<uint8_t *>(address(q_out)),
                       static_cast<float *>(address(w_out)), static_cast<int32_t *>(address(len_out)),
                       w.stream(o[7], o[8] == Py_True)));
  });
}

// (EchoError, raw_stream, addresses of echo_last_error, echo_page_step, echo_quant_fp8,
// echo_matmul_fp8, echo_qk_norm_rope, echo_indexer_qk, echo_newest_queries)
PyObject *setup(PyObject *, PyObject *const *o, Py_ssize_t n_args) {
  return guarded(n_args, 9, [&] {
    auto fn = [&](int i) { return reinterpret_cast<void *>(integer(o[i])); };
    Py_INCREF(o[0]);
    Py_INCREF(o[1]);
    Py_XSETREF(g_error, o[0]);
    Py_XSETREF(g_raw_stream, o[1]);
    g_last_error = reinterpret_cast<decltype(g_last_error)>(fn(2));
    g_page_step = reinterpret_cast<decltype(g_page_step)>(fn(3));
    g_quant = reinterpret_cast<decltype(g_quant)>(fn(4));
    g_matmul = reinterpret_cast<decltype(g_matmul)>(fn(5));
    g_rope = reinterpret_cast<decltype(g_rope)>(fn(6));
    g_indexer = reinterpret_cast<decltype(g_indexer)>(fn(7));
    g_newest = reinterpret_cast<decltype(g_newest)>(fn(8));
  });
}

#define CALL(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(setup), CALL(page_step), CALL(quant_fp8), CALL(matmul_fp8), CALL(qk_norm_rope),
                         CALL(indexer_qk), CALL(newest_queries), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_calls() { return PyModule_Create(&module); }
