/* Argument marshalling of the language-model entry points for Python: a
 * call whose kernel takes two microseconds should not spend fifteen on its
 * arguments.  vec() checks a tensor and gives its address; token_probs,
 * verify_drafts and adamw check the tensors that they take, the others take
 * plain numbers; all call libpp, whose functions init() is given (lm.py). */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <math.h>

#include "pp.h"

static __typeof__(&pp_vocab_grammar) f_vocab;
static __typeof__(&pp_grammar_states) f_states;
static __typeof__(&pp_logits) f_logits;
static __typeof__(&pp_embed) f_embed;
static __typeof__(&pp_embed_grad_noalloc) f_grad;
static __typeof__(&pp_embed_grad_scratch) f_scratch;
static __typeof__(&pp_token_probs) f_probs;
static __typeof__(&pp_verify_drafts) f_verify;
static __typeof__(&pp_adamw) f_adamw;
static PyObject *ftypes[3], *itypes[4];  /* the dtypes of pp_ftype and pp_itype, from types() */
static PyObject *s_is_leaf, *s_shape, *s_stride, *s_dtype, *s_get_device, *s_numel, *s_is_contiguous, *s_dim, *s_data_ptr;

/* a method without arguments that gives an integer; -1 and an error set on failure */
static long long ask(PyObject* t, PyObject* name) {
  PyObject* r = PyObject_CallMethodNoArgs(t, name);
  if (!r) return -1;
  const long long v = PyLong_AsLongLong(r);
  Py_DECREF(r);
  return v;
}

static int want(Py_ssize_t n, Py_ssize_t args) {
  if (n == args) return 1;
  PyErr_Format(PyExc_TypeError, "want %zd arguments, got %zd", args, n);
  return 0;
}

/* vec(t, dtype, device, n, name): the address of a contiguous vector of at
 * least n elements on the device, 0 for None; ValueError for anything else */
static PyObject* vec(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (!want(n, 5)) return NULL;
  PyObject* t = a[0];
  if (t == Py_None) return PyLong_FromLong(0);
  PyObject* dtype = PyObject_GetAttr(t, s_dtype);
  if (!dtype) return NULL;
  int ok = dtype == a[1];
  Py_DECREF(dtype);
  ok = ok && ask(t, s_get_device) == PyLong_AsLongLong(a[2]) && ask(t, s_dim) == 1 &&
       ask(t, s_numel) >= PyLong_AsLongLong(a[3]) && ask(t, s_is_contiguous) == 1;
  if (PyErr_Occurred()) return NULL;
  if (ok) return PyObject_CallMethodNoArgs(t, s_data_ptr);
  PyErr_Format(PyExc_ValueError, "%U: want %S contiguous elements of %S on the other tensors' device", a[4], a[3], a[1]);
  return NULL;
}

/* a[0 .. n - 1] as integers; floats (at most one, at index `real`) to *x */
static int numbers(PyObject* const* a, Py_ssize_t n, long long* v, Py_ssize_t real, double* x) {
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (i == real) *x = PyFloat_AsDouble(a[i]);
    else v[i] = PyLong_AsLongLong(a[i]);
  }
  return !PyErr_Occurred();
}

static PyObject* bad(const char* what) {
  PyErr_SetString(PyExc_ValueError, what);
  return NULL;
}

/* the place of a tensor's dtype among n, or -1 */
static int kind(PyObject* t, PyObject** dtypes, int n) {
  PyObject* dtype = PyObject_GetAttr(t, s_dtype);
  if (!dtype) return -1;
  int k = n - 1;
  while (k >= 0 && dtype != dtypes[k]) --k;
  Py_DECREF(dtype);
  return k;
}

struct matrix {
  void* p;
  int type;
  long long rows, cols, stride;
};

/* a matrix of one of n dtypes on the device, with contiguous rows; ValueError for anything else */
static int matrix(PyObject* t, PyObject** dtypes, int n, long long device, const char* name, struct matrix* m) {
  m->type = kind(t, dtypes, n);
  if (PyErr_Occurred()) return 0;
  PyObject *shape = PyObject_GetAttr(t, s_shape), *stride = shape ? PyObject_CallMethodNoArgs(t, s_stride) : NULL;
  int ok = shape && stride && m->type >= 0 && ask(t, s_get_device) == device && PyTuple_Check(shape) && PyTuple_GET_SIZE(shape) == 2 &&
           PyTuple_Check(stride) && PyTuple_GET_SIZE(stride) == 2;
  if (ok) {
    m->rows = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 0));
    m->cols = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 1));
    m->stride = PyLong_AsLongLong(PyTuple_GET_ITEM(stride, 0));
    m->p = (void*)(uintptr_t)ask(t, s_data_ptr);
    ok = m->cols <= 1 || m->rows == 0 || PyLong_AsLongLong(PyTuple_GET_ITEM(stride, 1)) == 1;
  }
  Py_XDECREF(shape);
  Py_XDECREF(stride);
  if (!ok && !PyErr_Occurred()) {
    PyErr_Format(PyExc_ValueError, "%s: want 2 dimensions, the last contiguous, of %S%s on the other tensors' device, got %S", name, dtypes[0],
                 n > 1 ? " (or another of its kind)" : "", t);
    return 0;
  }
  return !PyErr_Occurred();
}

/* the address of a contiguous vector of at least n elements, NULL for None; ValueError for anything else */
static int vector(PyObject* t, PyObject* dtype, long long device, long long n, const char* name, void** p) {
  *p = NULL;
  if (t == Py_None) return 1;
  const int ok = kind(t, &dtype, 1) == 0 && ask(t, s_get_device) == device && ask(t, s_dim) == 1 && ask(t, s_numel) >= n && ask(t, s_is_contiguous) == 1;
  if (PyErr_Occurred()) return 0;
  if (!ok) {
    PyErr_Format(PyExc_ValueError, "%s: want %lld contiguous elements of %S on the other tensors' device", name, n, dtype);
    return 0;
  }
  *p = (void*)(uintptr_t)ask(t, s_data_ptr);
  return !PyErr_Occurred();
}

#define PTR(i) ((void*)(uintptr_t)v[i])
#define SIZE(i) ((size_t)v[i])
#define CALL(x)               \
  pp_rc rc;                   \
  Py_BEGIN_ALLOW_THREADS      \
  rc = x;                     \
  Py_END_ALLOW_THREADS        \
  return PyLong_FromLong(rc)

static PyObject* vocab_grammar(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long v[10];
  if (!want(n, 10) || !numbers(a, n, v, -1, NULL)) return NULL;
  CALL(f_vocab(PTR(0), PTR(1), SIZE(2), SIZE(3), PTR(4), v[5], PTR(6), PTR(7), SIZE(8), PTR(9)));
}

static PyObject* grammar_states(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long v[15];
  if (!want(n, 15) || !numbers(a, n, v, -1, NULL)) return NULL;
  CALL(f_states(PTR(0), SIZE(1), (int)v[2], PTR(3), (pp_itype)v[4], SIZE(5), SIZE(6), SIZE(7), PTR(8), PTR(9), SIZE(10),
                (uint8_t)v[11], PTR(12), SIZE(13), PTR(14)));
}

/* in, type, rows, vocab, in_stride, the 20 fields of pp_logit_opts in order, out, out_stride, stream */
static PyObject* logits(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long v[28];
  if (!want(n, 28) || !numbers(a, n, v, -1, NULL)) return NULL;
  const pp_logit_opts o = {PTR(5), PTR(6), PTR(7), PTR(8), SIZE(9), SIZE(10), SIZE(11), PTR(12), PTR(13), PTR(14),
                           PTR(15), PTR(16), PTR(17), SIZE(18), PTR(19), SIZE(20), PTR(21), SIZE(22), (int32_t)v[23],
                           (int32_t)v[24]};
  CALL(f_logits(PTR(0), (pp_ftype)v[1], SIZE(2), SIZE(3), SIZE(4), &o, PTR(25), SIZE(26), PTR(27)));
}

static PyObject* embed(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long v[15];
  double scale = 0;
  if (!want(n, 15) || !numbers(a, n, v, 9, &scale)) return NULL;
  CALL(f_embed(PTR(0), (pp_itype)v[1], SIZE(2), SIZE(3), PTR(4), (pp_ftype)v[5], SIZE(6), SIZE(7), SIZE(8), (float)scale,
               v[10], PTR(11), (pp_ftype)v[12], SIZE(13), PTR(14)));
}

static PyObject* embed_grad(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long v[18];
  double scale = 0;
  if (!want(n, 18) || !numbers(a, n, v, 9, &scale)) return NULL;
  CALL(f_grad(PTR(0), (pp_itype)v[1], SIZE(2), SIZE(3), PTR(4), (pp_ftype)v[5], SIZE(6), SIZE(7), SIZE(8), (float)scale,
              v[10], (int)v[11], PTR(12), (pp_ftype)v[13], SIZE(14), PTR(15), SIZE(16), PTR(17)));
}

/* logits, temperature, top_k, out, stream: a result of the logits' shape */
static PyObject* token_probs(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (!want(n, 5)) return NULL;
  const long long device = ask(a[0], s_get_device), stream = PyLong_AsLongLong(a[4]);
  struct matrix x, p;
  void *t, *k;
  if (PyErr_Occurred() || !matrix(a[0], ftypes, 3, device, "logits", &x) || !matrix(a[3], ftypes, 1, device, "out", &p)) return NULL;
  if (p.rows != x.rows || p.cols != x.cols) return bad("out: want the shape of the logits");
  if (!vector(a[1], ftypes[0], device, x.rows, "temperature", &t) || !vector(a[2], itypes[2], device, x.rows, "top_k", &k)) return NULL;
  CALL(f_probs(x.p, (pp_ftype)x.type, x.rows, x.cols, x.stride, t, k, p.p, p.stride, (cudaStream_t)(uintptr_t)stream));
}

/* target, drafts, accept, sample, draft_probs, lengths, target_row, draft_row, tokens, counts, stream */
static PyObject* verify_drafts(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (!want(n, 11)) return NULL;
  const long long device = ask(a[0], s_get_device), stream = PyLong_AsLongLong(a[10]);
  struct matrix p, d, u, q = {NULL, 0, 0, 0, 0}, out;
  void *sample, *lengths, *row, *qrow, *counts;
  if (PyErr_Occurred() || !matrix(a[0], ftypes, 3, device, "target", &p) || !matrix(a[1], itypes, 4, device, "drafts", &d) ||
      !matrix(a[2], ftypes, 1, device, "accept", &u) || !matrix(a[8], itypes + 2, 1, device, "out", &out))
    return NULL;
  const long long many = d.rows, drafts = d.cols;
  if (p.cols < 1) return bad("target: want a token at least");
  if (u.rows != many || u.cols != drafts) return bad("accept: want a number for each draft");
  if (out.rows != many || out.cols != drafts + 1) return bad("out: want tokens, one column more than drafts, and a count for each request");
  if (a[6] == Py_None && p.rows < many * (drafts + 1)) return bad("target: want a row for each draft and one more a request");
  if (a[4] != Py_None) {
    if (!matrix(a[4], ftypes + p.type, 1, device, "draft_probs", &q)) return NULL;
    if (q.cols != p.cols) return bad("draft_probs: want the target's vocabulary");
    if (a[7] == Py_None && q.rows < many * drafts) return bad("draft_probs: want a row for each draft");
    if (!q.p) q.p = p.p; /* no rows have no address, and are still not those of sure drafts */
  }
  if (!vector(a[3], ftypes[0], device, many, "sample", &sample) || !vector(a[5], itypes[2], device, many, "lengths", &lengths) ||
      !vector(a[6], itypes[2], device, many, "target_row", &row) || !vector(a[7], itypes[2], device, many, "draft_row", &qrow) ||
      !vector(a[9], itypes[2], device, many, "out's counts", &counts))
    return NULL;
  if (!sample && many) return bad("sample: want a number for each request");
  const pp_draft_opts o = {q.p, qrow, q.rows, q.stride, row, lengths};
  CALL(f_verify(p.p, (pp_ftype)p.type, p.rows, p.cols, p.stride, d.p, (pp_itype)d.type, many, drafts, d.stride, u.p, u.stride, sample,
                &o, out.p, out.stride, counts, (cudaStream_t)(uintptr_t)stream));
}

/* a contiguous floating tensor of n elements on the device: its address and type */
static int tensor_of(PyObject* t, long long device, unsigned long long n, void** p, int32_t* type) {
  *type = kind(t, ftypes, 3);
  if (*type < 0) return 0;
  if (ask(t, s_get_device) != device || (unsigned long long)ask(t, s_numel) != n || ask(t, s_is_contiguous) != 1) return 0;
  *p = (void*)(uintptr_t)ask(t, s_data_ptr);
  return !PyErr_Occurred();
}

static int same_twice(const pp_adamw_tensor* t, size_t n) {
  size_t size = 4;
  while (size < 2 * n) size *= 2;
  void** seen = PyMem_Calloc(size, sizeof *seen);
  if (!seen) return PyErr_NoMemory(), 1;
  int twice = 0;
  for (size_t i = 0; i < n && !twice; ++i) {
    if (!t[i].n) continue;
    size_t at = ((uintptr_t)t[i].d_param >> 4) * 0x9E3779B97F4A7C15u >> 20 & (size - 1);
    while (seen[at] && seen[at] != t[i].d_param) at = (at + 1) & (size - 1);
    twice = seen[at] != NULL;
    seen[at] = t[i].d_param;
  }
  PyMem_Free(seen);
  if (twice) PyErr_SetString(PyExc_ValueError, "params: the same tensor twice");
  return twice;
}

/* params, grads (None: left out), their elements, their places, weight decays (a number or a sequence), device, then the
 * ten fields of pp_adamw_state and the seven of pp_adamw_opts in order, stream */
static PyObject* adamw(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (!want(n, 24)) return NULL;
  PyObject* seq[5] = {NULL};
  pp_adamw_tensor* t = NULL;
  PyObject* result = NULL;
  const int one = PyFloat_Check(a[4]) || PyLong_Check(a[4]) || (PyNumber_Check(a[4]) && !PySequence_Check(a[4]));
  for (int k = 0; k < (one ? 4 : 5); ++k)
    if (!(seq[k] = PySequence_Fast(a[k], "want sequences of tensors and numbers"))) goto done;
  const Py_ssize_t count = PySequence_Fast_GET_SIZE(seq[2]);
  for (int k = 0; k < (one ? 4 : 5); ++k)
    if (PySequence_Fast_GET_SIZE(seq[k]) != count) {
      static const char* const what[] = {"params", "grads", "sizes", "places", "weight_decay"};
      PyErr_Format(PyExc_ValueError, "%s: want %zd, one for each tensor of the state, got %zd", what[k], count, PySequence_Fast_GET_SIZE(seq[k]));
      goto done;
    }
  long long v[24] = {0};
  double real[4];
  for (int i = 5; i < 24; ++i) {
    if (i >= 16 && i < 20) real[i - 16] = PyFloat_AsDouble(a[i]);
    else v[i] = PyLong_AsLongLong(a[i]);
  }
  const double decay = one ? PyFloat_AsDouble(a[4]) : 0;
  if (PyErr_Occurred()) goto done;
  if (!(t = PyMem_Calloc(count ? count : 1, sizeof *t))) {
    PyErr_NoMemory();
    goto done;
  }
  size_t used = 0;
  for (Py_ssize_t i = 0; i < count; ++i) {
    PyObject *p = PySequence_Fast_GET_ITEM(seq[0], i), *g = PySequence_Fast_GET_ITEM(seq[1], i);
    if (g == Py_None) continue;
    pp_adamw_tensor* e = &t[used];
    e->n = PyLong_AsUnsignedLongLong(PySequence_Fast_GET_ITEM(seq[2], i));
    e->first = PyLong_AsUnsignedLongLong(PySequence_Fast_GET_ITEM(seq[3], i));
    e->weight_decay = (float)(one ? decay : PyFloat_AsDouble(PySequence_Fast_GET_ITEM(seq[4], i)));
    void* grad = NULL;
    const int fine = !PyErr_Occurred() && tensor_of(p, v[5], e->n, &e->d_param, &e->param_type) &&
                     tensor_of(g, v[5], e->n, &grad, &e->grad_type);
    if (PyErr_Occurred()) goto done;
    if (!isfinite(e->weight_decay)) {
      PyErr_Format(PyExc_ValueError, "weight_decay: want a number that 32 bits hold (tensor %zd)", i);
      goto done;
    }
    if (!fine) {
      PyErr_Format(PyExc_ValueError, "params and grads: want %llu contiguous elements of float32, float16 or bfloat16 on the state's device (tensor %zd)", (unsigned long long)e->n, i);
      goto done;
    }
    PyObject* leaf = PyObject_GetAttr(p, s_is_leaf);
    if (!leaf) goto done;
    Py_DECREF(leaf);
    if (leaf == Py_False) {
      PyErr_Format(PyExc_ValueError, "params: want leaves of the graph (tensor %zd)", i);
      goto done;
    }
    e->d_grad = grad;
    ++used;
  }
  if (same_twice(t, used)) goto done;
  {
    const pp_adamw_state s = {PTR(6), PTR(7), PTR(8), PTR(9), PTR(10), PTR(11), (uint64_t)v[12], (int32_t)v[13], (uint32_t)v[14],
                              (int32_t)v[15]};
    const pp_adamw_opts o = {real[0], real[1], real[2], real[3], PTR(20), PTR(21), PTR(22)};
    pp_rc rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f_adamw(t, used, &s, &o, PTR(23));
    Py_END_ALLOW_THREADS
    result = PyLong_FromLong(rc);
  }
done:
  PyMem_Free(t);
  for (int k = 0; k < 5; ++k) Py_XDECREF(seq[k]);
  return result;
}

static PyObject* types(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (!want(n, 7)) return NULL;
  for (int k = 0; k < 7; ++k) {
    Py_INCREF(a[k]);
    if (k < 3) Py_XSETREF(ftypes[k], a[k]);
    else Py_XSETREF(itypes[k - 3], a[k]);
  }
  Py_RETURN_NONE;
}

static PyObject* embed_grad_scratch(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long v[3];
  if (!want(n, 3) || !numbers(a, n, v, -1, NULL)) return NULL;
  return PyLong_FromSize_t(f_scratch(SIZE(0), SIZE(1), SIZE(2)));
}

static PyObject* init(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long v[9];
  if (!want(n, 9) || !numbers(a, n, v, -1, NULL)) return NULL;
  f_vocab = (__typeof__(f_vocab))(uintptr_t)v[0];
  f_states = (__typeof__(f_states))(uintptr_t)v[1];
  f_logits = (__typeof__(f_logits))(uintptr_t)v[2];
  f_embed = (__typeof__(f_embed))(uintptr_t)v[3];
  f_grad = (__typeof__(f_grad))(uintptr_t)v[4];
  f_scratch = (__typeof__(f_scratch))(uintptr_t)v[5];
  f_probs = (__typeof__(f_probs))(uintptr_t)v[6];
  f_verify = (__typeof__(f_verify))(uintptr_t)v[7];
  f_adamw = (__typeof__(f_adamw))(uintptr_t)v[8];
  Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {FAST(init), FAST(vec), FAST(vocab_grammar), FAST(grammar_states),
                                FAST(logits), FAST(embed), FAST(embed_grad), FAST(embed_grad_scratch),
                                FAST(types), FAST(token_probs), FAST(verify_drafts), FAST(adamw),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "pp_bind", NULL, -1, methods};

PyMODINIT_FUNC PyInit_pp_bind(void) {
  s_is_leaf = PyUnicode_InternFromString("is_leaf");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_dtype = PyUnicode_InternFromString("dtype");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_numel = PyUnicode_InternFromString("numel");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_dim = PyUnicode_InternFromString("dim");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  if (!s_is_leaf || !s_shape || !s_stride || !s_dtype || !s_get_device || !s_numel || !s_is_contiguous || !s_dim || !s_data_ptr) return NULL;
  return PyModule_Create(&module);
}
