/* Argument marshalling of the language-model entry points for Python: a
 * call whose kernel takes two microseconds should not spend fifteen on its
 * arguments.  vec() checks a tensor and gives its address; the others take
 * plain numbers and call libpp, whose functions init() is given (lm.py). */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

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
static PyObject* ftypes[3];  /* the dtypes of pp_ftype, from types() */
static PyObject *s_is_leaf, *s_dtype, *s_get_device, *s_numel, *s_is_contiguous, *s_dim, *s_data_ptr;

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

static PyObject* token_probs(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long v[10];
  if (!want(n, 10) || !numbers(a, n, v, -1, NULL)) return NULL;
  CALL(f_probs(PTR(0), (pp_ftype)v[1], SIZE(2), SIZE(3), SIZE(4), PTR(5), PTR(6), PTR(7), SIZE(8), PTR(9)));
}

/* pp_verify_drafts' arguments, with the six fields of pp_draft_opts in its place */
static PyObject* verify_drafts(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long v[23];
  if (!want(n, 23) || !numbers(a, n, v, -1, NULL)) return NULL;
  const pp_draft_opts o = {PTR(13), PTR(14), SIZE(15), SIZE(16), PTR(17), PTR(18)};
  CALL(f_verify(PTR(0), (pp_ftype)v[1], SIZE(2), SIZE(3), SIZE(4), PTR(5), (pp_itype)v[6], SIZE(7), SIZE(8), SIZE(9),
                PTR(10), SIZE(11), PTR(12), &o, PTR(19), SIZE(20), PTR(21), PTR(22)));
}

/* the pp_ftype of a tensor, or -1 */
static int ftype(PyObject* t) {
  PyObject* dtype = PyObject_GetAttr(t, s_dtype);
  if (!dtype) return -1;
  int k = 2;
  while (k >= 0 && dtype != ftypes[k]) --k;
  Py_DECREF(dtype);
  return k;
}

/* a contiguous floating tensor of n elements on the device: its address and type */
static int tensor_of(PyObject* t, long long device, unsigned long long n, void** p, int32_t* type) {
  *type = ftype(t);
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
  const int one = PyFloat_Check(a[4]) || PyLong_Check(a[4]);
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
  if (!want(n, 3)) return NULL;
  for (int k = 0; k < 3; ++k) {
    Py_INCREF(a[k]);
    Py_XSETREF(ftypes[k], a[k]);
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
  s_dtype = PyUnicode_InternFromString("dtype");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_numel = PyUnicode_InternFromString("numel");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_dim = PyUnicode_InternFromString("dim");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  if (!s_is_leaf || !s_dtype || !s_get_device || !s_numel || !s_is_contiguous || !s_dim || !s_data_ptr) return NULL;
  return PyModule_Create(&module);
}
