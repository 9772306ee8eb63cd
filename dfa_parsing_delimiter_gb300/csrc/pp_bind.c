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
static PyObject *s_dtype, *s_get_device, *s_numel, *s_is_contiguous, *s_dim, *s_data_ptr;

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

static PyObject* embed_grad_scratch(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long v[3];
  if (!want(n, 3) || !numbers(a, n, v, -1, NULL)) return NULL;
  return PyLong_FromSize_t(f_scratch(SIZE(0), SIZE(1), SIZE(2)));
}

static PyObject* init(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long v[6];
  if (!want(n, 6) || !numbers(a, n, v, -1, NULL)) return NULL;
  f_vocab = (__typeof__(f_vocab))(uintptr_t)v[0];
  f_states = (__typeof__(f_states))(uintptr_t)v[1];
  f_logits = (__typeof__(f_logits))(uintptr_t)v[2];
  f_embed = (__typeof__(f_embed))(uintptr_t)v[3];
  f_grad = (__typeof__(f_grad))(uintptr_t)v[4];
  f_scratch = (__typeof__(f_scratch))(uintptr_t)v[5];
  Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {FAST(init), FAST(vec), FAST(vocab_grammar), FAST(grammar_states),
                                FAST(logits), FAST(embed), FAST(embed_grad), FAST(embed_grad_scratch),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "pp_bind", NULL, -1, methods};

PyMODINIT_FUNC PyInit_pp_bind(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_numel = PyUnicode_InternFromString("numel");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_dim = PyUnicode_InternFromString("dim");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  if (!s_dtype || !s_get_device || !s_numel || !s_is_contiguous || !s_dim || !s_data_ptr) return NULL;
  return PyModule_Create(&module);
}
