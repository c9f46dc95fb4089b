/* q8_bind.c -- the Python side of the operators on rows in 8 bits.
 *
 * A serving loop makes these calls with a row or a few, where a kernel takes
 * 3 to 6 microseconds and the call's own cost shows: marshalling a dozen
 * arguments through ctypes took 1.5 of them, this module takes 0.5.  It
 * converts the arguments (numbers, type letters, device tensors or addresses,
 * the stream) and calls the C ABI; what that refuses raises XsymvError.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/xsymv.h"

static PyObject *error_class;   /* XsymvError(name, code) */
static PyObject *current;       /* the current stream's handle, called without arguments */
static PyObject *s_data_ptr, *s_cuda_stream;

/* Positions of a call's arguments that could not be converted are reported by
 * the exception itself; `ok` drops to 0 and the rest is skipped. */
static int number(PyObject *o, int *ok)
{
    if (!*ok) return 0;
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) {
        *ok = 0;
    } else if (v > 2147483647L || v < -2147483647L - 1) {
        PyErr_SetString(PyExc_OverflowError, "an argument is outside the C int range");
        *ok = 0;
    }
    return (int)v;
}

static void *address(PyObject *o, int *ok)
{
    if (!*ok || o == Py_None) return NULL;
    if (PyLong_Check(o)) {
        void *p = PyLong_AsVoidPtr(o);
        if (p == NULL && PyErr_Occurred()) *ok = 0;
        return p;
    }
    PyObject *r = PyObject_CallMethodNoArgs(o, s_data_ptr);
    if (r == NULL) {
        *ok = 0;
        return NULL;
    }
    void *p = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    if (p == NULL && PyErr_Occurred()) *ok = 0;
    return p;
}

static char letter(PyObject *o, int *ok)
{
    if (!*ok) return 0;
    Py_ssize_t len = 0;
    const char *s = NULL;
    if (PyUnicode_Check(o)) {
        s = PyUnicode_AsUTF8AndSize(o, &len);
    } else if (PyBytes_Check(o)) {
        s = PyBytes_AS_STRING(o);
        len = PyBytes_GET_SIZE(o);
    } else {
        PyErr_SetString(PyExc_TypeError, "a type letter is a string");
    }
    if (s == NULL) *ok = 0;
    return s != NULL && len > 0 ? s[0] : 0;
}

static float real(PyObject *o, int *ok)
{
    if (!*ok) return 0.0f;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) *ok = 0;
    return (float)v;
}

static void *stream_of(PyObject *o, int *ok)
{
    if (!*ok) return NULL;
    PyObject *r;
    if (o == Py_None) {
        r = PyObject_CallNoArgs(current);
    } else if (PyLong_Check(o)) {
        Py_INCREF(o);
        r = o;
    } else {
        r = PyObject_GetAttr(o, s_cuda_stream);
    }
    if (r == NULL) {
        *ok = 0;
        return NULL;
    }
    void *p = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    if (p == NULL && PyErr_Occurred()) *ok = 0;
    return p;
}

static PyObject *outcome(const char *name, int rc)
{
    if (rc == 0) Py_RETURN_NONE;
    PyObject *e = PyObject_CallFunction(error_class, "si", name, rc);
    if (e != NULL) {
        PyErr_SetObject(error_class, e);
        Py_DECREF(e);
    }
    return NULL;
}

static int counted(const char *name, Py_ssize_t n, Py_ssize_t want)
{
    if (n == want) return 1;
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments and a stream", name, want - 1);
    return 0;
}

#define NUM(i) number(a[i], &ok)
#define PTR(i) address(a[i], &ok)
/* Evaluates the arguments in order, then the call without the interpreter's lock. */
#define CALL(NAME, ARGS)                 \
    int rc = 0;                          \
    if (!ok) return NULL;                \
    Py_BEGIN_ALLOW_THREADS rc = NAME ARGS; \
    Py_END_ALLOW_THREADS return outcome(#NAME, rc)

#define OPERATORS(L, T)                                                                           \
    static PyObject *norm_##L(PyObject *self, PyObject *const *a, Py_ssize_t n)                   \
    {                                                                                             \
        int ok = 1;                                                                               \
        if (!counted("xsymv_q8norm_" #L, n, 16)) return NULL;                                     \
        const int m = NUM(0), k = NUM(1);                                                         \
        const void *x = PTR(2);                                                                   \
        const int ldx = NUM(3);                                                                   \
        const char rt = letter(a[4], &ok);                                                        \
        const void *r = PTR(5);                                                                   \
        const int ldr = NUM(6);                                                                   \
        const char wt = letter(a[7], &ok);                                                        \
        const void *w = PTR(8);                                                                   \
        const float eps = real(a[9], &ok);                                                        \
        void *h = PTR(10);                                                                        \
        const int ldh = NUM(11);                                                                  \
        void *q = PTR(12);                                                                        \
        const int ldq = NUM(13);                                                                  \
        void *sc = PTR(14), *st = stream_of(a[15], &ok);                                          \
        CALL(xsymv_q8norm_##L, (m, k, x, ldx, rt, r, ldr, wt, w, eps, h, ldh, q, ldq, sc, st));   \
    }                                                                                             \
    static PyObject *glu_##L(PyObject *self, PyObject *const *a, Py_ssize_t n)                    \
    {                                                                                             \
        int ok = 1;                                                                               \
        if (!counted("xsymv_q8glu_" #L, n, 10)) return NULL;                                      \
        const int m = NUM(0), k = NUM(1);                                                         \
        const void *g = PTR(2);                                                                   \
        const int ldg = NUM(3);                                                                   \
        const void *u = PTR(4);                                                                   \
        const int ldu = NUM(5);                                                                   \
        void *q = PTR(6);                                                                         \
        const int ldq = NUM(7);                                                                   \
        void *sc = PTR(8), *st = stream_of(a[9], &ok);                                            \
        CALL(xsymv_q8glu_##L, (m, k, g, ldg, u, ldu, q, ldq, sc, st));                            \
    }                                                                                             \
    static PyObject *store_##L(PyObject *self, PyObject *const *a, Py_ssize_t n)                  \
    {                                                                                             \
        int ok = 1;                                                                               \
        if (!counted("xsymv_q8store_" #L, n, 10)) return NULL;                                    \
        const int m = NUM(0), k = NUM(1);                                                         \
        const void *x = PTR(2);                                                                   \
        const int ldx = NUM(3);                                                                   \
        const void *slot = PTR(4);                                                                \
        const int cap = NUM(5);                                                                   \
        void *q = PTR(6);                                                                         \
        const int ldq = NUM(7);                                                                   \
        void *sc = PTR(8), *st = stream_of(a[9], &ok);                                            \
        CALL(xsymv_q8store_##L, (m, k, x, ldx, slot, cap, q, ldq, sc, st));                       \
    }                                                                                             \
    static PyObject *read_##L(PyObject *self, PyObject *const *a, Py_ssize_t n)                   \
    {                                                                                             \
        int ok = 1;                                                                               \
        if (!counted("xsymv_q8read_" #L, n, 10)) return NULL;                                     \
        const int m = NUM(0), k = NUM(1);                                                         \
        const void *q = PTR(2);                                                                   \
        const int ldq = NUM(3);                                                                   \
        const void *sc = PTR(4), *slot = PTR(5);                                                  \
        const int cap = NUM(6);                                                                   \
        void *out = PTR(7);                                                                       \
        const int ldo = NUM(8);                                                                   \
        void *st = stream_of(a[9], &ok);                                                          \
        CALL(xsymv_q8read_##L, (m, k, q, ldq, sc, slot, cap, out, ldo, st));                      \
    }                                                                                             \
    static PyObject *gemm_##L(PyObject *self, PyObject *const *a, Py_ssize_t n)                   \
    {                                                                                             \
        int ok = 1;                                                                               \
        if (!counted("xsymv_q8gemm_" #L, n, 13)) return NULL;                                     \
        const int m = NUM(0), cols = NUM(1), k = NUM(2);                                          \
        const void *q = PTR(3);                                                                   \
        const int lda = NUM(4);                                                                   \
        const void *sa = PTR(5), *w = PTR(6);                                                     \
        const int ldw = NUM(7);                                                                   \
        const void *sw = PTR(8), *bias = PTR(9);                                                  \
        void *c = PTR(10);                                                                        \
        const int ldc = NUM(11);                                                                  \
        void *st = stream_of(a[12], &ok);                                                         \
        CALL(xsymv_q8gemm_##L, (m, cols, k, q, lda, sa, w, ldw, sw, bias, c, ldc, st));           \
    }

OPERATORS(s, float)
OPERATORS(h, xhalf)
OPERATORS(b, xbfloat16)

static PyObject *setup(PyObject *self, PyObject *args)
{
    PyObject *e, *c;
    if (!PyArg_ParseTuple(args, "OO", &e, &c)) return NULL;
    Py_INCREF(e);
    Py_INCREF(c);
    Py_XDECREF(error_class);
    Py_XDECREF(current);
    error_class = e;
    current = c;
    Py_RETURN_NONE;
}

#define ENTRIES(L)                                                   \
    {"norm_" #L, (PyCFunction)(void *)norm_##L, METH_FASTCALL, 0},   \
    {"glu_" #L, (PyCFunction)(void *)glu_##L, METH_FASTCALL, 0},     \
    {"store_" #L, (PyCFunction)(void *)store_##L, METH_FASTCALL, 0}, \
    {"read_" #L, (PyCFunction)(void *)read_##L, METH_FASTCALL, 0},   \
    {"gemm_" #L, (PyCFunction)(void *)gemm_##L, METH_FASTCALL, 0}

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, "setup(error class, function giving the current stream)"},
    ENTRIES(s), ENTRIES(h), ENTRIES(b),
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_q8_bind", NULL, -1, methods};

PyMODINIT_FUNC PyInit__q8_bind(void)
{
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    if (s_data_ptr == NULL || s_cuda_stream == NULL) return NULL;
    return PyModule_Create(&module);
}
