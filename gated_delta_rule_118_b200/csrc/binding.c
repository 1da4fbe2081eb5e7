/*
 * binding.c -- calls of the hybrid block's entry points from Python (module _call).
 *
 * The same calls can be made through ctypes, which takes 2 to 4 microseconds to
 * convert the arguments of one; for a single decoded token that is as long as the
 * kernel.  The module holds the addresses of libgdn2.so's functions (given once by
 * init, so that both ways use one loaded library) and converts plain integers,
 * floats, None (a null pointer) and tuples of strides.  Every function returns the
 * status code.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "gdn2.h"

static const char *const kNames[] = {"gdn2_swa_fwd", "gdn2_swa_bwd", "gdn2_swa_decode", "gdn2_scan_fwd",
                                     "gdn2_scan_bwd", "gdn2_scan_step", "gdn2_block_norm_fwd", "gdn2_block_norm_bwd"};
enum { SWA_FWD, SWA_BWD, SWA_DECODE, SCAN_FWD, SCAN_BWD, SCAN_STEP, NORM_FWD, NORM_BWD, COUNT };
static void *fn[COUNT];

static void *ptr(PyObject *o) { return o == Py_None ? NULL : PyLong_AsVoidPtr(o); }
static int num(PyObject *o)
{
    const long v = PyLong_AsLong(o);
    if ((v > 0x7fffffffL || v < -0x7fffffffL - 1) && !PyErr_Occurred())
        PyErr_SetString(PyExc_OverflowError, "a size does not fit 32 bits");
    return (int)v;
}
static float real(PyObject *o) { return (float)PyFloat_AsDouble(o); }
static const long long *strides(PyObject *o, long long *buf, int n)
{
    if (o == Py_None) return NULL;
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != n) {
        PyErr_SetString(PyExc_TypeError, "strides must be a tuple of the expected length");
        return NULL;
    }
    for (int i = 0; i < n; ++i) buf[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(o, i));
    return buf;
}
static int ready(int which, Py_ssize_t got, Py_ssize_t want)
{
    if (!fn[which]) {
        PyErr_SetString(PyExc_RuntimeError, "_call.init has not been called");
        return 0;
    }
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", kNames[which], want, got);
        return 0;
    }
    return 1;
}

#define P(i) void *p##i = ptr(a[i])
#define I(i) int p##i = num(a[i])
#define F(i) float p##i = real(a[i])
#define CALL(which, ...)                                                   \
    gdn2_status st;                                                        \
    if (PyErr_Occurred()) return NULL;                                     \
    Py_BEGIN_ALLOW_THREADS st = ((__typeof__(&which))f)(__VA_ARGS__);      \
    Py_END_ALLOW_THREADS return PyLong_FromLong((long)st);

static PyObject *init(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    if (n != COUNT) {
        PyErr_SetString(PyExc_TypeError, "init takes one address per function");
        return NULL;
    }
    for (int i = 0; i < COUNT; ++i) fn[i] = ptr(a[i]);
    if (PyErr_Occurred()) return NULL;
    Py_RETURN_NONE;
}

static PyObject *swa_fwd(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    void *f = fn[SWA_FWD];
    long long buf[9];
    if (!ready(SWA_FWD, n, 18)) return NULL;
    P(0); P(1); P(2); P(3); P(4); P(5); I(6); I(7); I(8); I(9); I(10); I(11); I(12); I(13); F(14); I(16); P(17);
    const long long *s = strides(a[15], buf, 9);
    CALL(gdn2_swa_fwd, p0, p1, p2, p3, p4, p5, p6, p7, p8, p9, p10, p11, p12, p13, p14, s, (gdn2_dtype)p16, p17)
}

static PyObject *swa_bwd(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    void *f = fn[SWA_BWD];
    long long buf[9];
    if (!ready(SWA_BWD, n, 22)) return NULL;
    P(0); P(1); P(2); P(3); P(4); P(5); P(6); P(7); P(8); P(9);
    I(10); I(11); I(12); I(13); I(14); I(15); I(16); I(17); F(18); I(20); P(21);
    const long long *s = strides(a[19], buf, 9);
    CALL(gdn2_swa_bwd, p0, p1, p2, p3, p4, p5, p6, p7, p8, p9, p10, p11, p12, p13, p14, p15, p16, p17, p18, s,
         (gdn2_dtype)p20, p21)
}

static PyObject *swa_decode(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    void *f = fn[SWA_DECODE];
    long long buf[6];
    if (!ready(SWA_DECODE, n, 18)) return NULL;
    P(0); P(1); P(2); P(3); P(4); P(5); P(6); I(7); I(8); I(9); I(10); I(11); I(12); I(13); F(14); I(16); P(17);
    const long long *s = strides(a[15], buf, 6);
    CALL(gdn2_swa_decode, p0, p1, p2, p3, p4, p5, p6, p7, p8, p9, p10, p11, p12, p13, p14, s, (gdn2_dtype)p16, p17)
}

static PyObject *scan_fwd(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    void *f = fn[SCAN_FWD];
    if (!ready(SCAN_FWD, n, 12)) return NULL;
    P(0); P(1); P(2); P(3); P(4); P(5); P(6); I(7); I(8); I(9); I(10); P(11);
    CALL(gdn2_scan_fwd, p0, p1, p2, p3, p4, p5, p6, p7, p8, p9, (gdn2_dtype)p10, p11)
}

static PyObject *scan_bwd(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    void *f = fn[SCAN_BWD];
    if (!ready(SCAN_BWD, n, 15)) return NULL;
    P(0); P(1); P(2); P(3); P(4); P(5); P(6); P(7); P(8); P(9); I(10); I(11); I(12); I(13); P(14);
    CALL(gdn2_scan_bwd, p0, p1, p2, p3, p4, p5, p6, p7, p8, p9, p10, p11, p12, (gdn2_dtype)p13, p14)
}

static PyObject *scan_step(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    void *f = fn[SCAN_STEP];
    if (!ready(SCAN_STEP, n, 9)) return NULL;
    P(0); P(1); P(2); P(3); P(4); I(5); I(6); I(7); P(8);
    CALL(gdn2_scan_step, p0, p1, p2, p3, p4, p5, p6, (gdn2_dtype)p7, p8)
}

static PyObject *block_norm_fwd(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    void *f = fn[NORM_FWD];
    if (!ready(NORM_FWD, n, 13)) return NULL;
    P(0); P(1); P(2); P(3); P(4); P(5); F(6); P(7); P(8);
    const long long rows = PyLong_AsLongLong(a[9]);
    I(10); I(11); P(12);
    CALL(gdn2_block_norm_fwd, p0, p1, p2, p3, p4, p5, p6, p7, p8, rows, p10, (gdn2_dtype)p11, p12)
}

static PyObject *block_norm_bwd(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    void *f = fn[NORM_BWD];
    if (!ready(NORM_BWD, n, 19)) return NULL;
    P(0); P(1); P(2); P(3); P(4); P(5); F(6); P(7); P(8); P(9); P(10); P(11); P(12); P(13); P(14);
    const long long rows = PyLong_AsLongLong(a[15]);
    I(16); I(17); P(18);
    CALL(gdn2_block_norm_bwd, p0, p1, p2, p3, p4, p5, p6, p7, p8, p9, p10, p11, p12, p13, p14, rows, p16,
         (gdn2_dtype)p17, p18)
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {METHOD(init), METHOD(swa_fwd), METHOD(swa_bwd), METHOD(swa_decode), METHOD(scan_fwd),
                                METHOD(scan_bwd), METHOD(scan_step), METHOD(block_norm_fwd), METHOD(block_norm_bwd),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_call", "Calls of libgdn2.so.", -1, methods,
                                    NULL, NULL, NULL, NULL};
PyMODINIT_FUNC PyInit__call(void) { return PyModule_Create(&module); }
