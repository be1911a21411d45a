/* Argument marshalling of the rotary write, the scored attention and the
 * eviction for CPython: the tensors' checks and the C call in one step.
 *
 * A small call's time is its marshalling: ten tensors' type, device,
 * contiguity and address through the interpreter and ctypes take longer than
 * the kernels.  Here each tensor costs four look-ups of its own methods
 * (torch's headers are not needed), and the entry points of include/pkv.h are
 * called through their addresses, which the binding passes in.
 *
 *   setup(bfloat16, int32, int64, float32, uint8)    torch's dtype objects
 *   call(which, address, device, *arguments) -> pkv_status, or -(i + 1) when
 *       argument i is not a tensor of its type on that device (contiguous,
 *       but for the rotary write's rows): the binding then says what is wrong.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <limits.h>
#include <stdint.h>

#include "../../include/pkv.h"

enum { MAX_ARGS = 32 };

static const char g_letters[] = "bilfu";
static PyObject *g_dtype[5]; /* b: bfloat16, i: int32, l: int64, f: float32, u: uint8 */
static PyObject *s_dtype, *s_get_device, *s_is_contiguous, *s_data_ptr;

/* One letter an argument of the C call (the stream last): b, i, l, f, u a
 * contiguous tensor of that type (upper case: or None), r a bfloat16 tensor
 * with strides of its own, n an int, q an int64, x the scale, s bytes or
 * None, p an address or None. */
static const char *const g_specs[] = {
    "rrrrqqqqbblinsfqnnnnnnqIq", /* pkv_rope_kv_write */
    "bbBBbbininnnnqxFfqnnpqIq",  /* pkv_paged_attention_decode_scored */
    "bbnbbiniinnnnnqxFfqnpqIq",  /* pkv_paged_attention_prefill_scored */
    "bbiniinifqfqinnnnnqIq",     /* pkv_evict_tokens */
};

typedef union {
    int64_t i;
    void *p;
} slot;

static int raise_not_setup(void) {
    PyErr_SetString(PyExc_RuntimeError, "marshal.setup has not been called");
    return -1;
}

/* 1: converted; 0: not such a tensor; -1: a Python error. */
static int tensor_arg(PyObject *t, PyObject *dtype, int contiguous, long dev, void **out) {
    PyObject *x = PyObject_GetAttr(t, s_dtype);
    if (!x) {
        if (!PyErr_ExceptionMatches(PyExc_AttributeError)) return -1;
        PyErr_Clear();
        return 0;
    }
    Py_DECREF(x);
    if (x != dtype) return 0; /* torch's dtypes are singletons */
    x = PyObject_CallMethodNoArgs(t, s_get_device);
    if (!x) return -1;
    const long d = PyLong_AsLong(x);
    Py_DECREF(x);
    if (d == -1 && PyErr_Occurred()) return -1;
    if (d != dev) return 0;
    if (contiguous) {
        x = PyObject_CallMethodNoArgs(t, s_is_contiguous);
        if (!x) return -1;
        Py_DECREF(x);
        if (x != Py_True) return 0;
    }
    x = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!x) return -1;
    *out = PyLong_AsVoidPtr(x);
    Py_DECREF(x);
    return *out == NULL && PyErr_Occurred() ? -1 : 1;
}

static int int_arg(PyObject *o, int is_int, int64_t *out) {
    PyObject *i = PyNumber_Index(o);
    if (!i) return -1;
    *out = PyLong_AsLongLong(i);
    Py_DECREF(i);
    if (*out == -1 && PyErr_Occurred()) return -1;
    if (is_int && (*out < INT_MIN || *out > INT_MAX)) {
        PyErr_SetString(PyExc_OverflowError, "argument does not fit in an int");
        return -1;
    }
    return 0;
}

static PyObject *marshal_setup(PyObject *self, PyObject *const *args, Py_ssize_t n) {
    (void)self;
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "setup takes five dtypes");
        return NULL;
    }
    for (int i = 0; i < 5; ++i) {
        Py_INCREF(args[i]);
        Py_XSETREF(g_dtype[i], args[i]);
    }
    Py_RETURN_NONE;
}

static PyObject *marshal_call(PyObject *self, PyObject *const *args, Py_ssize_t n) {
    (void)self;
    int64_t which, address, dev;
    if (n < 3 || int_arg(args[0], 1, &which) || int_arg(args[1], 0, &address) || int_arg(args[2], 1, &dev)) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "call(which, address, device, *arguments)");
        return NULL;
    }
    if (which < 0 || which >= (int)(sizeof g_specs / sizeof g_specs[0]) || address == 0 ||
        (size_t)(n - 3) != strlen(g_specs[which])) {
        PyErr_SetString(PyExc_TypeError, "call: unknown entry point or wrong number of arguments");
        return NULL;
    }
    if (!g_dtype[4]) {
        raise_not_setup();
        return NULL;
    }
    args += 3;
    const char *spec = g_specs[which];
    slot a[MAX_ARGS];
    float scale = 0.f;
    for (int i = 0; spec[i]; ++i) {
        PyObject *o = args[i];
        char c = spec[i];
        a[i].i = 0;
        if (c == 'n' || c == 'q') {
            if (int_arg(o, c == 'n', &a[i].i)) return NULL;
        } else if (c == 'x') {
            const double v = PyFloat_AsDouble(o);
            if (v == -1.0 && PyErr_Occurred()) return NULL;
            scale = (float)v;
        } else if (c == 's') {
            if (o != Py_None && !(a[i].p = PyBytes_AsString(o))) return NULL;
        } else if (c == 'p') {
            if (o != Py_None) {
                a[i].p = PyLong_AsVoidPtr(o);
                if (!a[i].p && PyErr_Occurred()) return NULL;
            }
        } else {
            const int optional = c >= 'A' && c <= 'Z';
            if (optional) {
                if (o == Py_None) continue;
                c = (char)(c - 'A' + 'a');
            }
            const int strided = c == 'r';
            const char *letter = strchr(g_letters, strided ? 'b' : c);
            const int ok = tensor_arg(o, g_dtype[letter - g_letters], !strided, (long)dev, &a[i].p);
            if (ok < 0) return NULL;
            if (!ok) return PyLong_FromLong(-(i + 1));
        }
    }
    int code = PKV_ERR_INVALID_ARG;
    void *const fn = (void *)(intptr_t)address;
#define P(k) a[k].p
#define N(k) (int)a[k].i
#define Q(k) a[k].i
    Py_BEGIN_ALLOW_THREADS
    switch (which) {
        case 0:
            code = ((__typeof__(&pkv_rope_kv_write))fn)(
                P(0), P(1), P(2), P(3), Q(4), Q(5), Q(6), Q(7), P(8), P(9), P(10), P(11), N(12), P(13),
                P(14), Q(15), N(16), N(17), N(18), N(19), N(20), N(21), Q(22), P(23), P(24));
            break;
        case 1:
            code = ((__typeof__(&pkv_paged_attention_decode_scored))fn)(
                P(0), P(1), P(2), P(3), P(4), P(5), P(6), N(7), P(8), N(9), N(10), N(11), N(12), Q(13),
                scale, P(15), P(16), Q(17), N(18), N(19), P(20), (size_t)Q(21), P(22), P(23));
            break;
        case 2:
            code = ((__typeof__(&pkv_paged_attention_prefill_scored))fn)(
                P(0), P(1), N(2), P(3), P(4), P(5), N(6), P(7), P(8), N(9), N(10), N(11), N(12), N(13),
                Q(14), scale, P(16), P(17), Q(18), N(19), P(20), (size_t)Q(21), P(22), P(23));
            break;
        case 3:
            code = ((__typeof__(&pkv_evict_tokens))fn)(
                P(0), P(1), P(2), N(3), P(4), P(5), N(6), P(7), P(8), Q(9), P(10), Q(11), P(12), N(13),
                N(14), N(15), N(16), N(17), Q(18), P(19), P(20));
            break;
    }
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(code);
}

static PyMethodDef methods[] = {
    {"setup", (PyCFunction)(void (*)(void))marshal_setup, METH_FASTCALL, "setup(bfloat16, int32, int64, float32, uint8)"},
    {"call", (PyCFunction)(void (*)(void))marshal_call, METH_FASTCALL, "call(which, address, device, *arguments) -> code"},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void) {
    s_dtype = PyUnicode_InternFromString("dtype");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    if (!s_dtype || !s_get_device || !s_is_contiguous || !s_data_ptr) return NULL;
    return PyModule_Create(&module);
}
