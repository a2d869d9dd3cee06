/* native_calls.c -- CPython module `_native`: the recurrent entry points called on torch tensors.
 *
 * Marshalling only: every tensor argument (None for a NULL descriptor) becomes an mss_tensor_t on the
 * C stack and the library's function is called with them.  The same through ctypes costs about 1.6 us
 * a tensor in the interpreter, more than the kernels of a one-token step take; here it is five attribute
 * reads, about 0.3 us.  Device memory is not touched and no torch header is needed: a tensor is asked by
 * its public attributes (data_ptr, dtype, shape, is_contiguous, get_device).
 *
 * Every function returns the library's status.  Host tensors and tensors of two devices raise
 * ValueError before the call.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <limits.h>
#include <stdint.h>
#include <string.h>

#include "mamba_scan.h"

enum { MOST = 16 };

static PyObject *s_data_ptr, *s_dtype, *s_shape, *s_stride, *s_is_contiguous, *s_get_device;
static PyObject *dtypes[3]; /* torch.float32, torch.bfloat16, torch.int32, in the order of mss_dtype_t */

static int whole(PyObject* o, int64_t* v) {
    *v = PyLong_AsLongLong(o);
    return *v == -1 && PyErr_Occurred() ? -1 : 0;
}

/* A method without arguments that gives a whole number. */
static int ask(PyObject* t, PyObject* name, int64_t* v) {
    PyObject* r = PyObject_CallMethodNoArgs(t, name);
    if (!r) return -1;
    int bad = 0;
    if (name == s_data_ptr) { /* addresses use all 64 bits */
        *v = (int64_t)PyLong_AsUnsignedLongLong(r);
        bad = *v == -1 && PyErr_Occurred() ? -1 : 0;
    } else {
        bad = whole(r, v);
    }
    Py_DECREF(r);
    return bad;
}

/* The first four entries of a tuple of whole numbers (steals the reference). */
static int four(PyObject* tuple, int64_t* out, int32_t* n) {
    if (!tuple) return -1;
    int bad = 0;
    if (!PyTuple_Check(tuple)) {
        PyErr_SetString(PyExc_TypeError, "libmamba_scan takes torch tensors");
        bad = -1;
    } else {
        const Py_ssize_t k = PyTuple_GET_SIZE(tuple);
        *n = (int32_t)k; /* more than four: refused by the library */
        for (Py_ssize_t j = 0; j < k && j < 4 && !bad; ++j) bad = whole(PyTuple_GET_ITEM(tuple, j), &out[j]);
    }
    Py_DECREF(tuple);
    return bad;
}

/* Fills d from tensor t; *device is the call's device so far, INT_MIN for none. */
static int describe(PyObject* t, mss_tensor_t* d, int64_t* device) {
    memset(d, 0, sizeof *d);
    int64_t at, dev;
    if (ask(t, s_get_device, &dev)) return -1;
    if (dev < 0) {
        PyErr_SetString(PyExc_ValueError, "libmamba_scan takes device tensors");
        return -1;
    }
    if (*device == INT_MIN) *device = dev;
    if (dev != *device) {
        PyErr_Format(PyExc_ValueError, "libmamba_scan takes tensors of one device, got %lld and %lld",
                     (long long)*device, (long long)dev);
        return -1;
    }
    if (ask(t, s_data_ptr, &at)) return -1;
    d->data = (void*)(intptr_t)at;
    PyObject* dtype = PyObject_GetAttr(t, s_dtype);
    if (!dtype) return -1;
    d->dtype = -1; /* any other type: refused by the library */
    for (int k = 0; k < 3; ++k)
        if (dtype == dtypes[k]) d->dtype = k;
    Py_DECREF(dtype);
    if (four(PyObject_GetAttr(t, s_shape), d->shape, &d->ndim)) return -1;
    PyObject* dense = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (!dense) return -1;
    Py_DECREF(dense);
    if (dense == Py_True && d->ndim <= 4) { /* the usual case, without asking for the strides */
        int64_t step = 1;
        for (int k = d->ndim - 1; k >= 0; --k) {
            d->stride[k] = step;
            step *= d->shape[k];
        }
        return 0;
    }
    int32_t n;
    return four(PyObject_CallMethodNoArgs(t, s_stride), d->stride, &n);
}

/* The arguments of a call: descriptors p[k] (NULL for None) and whole numbers v[k], as `kinds` says
 * ('t' a tensor or None, 'i' a whole number), and the stream that ends them. */
typedef struct {
    mss_tensor_t d[MOST];
    const mss_tensor_t* p[MOST];
    int v[MOST];
    void* stream;
} Call;

static int take(Call* c, const char* kinds, PyObject* const* args, Py_ssize_t n) {
    const Py_ssize_t want = (Py_ssize_t)strlen(kinds);
    if (n != want + 1) {
        PyErr_Format(PyExc_TypeError, "%zd arguments and a stream wanted, got %zd", want, n);
        return -1;
    }
    int64_t device = INT_MIN;
    for (Py_ssize_t k = 0; k < want; ++k) {
        c->p[k] = NULL;
        if (kinds[k] == 'i') {
            int64_t v;
            if (whole(args[k], &v)) return -1;
            if (v < INT_MIN || v > INT_MAX) {
                PyErr_SetString(PyExc_OverflowError, "a whole number of 32 bits is wanted");
                return -1;
            }
            c->v[k] = (int)v;
        } else if (args[k] != Py_None) {
            if (describe(args[k], &c->d[k], &device)) return -1;
            c->p[k] = &c->d[k];
        }
    }
    c->stream = (void*)(uintptr_t)PyLong_AsUnsignedLongLong(args[want]);
    return PyErr_Occurred() ? -1 : 0;
}

#define ENTRY(NAME, KINDS, CALL)                                                          \
    static PyObject* NAME(PyObject* self, PyObject* const* args, Py_ssize_t n) {          \
        (void)self;                                                                       \
        Call c;                                                                           \
        if (take(&c, KINDS, args, n)) return NULL;                                        \
        int st;                                                                           \
        Py_BEGIN_ALLOW_THREADS st = CALL;                                                 \
        Py_END_ALLOW_THREADS return PyLong_FromLong(st);                                  \
    }

#define P c.p
ENTRY(gated_scan_fwd, "tttttttttt",
      mss_gated_scan_fwd(P[0], P[1], P[2], P[3], P[4], P[5], P[6], P[7], P[8], P[9], c.stream))
ENTRY(gated_scan_bwd, "tttttttttttttt",
      mss_gated_scan_bwd(P[0], P[1], P[2], P[3], P[4], P[5], P[6], P[7], P[8], P[9], P[10], P[11], P[12], P[13],
                         c.stream))
ENTRY(gated_state_update, "tttttt", mss_gated_state_update(P[0], P[1], P[2], P[3], P[4], P[5], c.stream))
ENTRY(causal_conv1d_bwd, "ttttittttttt",
      mss_causal_conv1d_bwd(P[0], P[1], P[2], P[3], c.v[4], P[5], P[6], P[7], P[8], P[9], P[10], P[11], c.stream))
ENTRY(beam_select, "tttittttt",
      mss_beam_select(P[0], P[1], P[2], c.v[3], P[4], P[5], P[6], P[7], P[8], c.stream))
#undef P

/* beam_reorder(sequence of tensors, parents, stream) */
static PyObject* beam_reorder(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    (void)self;
    if (n != 3) {
        PyErr_SetString(PyExc_TypeError, "states, parents and a stream wanted");
        return NULL;
    }
    PyObject* seq = PySequence_Tuple(args[0]); /* of its own: no other thread changes it meanwhile */
    if (!seq) return NULL;
    const Py_ssize_t k = PyTuple_GET_SIZE(seq);
    PyObject* result = NULL;
    mss_tensor_t par, *d = PyMem_Malloc((size_t)(k + 1) * sizeof *d);
    const mss_tensor_t** p = PyMem_Malloc((size_t)(k + 1) * sizeof *p);
    int64_t device = INT_MIN;
    if (!d || !p || k > INT_MAX) {
        PyErr_NoMemory();
        goto done;
    }
    if (describe(args[1], &par, &device)) goto done;
    for (Py_ssize_t j = 0; j < k; ++j) {
        if (describe(PyTuple_GET_ITEM(seq, j), &d[j], &device)) goto done;
        p[j] = &d[j];
    }
    void* stream = (void*)(uintptr_t)PyLong_AsUnsignedLongLong(args[2]);
    if (PyErr_Occurred()) goto done;
    int st;
    Py_BEGIN_ALLOW_THREADS st = mss_beam_reorder(p, (int)k, &par, stream);
    Py_END_ALLOW_THREADS result = PyLong_FromLong(st);
done:
    PyMem_Free(d);
    PyMem_Free((void*)p);
    Py_DECREF(seq);
    return result;
}

/* The _scratch queries: whole numbers in, (status, floats ...) out. */
static int sizes(PyObject* const* args, Py_ssize_t n, int64_t* v, Py_ssize_t want) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%zd sizes wanted, got %zd", want, n);
        return -1;
    }
    for (Py_ssize_t k = 0; k < n; ++k)
        if (whole(args[k], &v[k])) return -1;
    return 0;
}
static PyObject* gated_scan_scratch(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    (void)self;
    int64_t v[3], fwd = 0, bwd = 0;
    if (sizes(args, n, v, 3)) return NULL;
    const int st = mss_gated_scan_scratch(v[0], v[1], v[2], &fwd, &bwd);
    return Py_BuildValue("iLL", st, (long long)fwd, (long long)bwd);
}
static PyObject* causal_conv1d_bwd_scratch(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    (void)self;
    int64_t v[4], floats = 0;
    if (sizes(args, n, v, 4)) return NULL;
    const int st = mss_causal_conv1d_bwd_scratch(v[0], v[1], v[2], v[3], &floats);
    return Py_BuildValue("iL", st, (long long)floats);
}
static PyObject* beam_select_scratch(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    (void)self;
    int64_t v[4], floats = 0;
    if (sizes(args, n, v, 4)) return NULL;
    const int st = mss_beam_select_scratch(v[0], v[1], v[2], v[3], &floats);
    return Py_BuildValue("iL", st, (long long)floats);
}

/* set_dtypes(torch.float32, torch.bfloat16, torch.int32) */
static PyObject* set_dtypes(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    (void)self;
    if (n != 3) {
        PyErr_SetString(PyExc_TypeError, "three types wanted");
        return NULL;
    }
    for (int k = 0; k < 3; ++k) {
        Py_INCREF(args[k]);
        Py_XSETREF(dtypes[k], args[k]);
    }
    Py_RETURN_NONE;
}

#define METHOD(NAME) {#NAME, (PyCFunction)(void (*)(void))NAME, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {METHOD(gated_scan_fwd),    METHOD(gated_scan_bwd), METHOD(gated_state_update),
                                METHOD(causal_conv1d_bwd), METHOD(beam_select),    METHOD(beam_reorder),
                                METHOD(gated_scan_scratch), METHOD(causal_conv1d_bwd_scratch),
                                METHOD(beam_select_scratch), METHOD(set_dtypes), {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__native(void) {
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_get_device = PyUnicode_InternFromString("get_device");
    if (!s_is_contiguous || !s_data_ptr || !s_dtype || !s_shape || !s_stride || !s_get_device) return NULL;
    return PyModule_Create(&module);
}
