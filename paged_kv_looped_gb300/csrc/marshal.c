/*
 * Argument marshalling of the 8-bit cache's and the prompts' calls in their plain form (all arrays given, of the
 * stated types and shapes, on the current device), as a CPython module.  A decode step makes these calls
 * once per layer and plane; through the interpreter and ctypes their checks take 6 us a call, a launch 2.6.
 *
 * Each function returns the library's status, or None for a call that is not in the plain form: the
 * binding's own code then takes it, and says what is wrong with it where something is.  So nothing is
 * accepted here that is not accepted there.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "rlt.h"

static struct {
    PyObject *tensor, *bf16, *i32, *i64, *f32, *device, *stream;
    PyObject *s_dtype, *s_shape, *s_get_device, *s_data_ptr, *s_is_contiguous, *s_stride, *s_numel, *s_element_size,
        *s_cuda_stream;
    __typeof__(&rlt_kv8_append_rope) append;
    __typeof__(&rlt_paged_decode_attn_kv8) decode;
    __typeof__(&rlt_prefill_attn) prefill;
} g;

/* An int of the object, if it is one in [lo, hi]. */
static int as_int(PyObject *o, long long lo, long long hi, long long *v)
{
    if (o == NULL || !PyLong_Check(o))
        return 0;
    *v = PyLong_AsLongLong(o);
    return !(*v == -1 && PyErr_Occurred()) && *v >= lo && *v <= hi;
}

static int as_i32(PyObject *o, int32_t *v)
{
    long long x;
    if (!as_int(o, INT32_MIN, INT32_MAX, &x))
        return 0;
    *v = (int32_t)x;
    return 1;
}

static int as_double(PyObject *o, double *v)
{
    if (!PyFloat_Check(o) && !PyLong_Check(o))
        return 0;
    *v = PyFloat_AsDouble(o);
    return !(*v == -1.0 && PyErr_Occurred());
}

static int as_pointer(PyObject *o, void **p)
{
    if (o == NULL || !PyLong_Check(o))
        return 0;
    *p = PyLong_AsVoidPtr(o);
    return !(*p == NULL && PyErr_Occurred());
}

/* The int that a method without arguments returns. */
static int method_int(PyObject *t, PyObject *name, long long *v)
{
    PyObject *r = PyObject_CallMethodNoArgs(t, name);
    const int ok = as_int(r, INT64_MIN, INT64_MAX, v);
    Py_XDECREF(r);
    return ok;
}

static int ints_of(PyObject *tuple, int n, long long *v)
{
    int ok = tuple != NULL && PyTuple_Check(tuple) && PyTuple_GET_SIZE(tuple) == n;
    for (int i = 0; ok && i < n; ++i)
        ok = as_int(PyTuple_GET_ITEM(tuple, i), INT64_MIN, INT64_MAX, &v[i]);
    Py_XDECREF(tuple);
    return ok;
}

static int shape_of(PyObject *t, int n, long long *v)
{
    return PyObject_TypeCheck(t, (PyTypeObject *)g.tensor) && ints_of(PyObject_GetAttr(t, g.s_shape), n, v);
}

/* A tensor of this type on device dev. */
static int is_on(PyObject *t, PyObject *dtype, long long dev)
{
    if (!PyObject_TypeCheck(t, (PyTypeObject *)g.tensor))
        return 0;
    if (dtype != NULL) {
        PyObject *d = PyObject_GetAttr(t, g.s_dtype);
        Py_XDECREF(d);                           /* (types live as long as torch does) */
        if (d != dtype)
            return 0;
    }
    long long at;
    return method_int(t, g.s_get_device, &at) && at == dev;
}

static int contiguous(PyObject *t)
{
    PyObject *r = PyObject_CallMethodNoArgs(t, g.s_is_contiguous);
    const int ok = r == Py_True;
    Py_XDECREF(r);
    return ok;
}

static int data_ptr(PyObject *t, void **p)
{
    PyObject *r = PyObject_CallMethodNoArgs(t, g.s_data_ptr);
    const int ok = as_pointer(r, p);
    Py_XDECREF(r);
    return ok;
}

/* A contiguous tensor of this type and shape; None (where it may be) is a null pointer. */
static int array(PyObject *t, PyObject *dtype, long long dev, int n, long long a, long long b, long long c, int maybe,
                 void **p)
{
    const long long want[3] = {a, b, c};
    long long v[3];
    *p = NULL;
    if (t == Py_None)
        return maybe;
    if (!is_on(t, dtype, dev) || !shape_of(t, n, v))
        return 0;
    for (int i = 0; i < n; ++i)
        if (v[i] != want[i])
            return 0;
    return contiguous(t) && data_ptr(t, p);
}

/* Token rows [n][heads][d], n at least 1, whose heads are contiguous. */
static int rows(PyObject *t, long long dev, long long n, long long heads, long long d, void **p, int64_t *stride)
{
    long long v[3], s[3];
    if (!is_on(t, g.bf16, dev) || !shape_of(t, 3, v) || v[0] != n || v[1] != heads || v[2] != d ||
        !ints_of(PyObject_CallMethodNoArgs(t, g.s_stride), 3, s) || s[2] != 1 || (heads > 1 && s[1] != d))
        return 0;
    *stride = n > 1 ? s[0] : heads * d;
    return data_ptr(t, p);
}

/* The current device, and the stream's handle (None: the current one). */
static int here(PyObject *stream, long long *dev, void **handle)
{
    PyObject *r = PyObject_CallNoArgs(g.device);
    int ok = as_int(r, 0, INT32_MAX, dev);
    if (ok && stream == Py_None) {
        PyObject *s = PyObject_CallOneArg(g.stream, r);
        ok = as_pointer(s, handle);
        Py_XDECREF(s);
    } else if (ok && PyLong_Check(stream)) {
        ok = as_pointer(stream, handle);
    } else if (ok) {
        PyObject *s = PyObject_GetAttr(stream, g.s_cuda_stream);
        ok = as_pointer(s, handle);
        Py_XDECREF(s);
    }
    Py_XDECREF(r);
    return ok;
}

static PyObject *not_plain(void)
{
    PyErr_Clear();
    Py_RETURN_NONE;
}

static PyObject *answer(rlt_status st) { return PyLong_FromLong((long)st); }

/* append(pool address, pool device, kv heads, head_dim, bank, k, v, positions, slots, rot_dim, base, q, q_out, k_out,
 *        v_out, stream) */
static PyObject *append(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    void *pool, *stream, *k, *v, *pos, *loc, *q = NULL, *q_out = NULL, *k_out, *v_out;
    long long dev, at, hkv, d, tokens, shape[3] = {0, 0, 0};
    int32_t bank, rot;
    int64_t ks, vs, qs = 0;
    double base;
    (void)self;
    if (n != 16 || !as_pointer(a[0], &pool) || !as_int(a[1], 0, INT32_MAX, &at) || !as_int(a[2], 1, INT32_MAX, &hkv) ||
        !as_int(a[3], 1, INT32_MAX, &d) || !as_i32(a[4], &bank) || !as_i32(a[9], &rot) || !as_double(a[10], &base) ||
        !here(a[15], &dev, &stream) || at != dev || !shape_of(a[8], 1, &tokens) || tokens < 1 || tokens > INT32_MAX ||
        !rows(a[5], dev, tokens, hkv, d, &k, &ks) || !rows(a[6], dev, tokens, hkv, d, &v, &vs) ||
        !array(a[7], g.i64, dev, 1, tokens, 0, 0, 0, &pos) || !array(a[8], g.i64, dev, 1, tokens, 0, 0, 0, &loc))
        return not_plain();
    if ((a[11] == Py_None) != (a[12] == Py_None))
        return not_plain();
    if (a[11] != Py_None &&
        (!shape_of(a[11], 3, shape) || shape[1] > INT32_MAX || !rows(a[11], dev, tokens, shape[1], d, &q, &qs) ||
         !array(a[12], g.bf16, dev, 3, tokens, shape[1], d, 0, &q_out)))
        return not_plain();
    if (!array(a[13], g.bf16, dev, 3, tokens, hkv, d, 1, &k_out) || !array(a[14], g.bf16, dev, 3, tokens, hkv, d, 1, &v_out))
        return not_plain();
    rlt_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g.append(pool, bank, q, (int32_t)shape[1], qs, k, ks, v, vs, pos, loc, (int32_t)tokens, rot, base, q_out, k_out,
                  v_out, NULL, NULL, 0, stream);
    Py_END_ALLOW_THREADS
    return answer(st);
}

/* decode(pool address, pool device, head_dim, bank, q, page_table, seq_lens, max_seq_len, out, lse_out, workspace,
 *        scale, split_tokens, flags, stream) */
static PyObject *decode(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    void *pool, *stream, *q, *table, *lens, *out, *lse, *ws;
    long long dev, at, d, s[3], t[2], numel, size;
    int32_t bank, longest, split, flags;
    double scale;
    (void)self;
    if (n != 15 || !as_pointer(a[0], &pool) || !as_int(a[1], 0, INT32_MAX, &at) || !as_int(a[2], 1, INT32_MAX, &d) ||
        !as_i32(a[3], &bank) || !as_i32(a[7], &longest) || !as_double(a[11], &scale) || !as_i32(a[12], &split) ||
        !as_i32(a[13], &flags) || !here(a[14], &dev, &stream) || at != dev || !shape_of(a[4], 3, s) || s[2] != d ||
        s[0] > INT32_MAX || s[1] > INT32_MAX || !shape_of(a[5], 2, t) || t[0] != s[0] || t[1] > INT32_MAX ||
        !array(a[4], g.bf16, dev, 3, s[0], s[1], d, 0, &q) || !array(a[5], g.i32, dev, 2, t[0], t[1], 0, 0, &table) ||
        !array(a[6], g.i32, dev, 1, s[0], 0, 0, 0, &lens) || !array(a[8], g.bf16, dev, 3, s[0], s[1], d, 0, &out) ||
        !array(a[9], g.f32, dev, 2, s[0], s[1], 0, 1, &lse) || !is_on(a[10], NULL, dev) || !contiguous(a[10]) ||
        !data_ptr(a[10], &ws) || !method_int(a[10], g.s_numel, &numel) || !method_int(a[10], g.s_element_size, &size))
        return not_plain();
    rlt_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g.decode(pool, bank, q, (int32_t)s[1], table, (int32_t)t[1], lens, (int32_t)s[0], longest, (float)scale, out, lse,
                  ws, (size_t)(numel * size), split, (uint32_t)flags, stream);
    Py_END_ALLOW_THREADS
    return answer(st);
}

/* prefill(q, k, v, items, number of items, rows, max_key_tiles, total_key_tiles, query group, out, lse_out, scale,
 *         flags, stream) */
static PyObject *prefill(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    void *stream, *q, *k, *v, *items, *out, *lse;
    long long dev, s[3], sk[3], num_rows, group;
    int32_t num_items, longest, total, flags;
    int64_t qs, ks, vs;
    double scale;
    (void)self;
    if (n != 14 || !as_i32(a[4], &num_items) || num_items < 1 || !as_int(a[5], 0, INT32_MAX, &num_rows) ||
        !as_i32(a[6], &longest) || !as_i32(a[7], &total) || !as_int(a[8], 1, INT32_MAX, &group) ||
        !as_double(a[11], &scale) || !as_i32(a[12], &flags) || !here(a[13], &dev, &stream) || !shape_of(a[0], 3, s) ||
        !shape_of(a[1], 3, sk) || s[0] < 1 || s[0] < num_rows || s[0] > INT32_MAX || s[1] > INT32_MAX ||
        s[2] > INT32_MAX || sk[1] > INT32_MAX || group * sk[1] != s[1] || !rows(a[0], dev, s[0], s[1], s[2], &q, &qs) ||
        !rows(a[1], dev, s[0], sk[1], s[2], &k, &ks) || !rows(a[2], dev, s[0], sk[1], s[2], &v, &vs) ||
        !array(a[3], g.i32, dev, 2, num_items, 4, 0, 0, &items) ||
        !array(a[9], g.bf16, dev, 3, s[0], s[1], s[2], 0, &out) || !array(a[10], g.f32, dev, 2, s[0], s[1], 0, 1, &lse))
        return not_plain();
    rlt_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g.prefill(q, (int32_t)s[1], qs, k, ks, v, vs, (int32_t)sk[1], (int32_t)s[2], (int32_t)s[0], items, num_items,
                   longest, total, (float)scale, out, lse, (uint32_t)flags, stream);
    Py_END_ALLOW_THREADS
    return answer(st);
}

/* bind(Tensor, bfloat16, int32, int64, float32, current device, current stream of a device, addresses of the three
 *      entry points) */
static PyObject *bind(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    PyObject **const keep[7] = {&g.tensor, &g.bf16, &g.i32, &g.i64, &g.f32, &g.device, &g.stream};
    struct { PyObject **at; const char *name; } const names[] = {
        {&g.s_dtype, "dtype"}, {&g.s_shape, "shape"}, {&g.s_get_device, "get_device"}, {&g.s_data_ptr, "data_ptr"},
        {&g.s_is_contiguous, "is_contiguous"}, {&g.s_stride, "stride"}, {&g.s_numel, "numel"},
        {&g.s_element_size, "element_size"}, {&g.s_cuda_stream, "cuda_stream"}};
    void *fn[3];
    (void)self;
    if (n != 10 || !PyType_Check(a[0]) || !as_pointer(a[7], &fn[0]) || !as_pointer(a[8], &fn[1]) ||
        !as_pointer(a[9], &fn[2])) {
        PyErr_SetString(PyExc_TypeError, "bind: wrong arguments");
        return NULL;
    }
    for (int i = 0; i < 7; ++i) {
        Py_INCREF(a[i]);
        Py_XDECREF(*keep[i]);
        *keep[i] = a[i];
    }
    for (size_t i = 0; i < sizeof(names) / sizeof(names[0]); ++i)
        if (*names[i].at == NULL && (*names[i].at = PyUnicode_InternFromString(names[i].name)) == NULL)
            return NULL;
    g.append = (__typeof__(g.append))fn[0];
    g.decode = (__typeof__(g.decode))fn[1];
    g.prefill = (__typeof__(g.prefill))fn[2];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, NULL},
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, NULL},
    {"decode", (PyCFunction)(void (*)(void))decode, METH_FASTCALL, NULL},
    {"prefill", (PyCFunction)(void (*)(void))prefill, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
