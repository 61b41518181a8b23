/* calls.c -- argument marshalling of the block calls for Python: the plain case (contiguous CUDA tensors of the
 * expected types and shapes) straight from the tensors' attributes to the C ABI. It checks what the Python
 * functions check; whatever is not the plain case it leaves alone (-1), for those functions to handle or to
 * refuse. Through ctypes alone a call's marshalling takes 4 to 6 us of an Arm host, here about 1.5.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "moe_nvfp4.h"

typedef moe_status_t (*norm_fn)(const moe_norm_t*, const uint16_t*, int64_t, const void*, int64_t, int, void*, int64_t, uint16_t*,
                                int64_t, moe_stream_t);
typedef moe_status_t (*select_fn)(const moe_routing_t*, const void*, int, int64_t, int, int32_t*, float*, moe_stream_t);
typedef moe_status_t (*adapter_fn)(const moe_adapters_t*, const uint16_t*, int64_t, int, const int32_t*, const int32_t*, int,
                                   const uint16_t*, int64_t, uint16_t*, int64_t, void*, size_t, moe_stream_t);

static norm_fn f_norm;
static select_fn f_select;
static adapter_fn f_adapter;
static PyObject *t_bf16, *t_f32, *t_i32; /* torch's dtypes */
static PyObject *s_dtype, *s_is_cuda, *s_shape, *s_is_contiguous, *s_data_ptr;

static int is_true(PyObject* v)
{
    const int yes = v == Py_True;
    Py_XDECREF(v);
    return yes;
}

/* The type of t among bf16, fp32 and int32, or -1. */
static int dtype_of(PyObject* t)
{
    PyObject* v = PyObject_GetAttr(t, s_dtype);
    const int d = v == t_bf16 ? 0 : v == t_f32 ? 1 : v == t_i32 ? 2 : -1;
    Py_XDECREF(v);
    return d;
}

/* 1 and t's address where t is a contiguous CUDA tensor of nd dimensions, dims[i] each (a negative one is
 * filled in); 0 where it is not. */
static int whole(PyObject* t, int nd, int64_t* dims, void** p)
{
    PyObject* v;
    int i, good;
    if (!is_true(PyObject_GetAttr(t, s_is_cuda))) return 0;
    v = PyObject_GetAttr(t, s_shape);
    good = v && PyTuple_Check(v) && PyTuple_GET_SIZE(v) == nd;
    for (i = 0; good && i < nd; ++i) {
        const int64_t n = PyLong_AsLongLong(PyTuple_GET_ITEM(v, i));
        if (dims[i] < 0) dims[i] = n;
        good = n >= 0 && n == dims[i] && n <= INT32_MAX;
    }
    Py_XDECREF(v);
    if (!good || !is_true(PyObject_CallMethodNoArgs(t, s_is_contiguous))) return 0;
    v = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!v) return 0;
    *p = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return !PyErr_Occurred();
}

static PyObject* leave(void)
{
    PyErr_Clear();
    return PyLong_FromLong(-1);
}

/* numbers among the arguments; an error of their conversion is looked for once */
static int as_int(PyObject* v)
{
    const long i = PyLong_AsLong(v);
    if (i != (int)i) PyErr_SetString(PyExc_OverflowError, "an int of more than 32 bits");
    return (int)i;
}
static float as_float(PyObject* v) { return (float)PyFloat_AsDouble(v); }

/* norm_residual(y, residual, w_post, w_pre, gate, residual_scale, eps, w_offset, residual_out, x_out, stream) */
static PyObject* norm_residual(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    moe_norm_t d;
    void *y = NULL, *r = NULL, *ro = NULL, *x = NULL, *p = NULL;
    int64_t rows[2] = {-1, -1}, cols[1];
    moe_status_t s;
    (void)self;
    if (n != 11 || !f_norm) return leave();
    memset(&d, 0, sizeof d);
    if (a[0] != Py_None && (dtype_of(a[0]) != 0 || !whole(a[0], 2, rows, &y))) return leave();
    if (a[1] != Py_None) {
        d.residual_dtype = dtype_of(a[1]);
        if (d.residual_dtype < 0 || d.residual_dtype > 1 || !whole(a[1], 2, rows, &r)) return leave();
    }
    if (rows[0] < 0) return leave();
    if (dtype_of(a[8]) != d.residual_dtype || !whole(a[8], 2, rows, &ro)) return leave();
    if (a[9] != Py_None && (dtype_of(a[9]) != 0 || !whole(a[9], 2, rows, &x))) return leave();
    cols[0] = rows[1];
    if (a[2] != Py_None) {
        if (dtype_of(a[2]) != 0 || !whole(a[2], 1, cols, &p)) return leave();
        d.w_post = p;
    }
    if (a[3] != Py_None) {
        if (dtype_of(a[3]) != 0 || !whole(a[3], 1, cols, &p)) return leave();
        d.w_pre = p;
    }
    if (a[4] != Py_None) { /* [H], [T, 1], [T, H] or [1, 1]; [1, H] goes the other way */
        int64_t g[2] = {rows[0], 1};
        d.gate_dtype = dtype_of(a[4]);
        if (d.gate_dtype < 0 || d.gate_dtype > 1) return leave();
        if (whole(a[4], 1, cols, &p)) {
            d.gate_per_channel = 1;
        } else if (whole(a[4], 2, g, &p)) {
            d.gate_ld = 1;
        } else if (whole(a[4], 2, rows, &p)) {
            d.gate_per_channel = 1;
            d.gate_ld = rows[1];
        } else {
            return leave();
        }
        d.gate = p;
    }
    d.H = (int)rows[1];
    d.residual_scale = as_float(a[5]);
    d.eps = as_float(a[6]);
    d.w_offset = as_float(a[7]);
    p = PyLong_AsVoidPtr(a[10]);
    if (PyErr_Occurred()) return leave();
    Py_BEGIN_ALLOW_THREADS
    s = f_norm(&d, y, rows[1], r, rows[1], (int)rows[0], ro, rows[1], x, rows[1], p);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(s);
}

/* select_experts(logits, k, bias, score, n_group, topk_group, group_score, renormalize, scale, ids, weights, stream) */
static PyObject* select_experts(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    moe_routing_t d;
    void *l = NULL, *ids = NULL, *w = NULL, *p = NULL;
    int64_t rows[2] = {-1, -1}, out[2], cols[1];
    int lt;
    moe_status_t s;
    (void)self;
    if (n != 12 || !f_select) return leave();
    memset(&d, 0, sizeof d);
    lt = dtype_of(a[0]);
    if (lt < 0 || lt > 1 || !whole(a[0], 2, rows, &l)) return leave();
    d.E = (int)rows[1];
    d.k = as_int(a[1]);
    out[0] = rows[0];
    out[1] = d.k;
    if (d.k < 1 || dtype_of(a[9]) != 2 || !whole(a[9], 2, out, &ids) || dtype_of(a[10]) != 1 || !whole(a[10], 2, out, &w)) return leave();
    cols[0] = rows[1];
    if (a[2] != Py_None) {
        if (dtype_of(a[2]) != 1 || !whole(a[2], 1, cols, &p)) return leave();
        d.bias = p;
    }
    d.score = as_int(a[3]);
    d.n_group = as_int(a[4]);
    d.topk_group = as_int(a[5]);
    d.group_score = as_int(a[6]);
    d.renormalize = PyObject_IsTrue(a[7]);
    d.scale = as_float(a[8]);
    p = PyLong_AsVoidPtr(a[11]);
    if (PyErr_Occurred()) return leave();
    Py_BEGIN_ALLOW_THREADS
    s = f_select(&d, l, lt, rows[1], (int)rows[0], ids, w, p);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(s);
}

/* adapter_add(x, y, a, b, scale, seg_offsets, seg_adapter, out, ws, ws_bytes, stream) */
static PyObject* adapter_add(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    moe_adapters_t d;
    void *x = NULL, *y = NULL, *o = NULL, *off = NULL, *ids = NULL, *ws = NULL, *p = NULL;
    int64_t xs[2] = {-1, -1}, ys[2] = {-1, -1}, as[3] = {-1, -1, -1}, bs[3], ns[1], ss[1] = {-1};
    size_t ws_bytes;
    moe_status_t s;
    (void)self;
    if (n != 11 || !f_adapter) return leave();
    memset(&d, 0, sizeof d);
    if (dtype_of(a[0]) != 0 || !whole(a[0], 2, xs, &x)) return leave();
    ys[0] = xs[0];
    if (dtype_of(a[1]) != 0 || !whole(a[1], 2, ys, &y)) return leave();
    if (a[7] == a[1]) o = y;
    else if (dtype_of(a[7]) != 0 || !whole(a[7], 2, ys, &o)) return leave();
    as[2] = xs[1];
    if (dtype_of(a[2]) != 0 || !whole(a[2], 3, as, &p)) return leave();
    d.a = p;
    bs[0] = ns[0] = as[0];
    bs[1] = ys[1];
    bs[2] = as[1];
    if (dtype_of(a[3]) != 0 || !whole(a[3], 3, bs, &p)) return leave();
    d.b = p;
    if (dtype_of(a[4]) != 1 || !whole(a[4], 1, ns, &p)) return leave();
    d.scale = p;
    if (dtype_of(a[6]) != 2 || !whole(a[6], 1, ss, &ids)) return leave();
    d.n = (int)as[0];
    d.r = (int)as[1];
    d.K = (int)xs[1];
    d.N = (int)ys[1];
    ns[0] = ss[0] + 1;
    if (dtype_of(a[5]) != 2 || !whole(a[5], 1, ns, &off)) return leave();
    ws = PyLong_AsVoidPtr(a[8]);
    ws_bytes = PyLong_AsSize_t(a[9]);
    p = PyLong_AsVoidPtr(a[10]);
    if (PyErr_Occurred()) return leave();
    Py_BEGIN_ALLOW_THREADS
    s = f_adapter(&d, x, xs[1], (int)xs[0], off, ids, (int)ss[0], y, ys[1], o, ys[1], ws, ws_bytes, p);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(s);
}

/* bind(norm, select, adapter, bfloat16, float32, int32): the library's functions by address, torch's dtypes */
static PyObject* bind(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    void* f[3];
    int i;
    (void)self;
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "bind takes three addresses and three dtypes");
        return NULL;
    }
    for (i = 0; i < 3; ++i) f[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return NULL;
    f_norm = (norm_fn)f[0];
    f_select = (select_fn)f[1];
    f_adapter = (adapter_fn)f[2];
    Py_XSETREF(t_bf16, Py_NewRef(a[3]));
    Py_XSETREF(t_f32, Py_NewRef(a[4]));
    Py_XSETREF(t_i32, Py_NewRef(a[5]));
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, NULL},
                                {"norm_residual", (PyCFunction)(void (*)(void))norm_residual, METH_FASTCALL, NULL},
                                {"select_experts", (PyCFunction)(void (*)(void))select_experts, METH_FASTCALL, NULL},
                                {"adapter_add", (PyCFunction)(void (*)(void))adapter_add, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__calls(void)
{
    s_dtype = PyUnicode_InternFromString("dtype");
    s_is_cuda = PyUnicode_InternFromString("is_cuda");
    s_shape = PyUnicode_InternFromString("shape");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    if (!s_dtype || !s_is_cuda || !s_shape || !s_is_contiguous || !s_data_ptr) return NULL;
    return PyModule_Create(&module);
}
