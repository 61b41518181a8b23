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

typedef moe_status_t (*append_fn)(const moe_kv_cache_t*, const moe_requests_t*, const moe_rotary_t*, const uint16_t*, int64_t,
                                  const uint16_t*, int64_t, const uint16_t*, int64_t, int, uint16_t*, int64_t, void*, size_t, moe_stream_t);
typedef moe_status_t (*attention_fn)(const moe_kv_cache_t*, const moe_requests_t*, const moe_attention_t*, const uint16_t*, int64_t, int,
                                     uint16_t*, int64_t, float*, void*, size_t, moe_stream_t);
typedef moe_status_t (*quantize_fp8_fn)(const uint16_t*, int64_t, int, int, uint8_t*, float*, moe_stream_t);
typedef moe_status_t (*gemm_fp8_fn)(const uint8_t*, const float*, const uint8_t*, const float*, int, int, int, void*, int, int64_t, void*,
                                    size_t, moe_stream_t);

static norm_fn f_norm;
static select_fn f_select;
static adapter_fn f_adapter;
static append_fn f_append;
static attention_fn f_attention;
static quantize_fp8_fn f_quantize_fp8;
static gemm_fp8_fn f_gemm_fp8;
static PyObject *t_bf16, *t_f32, *t_i32, *t_e4m3; /* torch's dtypes */
static PyObject *s_dtype, *s_is_cuda, *s_shape, *s_is_contiguous, *s_data_ptr, *s_stride;

static int is_true(PyObject* v)
{
    const int yes = v == Py_True;
    Py_XDECREF(v);
    return yes;
}

/* The type of t among bf16, fp32, int32 and E4M3, or -1. */
static int dtype_of(PyObject* t)
{
    PyObject* v = PyObject_GetAttr(t, s_dtype);
    const int d = !v ? -1 : v == t_bf16 ? 0 : v == t_f32 ? 1 : v == t_i32 ? 2 : v == t_e4m3 ? 3 : -1;
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

/* The same of a tensor whose strides (in elements) go to ld; the last dimension's has to be 1. */
static int strided(PyObject* t, int nd, int64_t* dims, int64_t* ld, void** p)
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
    if (!good) return 0;
    v = PyObject_CallMethodNoArgs(t, s_stride);
    good = v && PyTuple_Check(v) && PyTuple_GET_SIZE(v) == nd;
    for (i = 0; good && i < nd; ++i) ld[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(v, i));
    Py_XDECREF(v);
    if (!good || ld[nd - 1] != 1) return 0;
    v = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!v) return 0;
    *p = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return !PyErr_Occurred();
}

/* Tokens [T, n, D] of bf16 whose heads lie side by side. */
static int heads(PyObject* t, int64_t* dims, int64_t* ld, void** p)
{
    int64_t s[3];
    if (dtype_of(t) != 0 || !strided(t, 3, dims, s, p) || s[1] != dims[2]) return 0;
    *ld = s[0];
    return 1;
}

/* k_cache, v_cache, k_scale, v_scale */
static int cache_of(PyObject* const* a, moe_kv_cache_t* c)
{
    int64_t dims[4] = {-1, -1, -1, -1}, ld[4], ld_v[4], n[1];
    const int dt = dtype_of(a[0]);
    void* p = NULL;
    if ((dt != 0 && dt != 3) || dtype_of(a[1]) != dt || !strided(a[0], 4, dims, ld, &c->k) || !strided(a[1], 4, dims, ld_v, &c->v)) return 0;
    if (ld[0] != ld_v[0] || ld[1] != ld_v[1] || ld[2] != ld_v[2]) return 0;
    c->dtype = dt == 0 ? MOE_DTYPE_BF16 : MOE_DTYPE_E4M3;
    c->n_pages = (int)dims[0];
    c->page_size = (int)dims[1];
    c->n_kv = (int)dims[2];
    c->D = (int)dims[3];
    c->ld_page = ld[0];
    c->ld_slot = ld[1];
    c->ld_head = ld[2];
    n[0] = dims[2];
    if (a[2] != Py_None) {
        if (dtype_of(a[2]) != 1 || !whole(a[2], 1, n, &p)) return 0;
        c->k_scale = p;
    }
    if (a[3] != Py_None) {
        if (dtype_of(a[3]) != 1 || !whole(a[3], 1, n, &p)) return 0;
        c->v_scale = p;
    }
    return 1;
}

/* seg_offsets, kv_len, pages */
static int requests_of(PyObject* const* a, moe_requests_t* r)
{
    int64_t n[1] = {-1}, dims[2] = {-1, -1}, ld[2];
    void* p = NULL;
    if (dtype_of(a[1]) != 2 || !whole(a[1], 1, n, &p)) return 0;
    r->kv_len = p;
    r->S = (int)n[0];
    dims[0] = n[0]++;
    if (dtype_of(a[0]) != 2 || !whole(a[0], 1, n, &p)) return 0;
    r->seg_offsets = p;
    if (dtype_of(a[2]) != 2 || !strided(a[2], 2, dims, ld, &p)) return 0;
    r->pages = p;
    r->max_pages = (int)dims[1];
    r->ld_pages = ld[0];
    return 1;
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
    if (PyErr_Occurred()) return leave(); /* before any Python code runs, which may clear it */
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

/* cache_append(q, k, v, k_cache, v_cache, k_scale, v_scale, seg_offsets, kv_len, pages, inv_freq, interleaved, w_q, w_k, eps,
 * w_offset, out, ws, ws_bytes, stream) */
static PyObject* cache_append(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    moe_kv_cache_t c;
    moe_requests_t r;
    moe_rotary_t d;
    void *q = NULL, *k = NULL, *v = NULL, *o = NULL, *ws, *p = NULL;
    int64_t kd[3] = {-1, -1, -1}, qd[3] = {-1, -1, -1}, ld_q = 0, ld_k, ld_v, ld_o = 0, one[1];
    size_t ws_bytes;
    moe_status_t s;
    (void)self;
    if (n != 20 || !f_append) return leave();
    memset(&c, 0, sizeof c);
    memset(&r, 0, sizeof r);
    memset(&d, 0, sizeof d);
    if (!heads(a[1], kd, &ld_k, &k) || !heads(a[2], kd, &ld_v, &v)) return leave();
    if (a[0] != Py_None) {
        qd[0] = kd[0];
        qd[2] = kd[2];
        if (!heads(a[0], qd, &ld_q, &q)) return leave();
        if (a[16] == a[0]) {
            o = q;
            ld_o = ld_q;
        } else if (!heads(a[16], qd, &ld_o, &o)) {
            return leave();
        }
        d.n_q = (int)qd[1];
    } else if (a[16] != Py_None) {
        return leave();
    }
    if (!cache_of(a + 3, &c) || c.n_kv != kd[1] || c.D != kd[2] || !requests_of(a + 7, &r)) return leave();
    if (a[10] != Py_None) {
        one[0] = -1;
        if (dtype_of(a[10]) != 1 || !whole(a[10], 1, one, &p) || one[0] > kd[2]) return leave();
        d.inv_freq = p;
        d.rot = (int)(2 * one[0]);
    }
    d.interleaved = PyObject_IsTrue(a[11]);
    one[0] = kd[2];
    if (a[12] != Py_None) {
        if (dtype_of(a[12]) != 0 || !whole(a[12], 1, one, &p)) return leave();
        d.w_q = p;
    }
    if (a[13] != Py_None) {
        if (dtype_of(a[13]) != 0 || !whole(a[13], 1, one, &p)) return leave();
        d.w_k = p;
    }
    d.eps = as_float(a[14]);
    d.w_offset = as_float(a[15]);
    ws = PyLong_AsVoidPtr(a[17]);
    ws_bytes = PyLong_AsSize_t(a[18]);
    p = PyLong_AsVoidPtr(a[19]);
    if (PyErr_Occurred()) return leave();
    Py_BEGIN_ALLOW_THREADS
    s = f_append(&c, &r, &d, q, ld_q, k, ld_k, v, ld_v, (int)kd[0], o, ld_o, ws, ws_bytes, p);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(s);
}

/* paged_attention(q, k_cache, v_cache, k_scale, v_scale, seg_offsets, kv_len, pages, max_new, scale, window, out, lse, ws, ws_bytes,
 * stream, report) */
static PyObject* paged_attention(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    moe_kv_cache_t c;
    moe_requests_t r;
    moe_attention_t d;
    void *q = NULL, *o = NULL, *lse = NULL, *ws, *p;
    int64_t qd[3] = {-1, -1, -1}, ld_q, ld_o;
    size_t ws_bytes;
    moe_status_t s;
    (void)self;
    if (n != 17 || !f_attention) return leave();
    memset(&c, 0, sizeof c);
    memset(&r, 0, sizeof r);
    if (!heads(a[0], qd, &ld_q, &q)) return leave();
    if (a[11] == a[0]) {
        o = q;
        ld_o = ld_q;
    } else if (!heads(a[11], qd, &ld_o, &o)) {
        return leave();
    }
    if (!cache_of(a + 1, &c) || c.D != qd[2] || !requests_of(a + 5, &r)) return leave();
    if (a[12] != Py_None && (dtype_of(a[12]) != 1 || !whole(a[12], 2, qd, &lse))) return leave();
    d.n_q = (int)qd[1];
    d.max_new = as_int(a[8]);
    d.scale = as_float(a[9]);
    d.window = as_int(a[10]);
    ws = PyLong_AsVoidPtr(a[13]);
    ws_bytes = PyLong_AsSize_t(a[14]);
    p = PyLong_AsVoidPtr(a[15]);
    d.report = PyLong_AsVoidPtr(a[16]);
    if (PyErr_Occurred()) return leave();
    Py_BEGIN_ALLOW_THREADS
    s = f_attention(&c, &r, &d, q, ld_q, (int)qd[0], o, ld_o, lse, ws, ws_bytes, p);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(s);
}

/* quantize_fp8(x, codes, scales, stream) */
static PyObject* quantize_fp8(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    void *x = NULL, *codes = NULL, *scales = NULL, *p;
    int64_t dims[2] = {-1, -1}, ld[2], sd[2];
    moe_status_t s;
    (void)self;
    if (n != 4 || !f_quantize_fp8) return leave();
    if (dtype_of(a[0]) != 0 || !strided(a[0], 2, dims, ld, &x) || dtype_of(a[1]) != 3 || !whole(a[1], 2, dims, &codes)) return leave();
    sd[0] = dims[0];
    sd[1] = (dims[1] + 127) / 128;
    if (dtype_of(a[2]) != 1 || !whole(a[2], 2, sd, &scales)) return leave();
    p = PyLong_AsVoidPtr(a[3]);
    if (PyErr_Occurred()) return leave();
    Py_BEGIN_ALLOW_THREADS
    s = f_quantize_fp8(x, ld[0], (int)dims[0], (int)dims[1], codes, scales, p);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(s);
}

/* gemm_fp8(a, a_scale, b, b_scale, out, ws, ws_bytes, stream) */
static PyObject* gemm_fp8(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    void *x = NULL, *xs = NULL, *w = NULL, *wsc = NULL, *o = NULL, *ws, *p;
    int64_t ad[2] = {-1, -1}, bd[2] = {-1, -1}, sd[2], od[2], ld[2];
    size_t ws_bytes;
    int dt;
    moe_status_t s;
    (void)self;
    if (n != 8 || !f_gemm_fp8) return leave();
    if (dtype_of(a[0]) != 3 || !whole(a[0], 2, ad, &x)) return leave();
    bd[1] = ad[1];
    if (dtype_of(a[2]) != 3 || !whole(a[2], 2, bd, &w)) return leave();
    sd[0] = ad[0];
    sd[1] = (ad[1] + 127) / 128;
    if (dtype_of(a[1]) != 1 || !whole(a[1], 2, sd, &xs)) return leave();
    sd[0] = (bd[0] + 127) / 128;
    if (dtype_of(a[3]) != 1 || !whole(a[3], 2, sd, &wsc)) return leave();
    od[0] = ad[0];
    od[1] = bd[0];
    dt = dtype_of(a[4]);
    if ((dt != 0 && dt != 1) || !strided(a[4], 2, od, ld, &o)) return leave();
    ws = PyLong_AsVoidPtr(a[5]);
    ws_bytes = PyLong_AsSize_t(a[6]);
    p = PyLong_AsVoidPtr(a[7]);
    if (PyErr_Occurred()) return leave();
    Py_BEGIN_ALLOW_THREADS
    s = f_gemm_fp8(x, xs, w, wsc, (int)ad[0], (int)bd[0], (int)ad[1], o, dt == 1 ? MOE_DTYPE_F32 : MOE_DTYPE_BF16, ld[0], ws, ws_bytes, p);
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

/* bind_attention(append, attention, quantize_fp8, gemm_fp8, float8_e4m3fn): the same for the attention half, after bind */
static PyObject* bind_attention(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    void* f[4];
    int i;
    (void)self;
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "bind_attention takes four addresses and a dtype");
        return NULL;
    }
    for (i = 0; i < 4; ++i) f[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return NULL;
    f_append = (append_fn)f[0];
    f_attention = (attention_fn)f[1];
    f_quantize_fp8 = (quantize_fp8_fn)f[2];
    f_gemm_fp8 = (gemm_fp8_fn)f[3];
    Py_XSETREF(t_e4m3, Py_NewRef(a[4]));
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, NULL},
                                {"bind_attention", (PyCFunction)(void (*)(void))bind_attention, METH_FASTCALL, NULL},
                                {"norm_residual", (PyCFunction)(void (*)(void))norm_residual, METH_FASTCALL, NULL},
                                {"select_experts", (PyCFunction)(void (*)(void))select_experts, METH_FASTCALL, NULL},
                                {"adapter_add", (PyCFunction)(void (*)(void))adapter_add, METH_FASTCALL, NULL},
                                {"cache_append", (PyCFunction)(void (*)(void))cache_append, METH_FASTCALL, NULL},
                                {"paged_attention", (PyCFunction)(void (*)(void))paged_attention, METH_FASTCALL, NULL},
                                {"quantize_fp8", (PyCFunction)(void (*)(void))quantize_fp8, METH_FASTCALL, NULL},
                                {"gemm_fp8", (PyCFunction)(void (*)(void))gemm_fp8, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__calls(void)
{
    s_dtype = PyUnicode_InternFromString("dtype");
    s_is_cuda = PyUnicode_InternFromString("is_cuda");
    s_shape = PyUnicode_InternFromString("shape");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_stride = PyUnicode_InternFromString("stride");
    if (!s_stride || !s_dtype || !s_is_cuda || !s_shape || !s_is_contiguous || !s_data_ptr) return NULL;
    return PyModule_Create(&module);
}
