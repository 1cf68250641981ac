/*
 * pa_block_calls.c -- the binding of the block-scaled and block-sparse calls, of
 * linear attention and of the sequence calls (CPython C API): checks of torch
 * tensors' types, shapes and devices, and the calls of include/pa.h, in one step.
 * A decode step makes several of these calls a layer; through ctypes the checks and
 * the marshalling of about 20 arguments took longer than the launch (8 against 4 us
 * a call).
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>

#include "pa.h"

static PyObject *t_i32, *t_i64, *t_f32, *t_u8, *t_i8, *t_f16, *t_bf16; /* torch dtypes */
static PyObject *error_class, *current_device, *raw_stream;    /* given by bind() */
static PyObject *n_shape, *n_dtype, *n_stride, *n_is_contiguous, *n_data_ptr, *n_get_device,
    *n_numel, *n_nbytes, *n_cuda_stream;

static int bad(const char *what)
{
    PyErr_SetString(PyExc_ValueError, what);
    return -1;
}

/* ---- what a tensor says of itself; -1 with an exception set on failure ---- */

static int64_t int_of(PyObject *v) /* steals v */
{
    if (!v)
        return -1;
    const int64_t x = PyLong_AsLongLong(v);
    Py_DECREF(v);
    return x;
}

/* A tuple of at most `most` integers (a shape, strides); its length. */
static int ints_of(PyObject *v, int64_t *out, int most) /* steals v */
{
    if (!v)
        return -1;
    if (!PyTuple_Check(v)) {
        Py_DECREF(v);
        PyErr_SetString(PyExc_TypeError, "a torch tensor is wanted");
        return -1;
    }
    const Py_ssize_t n = PyTuple_GET_SIZE(v);
    for (Py_ssize_t i = 0; i < n && i < most; ++i)
        out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(v, i));
    Py_DECREF(v);
    return PyErr_Occurred() ? -1 : (int)n;
}

static int shape_of(PyObject *t, int64_t *out, int most)
{
    return ints_of(PyObject_GetAttr(t, n_shape), out, most);
}

static int strides_of(PyObject *t, int64_t *out, int most)
{
    return ints_of(PyObject_CallMethodNoArgs(t, n_stride), out, most);
}

/* Whether t has this dtype; any: fp16 or bf16.  1, 0, or -1. */
static int has_dtype(PyObject *t, PyObject *want)
{
    PyObject *d = PyObject_GetAttr(t, n_dtype);
    if (!d)
        return -1;
    Py_DECREF(d); /* dtypes live as long as torch does */
    return d == want;
}

/* PA_FP16, PA_BF16, 2 for another dtype, or -1. */
static int half_kind(PyObject *t)
{
    PyObject *d = PyObject_GetAttr(t, n_dtype);
    if (!d)
        return -1;
    Py_DECREF(d);
    return d == t_f16 ? PA_FP16 : d == t_bf16 ? PA_BF16 : 2;
}

static int contiguous(PyObject *t)
{
    PyObject *v = PyObject_CallMethodNoArgs(t, n_is_contiguous);
    if (!v)
        return -1;
    const int yes = v == Py_True;
    Py_DECREF(v);
    return yes;
}

static void *pointer(PyObject *t)
{
    return (void *)(uintptr_t)int_of(PyObject_CallMethodNoArgs(t, n_data_ptr));
}

/* dtype, shape and contiguity at once: 0, or -1 with `what` raised. */
static int is(PyObject *t, PyObject *dtype, const int64_t *shape, int dims, const char *what)
{
    int64_t s[8];
    const int n = shape_of(t, s, 8);
    if (n < 0)
        return -1;
    int ok = n == dims;
    for (int i = 0; ok && i < dims; ++i)
        ok = s[i] == shape[i];
    if (ok) {
        ok = has_dtype(t, dtype);
        if (ok == 1)
            ok = contiguous(t);
    }
    return ok < 0 ? -1 : ok ? 0 : bad(what);
}

/* A contiguous int32 tensor of n numbers, of any shape. */
static int is_i32_of(PyObject *t, int64_t n, const char *what)
{
    const int64_t have = int_of(PyObject_CallMethodNoArgs(t, n_numel));
    if (have == -1 && PyErr_Occurred())
        return -1;
    int ok = have == n ? has_dtype(t, t_i32) : 0;
    if (ok == 1)
        ok = contiguous(t);
    return ok < 0 ? -1 : ok ? 0 : bad(what);
}

/* All tensors (NULLs left out) on the current device: a pointer of another one
 * would reach this device's kernels.  Its number, or -1. */
static int here(const char *const *names, PyObject *const *tensors, int n)
{
    int device = -2, mixed = 0;
    int at[16];
    for (int i = 0; i < n; ++i) {
        at[i] = -2;
        if (!tensors[i])
            continue;
        at[i] = (int)int_of(PyObject_CallMethodNoArgs(tensors[i], n_get_device));
        if (at[i] == -1 && PyErr_Occurred())
            return -1;
        if (at[i] < 0) {
            PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", names[i]);
            return -1;
        }
        mixed |= device != -2 && at[i] != device;
        device = at[i];
    }
    const int current = (int)int_of(PyObject_CallNoArgs(current_device));
    if (current == -1 && PyErr_Occurred())
        return -1;
    if (mixed || device != current)
        for (int i = 0; i < n; ++i)
            if (at[i] != -2 && at[i] != current) {
                PyErr_Format(PyExc_ValueError, "%s must be on the current device, cuda:%d",
                             names[i], current);
                return -1;
            }
    return current;
}

/* The raw handle of a stream argument: None (the current one), a number, or
 * an object with a cuda_stream. */
static int stream_of(PyObject *stream, int device, void **out)
{
    PyObject *v;
    if (stream == Py_None) {
        PyObject *d = PyLong_FromLong(device);
        if (!d)
            return -1;
        v = PyObject_CallOneArg(raw_stream, d);
        Py_DECREF(d);
    } else if (PyLong_Check(stream)) {
        v = Py_NewRef(stream);
    } else {
        v = PyObject_GetAttr(stream, n_cuda_stream);
    }
    if (!v)
        return -1;
    *out = (void *)(uintptr_t)PyLong_AsUnsignedLongLong(v);
    Py_DECREF(v);
    return PyErr_Occurred() ? -1 : 0;
}

/* Without the interpreter's lock, as through ctypes: a launch waits where the
 * device's queue is full, and other threads go on meanwhile.  The caller holds
 * the tensors. */
#define UNLOCKED(call)      \
    Py_BEGIN_ALLOW_THREADS  \
    call;                   \
    Py_END_ALLOW_THREADS

static PyObject *done(pa_status st, const char *where)
{
    if (st == PA_OK)
        Py_RETURN_NONE;
    PyObject *e = PyObject_CallFunction(error_class, "is", (int)st, where);
    if (e) {
        PyErr_SetObject(error_class, e);
        Py_DECREF(e);
    }
    return NULL;
}

static int to_int(PyObject *v, int *out)
{
    const long long x = PyLong_AsLongLong(v);
    if (x == -1 && PyErr_Occurred())
        return -1;
    if (x < INT32_MIN || x > INT32_MAX)
        return bad("a size does not fit 32 bits");
    *out = (int)x;
    return 0;
}

/* ---- arguments that several calls share ---- */

typedef struct {
    int64_t num_blocks, kv_heads, head_size;
    void *pool;
    float *scales; /* NULL: a 16-bit pool */
    int kind;      /* its dtype */
} Pool;

static int read_pool(PyObject *cache, PyObject *scales, int block_size, Pool *p)
{
    int64_t s[5];
    const int n = shape_of(cache, s, 5);
    if (n < 0)
        return -1;
    if (n != 5 || s[0] != 2 || s[2] != block_size)
        return bad("kv_cache must be [2, num_blocks, block_size, num_kv_heads, head_size]");
    const int c = contiguous(cache);
    if (c != 1)
        return c < 0 ? -1 : bad("kv_cache must be contiguous");
    p->num_blocks = s[1], p->kv_heads = s[3], p->head_size = s[4];
    p->scales = NULL;
    if (scales == Py_None) {
        p->kind = half_kind(cache);
        if (p->kind < 0 || p->kind == 2)
            return p->kind < 0 ? -1 : bad("a pool without kv_scales must be float16 or bfloat16");
    } else {
        const int u = has_dtype(cache, t_u8);
        if (u != 1)
            return u < 0 ? -1 : bad("a pool with kv_scales must be a uint8 tensor of e4m3 codes");
        const int64_t want[3] = {2, s[1], s[3]};
        if (is(scales, t_f32, want, 3,
               "kv_scales must be contiguous float32 [2, num_blocks, num_kv_heads]"))
            return -1;
        p->scales = (float *)pointer(scales);
        p->kind = PA_FP16;
    }
    p->pool = pointer(cache);
    return PyErr_Occurred() ? -1 : 0;
}

typedef struct {
    int64_t count, blocks, stride; /* requests; entries and stride of a table row */
} Requests;

static int read_requests(PyObject *tables, PyObject *seq_lens, PyObject *starts, Requests *r)
{
    int64_t s[2], st[2];
    r->count = int_of(PyObject_CallMethodNoArgs(seq_lens, n_numel));
    if (r->count < 0)
        return -1;
    if (is_i32_of(seq_lens, r->count, "seq_lens must be contiguous int32 [R]"))
        return -1;
    const int n = shape_of(tables, s, 2);
    if (n < 0 || (n == 2 && strides_of(tables, st, 2) < 0))
        return -1;
    int ok = n == 2 ? has_dtype(tables, t_i32) : 0;
    if (ok < 0)
        return -1;
    if (!ok || s[0] != r->count || (st[1] != 1 && s[1] != 1) || (st[0] < s[1] && r->count > 1))
        return bad("block_tables must be int32 [R, max_blocks] with contiguous rows");
    r->blocks = s[1];
    r->stride = st[0] > s[1] ? st[0] : s[1];
    return is_i32_of(starts, r->count + 1, "query_start_loc must be contiguous int32 [R + 1]");
}

typedef struct {
    int64_t seqs, heads, blocks;
    int kind;
} Queries;

static int read_queries(PyObject *q, int64_t head_size, PyObject *tables, PyObject *seq_lens,
                        Queries *r)
{
    int64_t s[3];
    const int n = shape_of(q, s, 3);
    if (n < 0)
        return -1;
    int ok = n == 3 && s[2] == head_size;
    r->kind = ok ? half_kind(q) : 2;
    ok = r->kind == 2 ? 0 : r->kind < 0 ? -1 : contiguous(q);
    if (ok != 1)
        return ok < 0 ? -1 : bad("q must be contiguous fp16/bf16 [B, H, head_size]");
    r->seqs = s[0], r->heads = s[1];
    const int m = shape_of(tables, s, 2);
    if (m < 0)
        return -1;
    ok = m == 2 && s[0] == r->seqs ? has_dtype(tables, t_i32) : 0;
    if (ok == 1)
        ok = contiguous(tables);
    if (ok != 1)
        return ok < 0 ? -1 : bad("block_tables must be contiguous int32 [B, max_blocks_per_seq]");
    r->blocks = s[1];
    return is_i32_of(seq_lens, r->seqs, "seq_lens must be contiguous int32 [B]");
}

static int read_out(PyObject *out, PyObject *lse, const Queries *r, int64_t head_size)
{
    const int64_t want[3] = {r->seqs, r->heads, head_size};
    if (is(out, r->kind == PA_BF16 ? t_bf16 : t_f16, want, 3, "out must be contiguous and match q"))
        return -1;
    return lse == Py_None ? 0 : is(lse, t_f32, want, 2, "lse must be contiguous float32 [B, H]");
}

static int read_lists(PyObject *lists, PyObject *lens, int64_t seqs, int64_t kv_heads, int64_t *most)
{
    int64_t s[3];
    const int n = shape_of(lists, s, 3);
    if (n < 0)
        return -1;
    int ok = n == 3 && s[0] == seqs && s[1] == kv_heads ? has_dtype(lists, t_i32) : 0;
    if (ok == 1)
        ok = contiguous(lists);
    if (ok != 1)
        return ok < 0 ? -1
                      : bad("block_lists must be contiguous int32 [B, num_kv_heads, max_selected]");
    *most = s[2];
    return is_i32_of(lens, seqs, "list_lens must be contiguous int32 [B]");
}

static int read_bounds(PyObject *bounds, PyObject *scale, int64_t nb, int64_t hkv, int64_t d)
{
    const int64_t want[4] = {nb, hkv, 2, d};
    if (is(bounds, t_i8, want, 4,
           "bounds must be contiguous int8 [num_blocks, num_kv_heads, 2, head_size]"))
        return -1;
    return is(scale, t_f32, want, 2,
              "bounds_scale must be contiguous float32 [num_blocks, num_kv_heads]");
}

static int read_workspace(PyObject *ws, void **p, size_t *bytes)
{
    const int c = contiguous(ws);
    if (c != 1)
        return c < 0 ? -1 : bad("workspace must be contiguous");
    *p = pointer(ws);
    *bytes = (size_t)int_of(PyObject_GetAttr(ws, n_nbytes));
    return PyErr_Occurred() ? -1 : 0;
}

static int count(Py_ssize_t n, Py_ssize_t want)
{
    if (n == want)
        return 0;
    PyErr_Format(PyExc_TypeError, "%zd arguments are wanted", want);
    return -1;
}

/* The sizes of pa.h's arguments are 32-bit; what a tensor's are not is refused. */
static int fit(const int64_t *v, int n)
{
    for (int i = 0; i < n; ++i)
        if (v[i] > INT32_MAX)
            return bad("a size does not fit 32 bits");
    return 0;
}

/* ---- the calls ---- */

/* key, value, kv_cache, kv_scales, block_tables, seq_lens, query_start_loc,
 * block_size, max_query_len, stream */
static PyObject *write_block(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    static const char *const names[] = {"key",          "value",    "kv_cache",       "kv_scales",
                                        "block_tables", "seq_lens", "query_start_loc"};
    int bs, most, device;
    Pool p;
    Requests r;
    int64_t s[3], ks[3], vs[3], v[3];
    void *stream;
    if (count(n, 10) || to_int(a[7], &bs) || to_int(a[8], &most))
        return NULL;
    if (a[3] == Py_None) {
        bad("kv_scales is required");
        return NULL;
    }
    if (read_pool(a[2], a[3], bs, &p) || read_requests(a[4], a[5], a[6], &r))
        return NULL;
    const int dk = shape_of(a[0], s, 3), dv = shape_of(a[1], v, 3);
    const int kind = half_kind(a[0]), other = half_kind(a[1]);
    if (dk < 0 || dv < 0 || kind < 0 || other < 0)
        return NULL;
    if (kind == 2 || other != kind || dk != 3 || dv != 3 || s[1] != p.kv_heads ||
        s[2] != p.head_size || v[0] != s[0] || v[1] != s[1] || v[2] != s[2]) {
        bad("key and value must be fp16/bf16 [T, num_kv_heads, head_size] alike");
        return NULL;
    }
    if (strides_of(a[0], ks, 3) < 0 || strides_of(a[1], vs, 3) < 0)
        return NULL;
    const int64_t row = p.kv_heads * p.head_size;
    if (ks[2] != 1 || vs[2] != 1 || (s[1] > 1 && (ks[1] != s[2] || vs[1] != s[2])) ||
        (s[0] > 1 && (ks[0] < row || vs[0] < row))) {
        bad("key and value must have contiguous rows that do not overlap");
        return NULL;
    }
    if (s[0] == 0 || r.count == 0)
        Py_RETURN_NONE;
    const int64_t sizes[] = {r.count, s[0], p.kv_heads, p.num_blocks, r.blocks};
    if (fit(sizes, 5) || (device = here(names, a, 7)) < 0 || stream_of(a[9], device, &stream))
        return NULL;
    void *const key = pointer(a[0]), *const value = pointer(a[1]);
    const int32_t *const tables = pointer(a[4]), *const lens = pointer(a[5]),
                        *const starts = pointer(a[6]);
    if (PyErr_Occurred())
        return NULL;
    pa_status st;
    UNLOCKED(st = pa_reshape_and_cache_fp8_block(
                      key, value, p.pool, p.scales, tables, r.stride, lens, starts, (int)r.count,
                      (int)s[0], most, (int)p.kv_heads, (int)p.head_size, bs, (int)p.num_blocks,
                      (int)r.blocks, s[0] > 1 ? ks[0] : row, s[0] > 1 ? vs[0] : row, (pa_dtype)kind,
                      stream));
    return done(st, "pa_reshape_and_cache_fp8_block");
}

/* out, q, kv_cache, kv_scales, block_tables, seq_lens, workspace, lse, scale,
 * block_size, max_seq_len, stream */
static PyObject *decode_block(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    static const char *const names[] = {"out",          "q",        "kv_cache",  "kv_scales",
                                        "block_tables", "seq_lens", "workspace", "lse"};
    int bs, most, device;
    Pool p;
    Queries r;
    void *stream, *ws;
    size_t bytes;
    if (count(n, 12) || to_int(a[9], &bs) || to_int(a[10], &most))
        return NULL;
    const double scale = PyFloat_AsDouble(a[8]);
    if (scale == -1.0 && PyErr_Occurred())
        return NULL;
    if (a[3] == Py_None) {
        bad("kv_scales is required");
        return NULL;
    }
    if (read_pool(a[2], a[3], bs, &p) || read_queries(a[1], p.head_size, a[4], a[5], &r) ||
        read_out(a[0], a[7], &r, p.head_size) || read_workspace(a[6], &ws, &bytes))
        return NULL;
    PyObject *const all[] = {a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7] == Py_None ? NULL : a[7]};
    const int64_t sizes[] = {r.seqs, r.heads, p.kv_heads, p.num_blocks, r.blocks};
    if (fit(sizes, 5) || (device = here(names, all, 8)) < 0 || stream_of(a[11], device, &stream))
        return NULL;
    void *const out = pointer(a[0]), *const q = pointer(a[1]);
    const int32_t *const tables = pointer(a[4]), *const lens = pointer(a[5]);
    float *const lse = all[7] ? pointer(all[7]) : NULL;
    if (PyErr_Occurred())
        return NULL;
    pa_status st;
    UNLOCKED(st = pa_decode_fp8_block(out, lse, q, p.pool, p.scales, tables, lens, (int)r.seqs,
                                      (int)r.heads, (int)p.kv_heads, (int)p.head_size, bs,
                                      (int)p.num_blocks, (int)r.blocks, (float)scale,
                                      (pa_dtype)r.kind, most, ws, bytes, stream));
    return done(st, "pa_decode_fp8_block");
}

/* bounds, bounds_scale, kv_cache, block_tables, seq_lens, query_start_loc,
 * kv_scales, block_size, max_query_len, stream */
static PyObject *update_bounds(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    static const char *const names[] = {"bounds",   "bounds_scale",    "kv_cache", "block_tables",
                                        "seq_lens", "query_start_loc", "kv_scales"};
    int bs, most, device;
    Pool p;
    Requests r;
    void *stream;
    if (count(n, 10) || to_int(a[7], &bs) || to_int(a[8], &most) ||
        read_pool(a[2], a[6], bs, &p) ||
        read_bounds(a[0], a[1], p.num_blocks, p.kv_heads, p.head_size) ||
        read_requests(a[3], a[4], a[5], &r))
        return NULL;
    if (r.count == 0)
        Py_RETURN_NONE;
    PyObject *const all[] = {a[0], a[1], a[2], a[3], a[4], a[5], a[6] == Py_None ? NULL : a[6]};
    const int64_t sizes[] = {r.count, p.kv_heads, p.num_blocks, r.blocks};
    if (fit(sizes, 4) || (device = here(names, all, 7)) < 0 || stream_of(a[9], device, &stream))
        return NULL;
    int8_t *const bounds = pointer(a[0]);
    float *const scale = pointer(a[1]);
    const int32_t *const tables = pointer(a[3]), *const lens = pointer(a[4]),
                        *const starts = pointer(a[5]);
    if (PyErr_Occurred())
        return NULL;
    pa_status st;
    UNLOCKED(st = pa_update_block_bounds(bounds, scale, p.pool, p.scales, tables, r.stride, lens,
                                         starts, (int)r.count, most, (int)p.kv_heads,
                                         (int)p.head_size, bs, (int)p.num_blocks, (int)r.blocks,
                                         (pa_dtype)p.kind, stream));
    return done(st, "pa_update_block_bounds");
}

/* block_lists, list_lens, q, bounds, bounds_scale, block_tables, seq_lens,
 * workspace, block_size, max_seq_len, num_sink_blocks, num_recent_blocks, stream */
static PyObject *select_blocks(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    static const char *const names[] = {"block_lists",  "list_lens",    "q",        "bounds",
                                        "bounds_scale", "block_tables", "seq_lens", "workspace"};
    int bs, most, sink, recent, device;
    Queries r;
    int64_t s[4], listed;
    void *stream, *ws;
    size_t bytes;
    if (count(n, 13) || to_int(a[8], &bs) || to_int(a[9], &most) || to_int(a[10], &sink) ||
        to_int(a[11], &recent))
        return NULL;
    const int dims = shape_of(a[3], s, 4);
    if (dims < 0)
        return NULL;
    if (dims != 4) {
        bad("bounds must be contiguous int8 [num_blocks, num_kv_heads, 2, head_size]");
        return NULL;
    }
    if (read_bounds(a[3], a[4], s[0], s[1], s[3]) || read_queries(a[2], s[3], a[5], a[6], &r) ||
        read_lists(a[0], a[1], r.seqs, s[1], &listed) || read_workspace(a[7], &ws, &bytes))
        return NULL;
    const int64_t sizes[] = {r.seqs, r.heads, s[0], s[1], r.blocks, listed};
    if (fit(sizes, 6) || (device = here(names, a, 8)) < 0 || stream_of(a[12], device, &stream))
        return NULL;
    int32_t *const lists = pointer(a[0]), *const lens = pointer(a[1]);
    const void *const q = pointer(a[2]);
    const int8_t *const bounds = pointer(a[3]);
    const float *const scale = pointer(a[4]);
    const int32_t *const tables = pointer(a[5]), *const seq_lens = pointer(a[6]);
    if (PyErr_Occurred())
        return NULL;
    pa_status st;
    UNLOCKED(st = pa_select_blocks(lists, lens, q, bounds, scale, tables, seq_lens, (int)r.seqs,
                                   (int)r.heads, (int)s[1], (int)s[3], bs, (int)s[0], (int)r.blocks,
                                   (int)listed, sink, recent, (pa_dtype)r.kind, most, ws, bytes,
                                   stream));
    return done(st, "pa_select_blocks");
}

/* out, q, kv_cache, block_tables, seq_lens, block_lists, list_lens, workspace,
 * kv_scales, lse, scale, block_size, stream */
static PyObject *decode_sparse(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    static const char *const names[] = {"out",         "q",         "kv_cache",  "block_tables", "seq_lens",
                                        "block_lists", "list_lens", "workspace", "kv_scales",    "lse"};
    int bs, device;
    Pool p;
    Queries r;
    int64_t listed;
    void *stream, *ws;
    size_t bytes;
    if (count(n, 13) || to_int(a[11], &bs))
        return NULL;
    const double scale = PyFloat_AsDouble(a[10]);
    if (scale == -1.0 && PyErr_Occurred())
        return NULL;
    if (read_pool(a[2], a[8], bs, &p) || read_queries(a[1], p.head_size, a[3], a[4], &r) ||
        read_out(a[0], a[9], &r, p.head_size))
        return NULL;
    if (!p.scales && r.kind != p.kind) {
        bad("q and a 16-bit kv_cache must share their dtype");
        return NULL;
    }
    if (read_lists(a[5], a[6], r.seqs, p.kv_heads, &listed) || read_workspace(a[7], &ws, &bytes))
        return NULL;
    PyObject *const all[] = {a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7],
                             a[8] == Py_None ? NULL : a[8], a[9] == Py_None ? NULL : a[9]};
    const int64_t sizes[] = {r.seqs, r.heads, p.kv_heads, p.num_blocks, r.blocks, listed};
    if (fit(sizes, 6) || (device = here(names, all, 10)) < 0 || stream_of(a[12], device, &stream))
        return NULL;
    void *const out = pointer(a[0]), *const q = pointer(a[1]);
    const int32_t *const tables = pointer(a[3]), *const seq_lens = pointer(a[4]),
                        *const lists = pointer(a[5]), *const lens = pointer(a[6]);
    float *const lse = all[9] ? pointer(all[9]) : NULL;
    if (PyErr_Occurred())
        return NULL;
    pa_status st;
    UNLOCKED(st = pa_decode_sparse(out, lse, q, p.pool, p.scales, tables, seq_lens, lists, lens,
                                   (int)r.seqs, (int)r.heads, (int)p.kv_heads, (int)p.head_size, bs,
                                   (int)p.num_blocks, (int)r.blocks, (int)listed, (float)scale,
                                   (pa_dtype)r.kind, ws, bytes, stream));
    return done(st, "pa_decode_sparse");
}

/* ---- linear attention ---- */

/* Rows [T, heads, head_size] of a tensor, contiguous but for the token stride. */
typedef struct {
    int64_t tokens, heads, head_size, stride;
    int kind;
} Rows;

static int read_rows(PyObject *t, Rows *r, const char *what)
{
    int64_t s[3], st[3];
    const int n = shape_of(t, s, 3);
    if (n < 0)
        return -1;
    if (n != 3)
        return bad(what);
    r->kind = half_kind(t);
    if (r->kind < 0 || strides_of(t, st, 3) < 0)
        return -1;
    r->tokens = s[0], r->heads = s[1], r->head_size = s[2];
    const int64_t row = s[1] * s[2];
    if (r->kind == 2 || (s[2] > 1 && st[2] != 1) || (s[1] > 1 && st[1] != s[2]) ||
        (s[0] > 1 && st[0] < row))
        return bad(what);
    r->stride = s[0] > 1 ? st[0] : row;
    return 0;
}

typedef struct {
    Rows q, k, v;
    int64_t decay_stride, num_states, seqs;
} Linear;

/* out, q, k, v, log_decay, states, src_states, dst_states */
static int read_linear(PyObject *const *a, Linear *l)
{
    int64_t s[4], st[2];
    if (read_rows(a[1], &l->q, "q must be fp16/bf16 [T, H, head_size] with contiguous rows") ||
        read_rows(a[2], &l->k, "k must be fp16/bf16 [T, num_kv_heads, head_size] with contiguous rows") ||
        read_rows(a[3], &l->v, "v must be fp16/bf16 [T, num_kv_heads, head_size] with contiguous rows"))
        return -1;
    if (l->k.kind != l->q.kind || l->v.kind != l->q.kind || l->k.tokens != l->q.tokens ||
        l->v.tokens != l->q.tokens || l->k.head_size != l->q.head_size ||
        l->v.head_size != l->q.head_size || l->v.heads != l->k.heads)
        return bad("q, k and v must share dtype, token count and head_size, k and v their heads");
    const int64_t want[3] = {l->q.tokens, l->q.heads, l->q.head_size};
    if (is(a[0], l->q.kind == PA_BF16 ? t_bf16 : t_f16, want, 3, "out must be contiguous and match q"))
        return -1;
    static const char *const decays =
        "log_decay must be float32 [num_kv_heads] or [T, num_kv_heads] with contiguous rows";
    const int n = shape_of(a[4], s, 4), f = has_dtype(a[4], t_f32);
    if (n < 0 || f < 0)
        return -1;
    if (!f || n < 1 || n > 2 || s[n - 1] != l->k.heads || (n == 2 && s[0] != l->q.tokens))
        return bad(decays);
    if (strides_of(a[4], st, 2) < 0)
        return -1;
    if (s[n - 1] > 1 && st[n - 1] != 1)
        return bad(decays);
    l->decay_stride = n == 1 ? 0 : s[0] > 1 ? st[0] : l->k.heads;
    const int m = shape_of(a[5], s, 4);
    if (m < 0)
        return -1;
    const int64_t states[4] = {m == 4 ? s[0] : 0, l->k.heads, l->q.head_size, l->q.head_size};
    if (is(a[5], t_f32, states, 4,
           "states must be contiguous float32 [num_states, num_kv_heads, head_size, head_size]"))
        return -1;
    l->num_states = s[0];
    l->seqs = int_of(PyObject_CallMethodNoArgs(a[7], n_numel));
    if (l->seqs < 0)
        return -1;
    if (is_i32_of(a[6], l->seqs, "src_states must be contiguous int32 [num_seqs]") ||
        is_i32_of(a[7], l->seqs, "dst_states must be contiguous int32 [num_seqs]"))
        return -1;
    const int64_t sizes[] = {l->q.tokens, l->q.heads, l->num_states, l->seqs};
    return fit(sizes, 4);
}

/* out, q, k, v, log_decay, states, src_states, dst_states, scale, stream */
static PyObject *linear_decode(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    static const char *const names[] = {"out",       "q",      "k",          "v",
                                        "log_decay", "states", "src_states", "dst_states"};
    Linear l;
    int device;
    void *stream, *p[8];
    if (count(n, 10))
        return NULL;
    const double scale = PyFloat_AsDouble(a[8]);
    if ((scale == -1.0 && PyErr_Occurred()) || read_linear(a, &l))
        return NULL;
    if (l.seqs != l.q.tokens) {
        bad("src_states and dst_states must have one number for each token");
        return NULL;
    }
    if ((device = here(names, a, 8)) < 0 || stream_of(a[9], device, &stream))
        return NULL;
    for (int i = 0; i < 8; ++i)
        p[i] = pointer(a[i]);
    if (PyErr_Occurred())
        return NULL;
    pa_status st;
    UNLOCKED(st = pa_linear_decode(p[0], p[1], p[2], p[3], p[4], l.decay_stride, p[5], p[6], p[7],
                                   (int)l.seqs, (int)l.q.heads, (int)l.k.heads, (int)l.q.head_size,
                                   (int)l.num_states, l.q.stride, l.k.stride, l.v.stride,
                                   (float)scale, (pa_dtype)l.q.kind, stream));
    return done(st, "pa_linear_decode");
}

/* out, q, k, v, log_decay, states, src_states, dst_states, query_start_loc,
 * workspace, scale, max_query_len, stream */
static PyObject *linear_prefill(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    static const char *const names[] = {"out",        "q",          "k",      "v",
                                        "log_decay",  "states",     "src_states",
                                        "dst_states", "query_start_loc", "workspace"};
    Linear l;
    int device, most;
    void *stream, *ws, *p[9];
    size_t bytes;
    if (count(n, 13) || to_int(a[11], &most))
        return NULL;
    const double scale = PyFloat_AsDouble(a[10]);
    if ((scale == -1.0 && PyErr_Occurred()) || read_linear(a, &l) ||
        is_i32_of(a[8], l.seqs + 1, "query_start_loc must be contiguous int32 [num_seqs + 1]") ||
        read_workspace(a[9], &ws, &bytes))
        return NULL;
    if ((device = here(names, a, 10)) < 0 || stream_of(a[12], device, &stream))
        return NULL;
    for (int i = 0; i < 9; ++i)
        p[i] = pointer(a[i]);
    if (PyErr_Occurred())
        return NULL;
    pa_status st;
    UNLOCKED(st = pa_linear_prefill(p[0], p[1], p[2], p[3], p[4], l.decay_stride, p[5], p[6], p[7],
                                    p[8], (int)l.seqs, (int)l.q.tokens, most, (int)l.q.heads,
                                    (int)l.k.heads, (int)l.q.head_size, (int)l.num_states,
                                    l.q.stride, l.k.stride, l.v.stride, (float)scale,
                                    (pa_dtype)l.q.kind, ws, bytes, stream));
    return done(st, "pa_linear_prefill");
}

/* ---- sequences ---- */

typedef struct {
    int64_t rows, blocks, num_blocks; /* rows, entries of one, blocks of the pool */
} Tables;

/* block_tables, seq_lens, ref_counts */
static int read_tables(PyObject *tables, PyObject *lens, PyObject *refs, Tables *t)
{
    int64_t s[2];
    const int n = shape_of(tables, s, 2);
    if (n < 0)
        return -1;
    int ok = n == 2 ? has_dtype(tables, t_i32) : 0;
    if (ok == 1)
        ok = contiguous(tables);
    if (ok != 1)
        return ok < 0 ? -1 : bad("block_tables must be contiguous int32 [rows, max_blocks_per_seq]");
    t->rows = s[0], t->blocks = s[1];
    t->num_blocks = int_of(PyObject_CallMethodNoArgs(refs, n_numel));
    if (t->num_blocks < 0)
        return -1;
    return is_i32_of(lens, t->rows, "seq_lens must be contiguous int32 [rows]") ||
                   is_i32_of(refs, t->num_blocks, "ref_counts must be contiguous int32 [num_blocks]")
               ? -1
               : fit(&t->num_blocks, 1);
}

static int read_tables_out(PyObject *tables, PyObject *lens, PyObject *refs, int64_t rows,
                           const Tables *t)
{
    const int64_t want[2] = {rows, t->blocks};
    if (is(tables, t_i32, want, 2,
           "tables_out must be contiguous int32 [rows, max_blocks_per_seq] as wide as block_tables"))
        return -1;
    if (lens && is_i32_of(lens, rows, "seq_lens_out must be contiguous int32 [rows]"))
        return -1;
    return is_i32_of(refs, t->num_blocks, "ref_counts_out must be contiguous int32 [num_blocks]");
}

/* A list or tuple of tensors [planes, num_blocks, ...] on `device`; their number. */
static int read_block_pools(PyObject *pools, int64_t num_blocks, int device, pa_block_pool *to)
{
    static const char *const wanted =
        "pools must be a list of contiguous CUDA tensors [planes, num_blocks, ...]";
    /* a tuple of its own: what the tensors' methods run, and other threads meanwhile, may
     * change a list */
    PyObject *list = PySequence_Tuple(pools);
    if (!list)
        return -1;
    const Py_ssize_t n = PyTuple_GET_SIZE(list);
    int st = n <= PA_MAX_POOLS ? 0 : bad("too many pools for one call");
    for (Py_ssize_t i = 0; i < n && !st; ++i) {
        PyObject *const t = PyTuple_GET_ITEM(list, i);
        int64_t s[2];
        const int dims = shape_of(t, s, 2);
        const int c = dims < 0 ? -1 : contiguous(t);
        if (c < 0) {
            st = -1;
            break;
        }
        const int64_t bytes = int_of(PyObject_GetAttr(t, n_nbytes));
        const int64_t on = int_of(PyObject_CallMethodNoArgs(t, n_get_device));
        if (PyErr_Occurred())
            st = -1;
        else if (!c || dims < 2 || s[1] != num_blocks || s[0] < 1 || s[0] > INT32_MAX || bytes <= 0)
            st = bad(wanted);
        else if (on != device)
            st = bad("pools must be on the current device");
        else {
            to[i].data = pointer(t);
            to[i].block_bytes = bytes / (s[0] * s[1]);
            to[i].planes = (int32_t)s[0];
            st = PyErr_Occurred() ? -1 : 0;
        }
    }
    Py_DECREF(list);
    return st ? -1 : (int)n;
}

/* tables_out, seq_lens_out, ref_counts_out, block_tables, seq_lens, ref_counts,
 * parents, block_size, stream */
static PyObject *fork_sequences(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    static const char *const names[] = {"tables_out", "seq_lens_out", "ref_counts_out", "block_tables",
                                        "seq_lens",   "ref_counts",   "parents"};
    Tables t;
    int bs, device;
    void *stream, *p[7];
    if (count(n, 9) || to_int(a[7], &bs) || read_tables(a[3], a[4], a[5], &t))
        return NULL;
    const int64_t rows = int_of(PyObject_CallMethodNoArgs(a[6], n_numel));
    if (rows < 0 || is_i32_of(a[6], rows, "parents must be contiguous int32 [rows of tables_out]") ||
        read_tables_out(a[0], a[1], a[2], rows, &t))
        return NULL;
    const int64_t sizes[] = {rows, t.rows, t.blocks};
    if (fit(sizes, 3) || (device = here(names, a, 7)) < 0 || stream_of(a[8], device, &stream))
        return NULL;
    for (int i = 0; i < 7; ++i)
        p[i] = pointer(a[i]);
    if (PyErr_Occurred())
        return NULL;
    pa_status st;
    UNLOCKED(st = pa_fork_sequences(p[0], p[1], p[2], p[3], p[4], p[5], p[6], (int)t.rows, (int)rows,
                                    (int)t.num_blocks, (int)t.blocks, bs, stream));
    return done(st, "pa_fork_sequences");
}

/* tables_out, seq_lens_out, ref_counts_out, slot_mapping, info, block_tables,
 * seq_lens, ref_counts, num_new, workspace, pools, block_size, stream */
static PyObject *extend_sequences(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    static const char *const names[] = {"tables_out", "seq_lens_out", "ref_counts_out", "slot_mapping",
                                        "info",       "block_tables", "seq_lens",       "ref_counts",
                                        "num_new",    "workspace"};
    Tables t;
    int bs, device, pools;
    size_t bytes;
    void *stream, *ws, *p[9];
    pa_block_pool pool[PA_MAX_POOLS];
    if (count(n, 13) || to_int(a[11], &bs) || read_tables(a[5], a[6], a[7], &t) ||
        read_tables_out(a[0], a[1], a[2], t.rows, &t) ||
        is_i32_of(a[4], 2, "info must be contiguous int32 [2]") ||
        is_i32_of(a[8], t.rows, "num_new must be contiguous int32 [rows]"))
        return NULL;
    const int64_t tokens = int_of(PyObject_CallMethodNoArgs(a[3], n_numel));
    if (tokens < 0 || is(a[3], t_i64, &tokens, 1, "slot_mapping must be contiguous int64 [T]") ||
        read_workspace(a[9], &ws, &bytes))
        return NULL;
    const int64_t sizes[] = {tokens, t.rows, t.blocks};
    if (fit(sizes, 3) || (device = here(names, a, 10)) < 0 ||
        (pools = read_block_pools(a[10], t.num_blocks, device, pool)) < 0 ||
        stream_of(a[12], device, &stream))
        return NULL;
    for (int i = 0; i < 9; ++i)
        p[i] = pointer(a[i]);
    if (PyErr_Occurred())
        return NULL;
    pa_status st;
    UNLOCKED(st = pa_extend_sequences(p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], pool,
                                      pools, (int)t.rows, (int)tokens, (int)t.num_blocks,
                                      (int)t.blocks, bs, ws, bytes, stream));
    return done(st, "pa_extend_sequences");
}

/* tables_out, ref_counts_out, new_ids, info, block_tables, seq_lens, ref_counts,
 * workspace, pools, block_size, stream */
static PyObject *compact_blocks(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    static const char *const names[] = {"tables_out",   "ref_counts_out", "new_ids",    "info",
                                        "block_tables", "seq_lens",       "ref_counts", "workspace"};
    Tables t;
    int bs, device, pools;
    size_t bytes;
    void *stream, *ws, *p[7];
    pa_block_pool pool[PA_MAX_POOLS];
    if (count(n, 11) || to_int(a[9], &bs) || read_tables(a[4], a[5], a[6], &t) ||
        read_tables_out(a[0], NULL, a[1], t.rows, &t) ||
        is_i32_of(a[2], t.num_blocks, "new_ids must be contiguous int32 [num_blocks]") ||
        is_i32_of(a[3], 2, "info must be contiguous int32 [2]") || read_workspace(a[7], &ws, &bytes))
        return NULL;
    const int64_t sizes[] = {t.rows, t.blocks};
    if (fit(sizes, 2) || (device = here(names, a, 8)) < 0 ||
        (pools = read_block_pools(a[8], t.num_blocks, device, pool)) < 0 ||
        stream_of(a[10], device, &stream))
        return NULL;
    for (int i = 0; i < 7; ++i)
        p[i] = pointer(a[i]);
    if (PyErr_Occurred())
        return NULL;
    pa_status st;
    UNLOCKED(st = pa_compact_blocks(p[0], p[1], p[2], p[3], p[4], p[5], p[6], pool, pools,
                                    (int)t.rows, (int)t.num_blocks, (int)t.blocks, bs, ws, bytes,
                                    stream));
    return done(st, "pa_compact_blocks");
}

/* The exception class of a failed call, and torch's functions for the current
 * device and its current raw stream. */
static PyObject *bind(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    if (count(n, 3))
        return NULL;
    Py_XSETREF(error_class, Py_NewRef(a[0]));
    Py_XSETREF(current_device, Py_NewRef(a[1]));
    Py_XSETREF(raw_stream, Py_NewRef(a[2]));
    Py_RETURN_NONE;
}

#define CALL(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {CALL(bind),          CALL(write_block),   CALL(decode_block),
                                CALL(update_bounds), CALL(select_blocks), CALL(decode_sparse),
                                CALL(linear_decode), CALL(linear_prefill),
                                CALL(fork_sequences), CALL(extend_sequences), CALL(compact_blocks),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "pa_block_calls", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit_pa_block_calls(void)
{
    PyObject *torch = PyImport_ImportModule("torch");
    if (!torch)
        return NULL;
    struct {
        PyObject **to;
        const char *name;
    } types[] = {{&t_i32, "int32"},   {&t_i64, "int64"},
                 {&t_f32, "float32"}, {&t_u8, "uint8"},
                 {&t_i8, "int8"},     {&t_f16, "float16"}, {&t_bf16, "bfloat16"}},
      names[] = {{&n_shape, "shape"},         {&n_dtype, "dtype"},
                 {&n_stride, "stride"},       {&n_is_contiguous, "is_contiguous"},
                 {&n_data_ptr, "data_ptr"},   {&n_get_device, "get_device"},
                 {&n_numel, "numel"},         {&n_nbytes, "nbytes"},
                 {&n_cuda_stream, "cuda_stream"}};
    int ok = 1;
    for (size_t i = 0; i < sizeof types / sizeof *types; ++i)
        ok &= (*types[i].to = PyObject_GetAttrString(torch, types[i].name)) != NULL;
    for (size_t i = 0; i < sizeof names / sizeof *names; ++i)
        ok &= (*names[i].to = PyUnicode_InternFromString(names[i].name)) != NULL;
    Py_DECREF(torch);
    return ok ? PyModule_Create(&module) : NULL;
}
