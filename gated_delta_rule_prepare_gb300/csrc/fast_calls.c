/* The binding's short calls in C: a decode step makes them once a layer, and Python's reading of
 * a tensor's attributes takes longer than the kernels (a rotary call: 12 us in Python).  Each
 * function takes the arguments of the Python function of its name, all of them, checks what is
 * passed down, and calls the library.  It returns the call's kda_status, or -1 for anything out of
 * the ordinary (another device, a wrong type or shape, no workspace): then nothing has been
 * called, and the Python function, which names what is wrong, does it all again. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "kda.h"

enum { D = KDA_HEAD_DIM };

static PyObject *n_dtype, *n_shape, *n_get_device, *n_data_ptr, *n_stride;
static PyObject *bf16, *f16, *f32, *i32, *u8, *raw_stream, *current_device;

/* The library's functions, by address: this module is linked to nothing. */
static kda_status (*lin_prefill_)(const float*, float*, const void*, const void*, const void*,
                                  const float*, void*, int, int, const int*, int, int, int, int,
                                  int, int64_t, int64_t, int64_t, int64_t, int64_t, float, void*,
                                  size_t, uint64_t);
static kda_status (*lin_decode_)(const float*, float*, const void*, const void*, const void*,
                                 const float*, void*, int, int, int, int, int, int, int64_t,
                                 int64_t, int64_t, int64_t, int64_t, float, float* const*, int,
                                 uint64_t);
static kda_status (*rope_)(const void*, const void*, void*, void*, int64_t, int, int, int, int,
                           int64_t, int64_t, int64_t, int64_t, const int*, int, const float*, int,
                           const uint8_t*, int, float, uint64_t);
static kda_status (*resize_)(int*, const int*, int*, int, int, int64_t, int, void*, size_t,
                             uint64_t);
static kda_status (*fork_)(const int*, const int*, const int*, const int*, int*, int*, int*, int*,
                           int*, int*, int, int, int64_t, int, void*, size_t, uint64_t);
static kda_status (*compact_)(const int*, const int*, int*, int*, int*, int*, int*, int, int,
                              int64_t, void*, size_t, uint64_t);
static kda_status (*copy_)(uint8_t* const*, int, int64_t, int, int, const int*, const int*,
                           const int*, int, uint64_t);

typedef struct {
    void* at;
    PyObject* dtype; /* borrowed: types live as long as torch */
    long device;
    int dims;
    int64_t shape[4], stride[4];
    int packed; /* contiguous */
} Tensor;

static int ints_of(PyObject* x, int64_t* out) { /* a tuple's, at most four; -1: others */
    if (!x || !PyTuple_Check(x) || PyTuple_GET_SIZE(x) > 4) return -1;
    const int n = (int)PyTuple_GET_SIZE(x);
    for (int i = 0; i < n; ++i) {
        out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(x, i));
        if (out[i] == -1 && PyErr_Occurred()) return -1;
    }
    return n;
}

static long long called(PyObject* o, PyObject* name) {
    PyObject* r = PyObject_CallMethodNoArgs(o, name);
    if (!r) return -1;
    const long long x = (long long)PyLong_AsUnsignedLongLongMask(r);
    Py_DECREF(r);
    return x;
}

/* Reads a tensor on device `dev` (below 0: any) that is not empty; 0: it is none. */
static int look(PyObject* o, Tensor* t, long dev) {
    if (o == Py_None) return 0;
    PyObject* x = PyObject_GetAttr(o, n_dtype);
    if (!x) return 0;
    t->dtype = x;
    Py_DECREF(x);
    t->device = (long)called(o, n_get_device);
    if (PyErr_Occurred() || t->device < 0 || (dev >= 0 && t->device != dev)) return 0;
    x = PyObject_GetAttr(o, n_shape);
    t->dims = ints_of(x, t->shape);
    Py_XDECREF(x);
    if (t->dims < 1) return 0;
    x = PyObject_CallMethodNoArgs(o, n_stride);
    const int strides = ints_of(x, t->stride);
    Py_XDECREF(x);
    if (strides != t->dims) return 0;
    int64_t size = 1;
    t->packed = 1;
    for (int i = t->dims - 1; i >= 0; --i) {
        if (t->shape[i] < 1) return 0;
        if (t->shape[i] > 1 && t->stride[i] != size) t->packed = 0;
        size *= t->shape[i];
    }
    t->at = (void*)(uintptr_t)called(o, n_data_ptr);
    return !PyErr_Occurred();
}

static int same(const Tensor* a, const Tensor* b, int dims) {
    for (int i = 0; i < dims; ++i)
        if (a->shape[i] != b->shape[i]) return 0;
    return 1;
}

/* A contiguous array of a type, and of a shape. */
static int array(PyObject* o, Tensor* t, long dev, PyObject* dtype, int dims, int64_t a, int64_t b) {
    return look(o, t, dev) && t->dtype == dtype && t->packed && t->dims == dims &&
           t->shape[0] == a && (dims < 2 || t->shape[1] == b);
}

/* The token-row stride of [.., rows, heads, 128]; 0: not such rows. */
static int64_t row_stride(const Tensor* t) {
    const int n = t->dims;
    if ((n != 3 && n != 4) || t->shape[n - 1] != D) return 0;
    const int64_t heads = t->shape[n - 2];
    if (t->packed) return heads * D;
    if (t->stride[n - 1] != 1 || (t->stride[n - 2] != D && heads > 1)) return 0;
    int64_t row = t->shape[n - 3] > 1 ? t->stride[n - 3] : heads * D;
    if (n == 4 && t->shape[0] > 1) {
        if (t->shape[1] == 1) row = t->stride[0];
        else if (t->stride[0] != t->shape[1] * row) return 0;
    }
    return row;
}

/* The stream of the current device, if that is `dev`. */
static int stream_of(long dev, uint64_t* stream) {
    PyObject* x = PyObject_CallNoArgs(current_device);
    if (!x) return 0;
    const long now = PyLong_AsLong(x);
    if (now != dev) {
        Py_DECREF(x);
        return 0;
    }
    PyObject* s = PyObject_CallOneArg(raw_stream, x);
    Py_DECREF(x);
    if (!s) return 0;
    *stream = (uint64_t)PyLong_AsUnsignedLongLongMask(s);
    Py_DECREF(s);
    return !PyErr_Occurred();
}

static PyObject* no(void) { /* nothing called */
    PyErr_Clear();
    return PyLong_FromLong(-1);
}
/* A function ends with a call of the library, made without the interpreter's lock: a launch may
 * wait for room in its stream, which may wait for a host function in Python. */
#define RETURN_CALL(call)                                \
    do {                                                 \
        kda_status status;                               \
        Py_BEGIN_ALLOW_THREADS                           \
        status = (call);                                 \
        Py_END_ALLOW_THREADS                             \
        return PyLong_FromLong(status);                  \
    } while (0)

static int in_type(const Tensor* t) {
    return t->dtype == bf16 ? KDA_BF16 : t->dtype == f16 ? KDA_F16 : -1;
}

static int number(PyObject* o, double* x) {
    *x = PyFloat_AsDouble(o);
    return !(*x == -1.0 && PyErr_Occurred());
}

static int whole(PyObject* o, int64_t least, int64_t most, int64_t* x) {
    *x = PyLong_AsLongLong(o);
    return !(*x == -1 && PyErr_Occurred()) && *x >= least && *x <= most;
}

/* What both calls of linear attention take of their rows. */
typedef struct {
    Tensor q, k, v, g, o;
    int64_t qs, ks, vs, gs, os, heads, qk_heads;
    int type;
} Rows;
static int lin_rows(PyObject* const* a, Rows* r) {
    if (!look(a[0], &r->q, -1) || (r->type = in_type(&r->q)) < 0) return 0;
    const long dev = r->q.device;
    if (!look(a[1], &r->k, dev) || !look(a[2], &r->v, dev) || !look(a[3], &r->g, dev) ||
        !look(a[4], &r->o, dev))
        return 0;
    const int n = r->q.dims;
    if (r->k.dtype != r->q.dtype || r->v.dtype != r->q.dtype || r->o.dtype != r->q.dtype ||
        r->g.dtype != f32 || r->k.dims != n || r->v.dims != n || r->o.dims != n)
        return 0;
    r->qs = row_stride(&r->q), r->ks = row_stride(&r->k);
    r->vs = row_stride(&r->v), r->os = row_stride(&r->o);
    if (r->qs < 1 || r->ks < 1 || r->vs < 1 || r->os < 1) return 0;
    if (!same(&r->q, &r->k, n) || !same(&r->v, &r->o, n) || !same(&r->q, &r->v, n - 2)) return 0;
    r->heads = r->v.shape[n - 2], r->qk_heads = r->q.shape[n - 2];
    if (!r->g.packed) return 0;
    if (r->g.dims == 1 && r->g.shape[0] == r->heads) r->gs = 0;
    else if (r->g.dims == n - 1 && same(&r->g, &r->q, n - 2) && r->g.shape[n - 2] == r->heads)
        r->gs = r->heads;
    else return 0;
    return r->heads <= INT32_MAX && r->q.shape[0] <= INT32_MAX && r->q.shape[1] <= INT32_MAX;
}
/* FP32 [n][heads][128][128], or None; 0: neither. */
static int state_of(PyObject* o, long dev, int64_t n, int64_t heads, void** at) {
    Tensor t;
    *at = NULL;
    if (o == Py_None) return 1;
    if (!look(o, &t, dev) || t.dtype != f32 || !t.packed || t.dims != 4 || t.shape[0] != n ||
        t.shape[1] != heads || t.shape[2] != D || t.shape[3] != D)
        return 0;
    *at = t.at;
    return 1;
}
/* A workspace's bytes; 0: none. */
static size_t space(PyObject* o, long dev, Tensor* t) {
    return look(o, t, dev) && t->packed && t->dims == 1 && t->dtype == u8 ? (size_t)t->shape[0] : 0;
}

/* q, k, v, g, out, state_in, state_out, t, cu_seqlens, scale, workspace */
static PyObject* lin_prefill(PyObject* self, PyObject* const* a, Py_ssize_t count) {
    Rows r;
    Tensor ws, cu;
    void *in, *out;
    double scale;
    uint64_t stream;
    if (count != 11 || !lin_rows(a, &r)) return no();
    const long dev = r.q.device;
    int64_t n = r.q.dims == 3 ? 1 : r.q.shape[0], t_pad = r.q.shape[r.q.dims - 3], t = t_pad;
    cu.at = NULL;
    if (a[8] != Py_None) {
        if (r.q.dims != 3 || a[7] != Py_None || !look(a[8], &cu, dev) || cu.dims != 1 ||
            !cu.packed || cu.dtype != i32 || cu.shape[0] > INT32_MAX)
            return no();
        n = cu.shape[0] - 1;
    } else if (a[7] != Py_None && !whole(a[7], 0, t_pad, &t)) {
        return no();
    }
    const size_t bytes = space(a[10], dev, &ws);
    if (!bytes || !state_of(a[5], dev, n, r.heads, &in) || !state_of(a[6], dev, n, r.heads, &out) ||
        !number(a[9], &scale) || !stream_of(dev, &stream))
        return no();
    RETURN_CALL(lin_prefill_(in, out, r.q.at, r.k.at, r.v.at, r.g.at, r.o.at, (int)t, (int)t_pad,
                             cu.at, (int)n, (int)r.heads, (int)r.qk_heads, D, r.type, r.qs, r.ks,
                             r.vs, r.gs, r.os, (float)scale, ws.at, bytes, stream));
}

/* q, k, v, g, out, state_in, state_out, snapshots, scale */
static PyObject* lin_decode(PyObject* self, PyObject* const* a, Py_ssize_t count) {
    Rows r;
    void *in, *out, *snaps[KDA_MAX_K];
    double scale;
    uint64_t stream;
    if (count != 9 || !lin_rows(a, &r)) return no();
    const long dev = r.q.device;
    const int64_t n = r.q.shape[0], krows = r.q.dims == 4 ? r.q.shape[1] : 1;
    const int list = PyList_Check(a[7]);
    if (!list && !PyTuple_Check(a[7])) return no();
    const Py_ssize_t n_snap = list ? PyList_GET_SIZE(a[7]) : PyTuple_GET_SIZE(a[7]);
    if (n_snap > KDA_MAX_K) return no();
    for (Py_ssize_t i = 0; i < n_snap; ++i) {
        PyObject* s = list ? PyList_GET_ITEM(a[7], i) : PyTuple_GET_ITEM(a[7], i);
        if (!state_of(s, dev, n, r.heads, snaps + i) || !snaps[i]) return no();
    }
    if (!state_of(a[5], dev, n, r.heads, &in) || !state_of(a[6], dev, n, r.heads, &out) ||
        !number(a[8], &scale) || !stream_of(dev, &stream))
        return no();
    RETURN_CALL(lin_decode_(in, out, r.q.at, r.k.at, r.v.at, r.g.at, r.o.at, (int)n, (int)krows,
                            (int)r.heads, (int)r.qk_heads, D, r.type, r.qs, r.ks, r.vs, r.gs, r.os,
                            (float)scale, n_snap ? (float* const*)snaps : NULL, (int)n_snap,
                            stream));
}

/* q, k, positions, inv_freq, q_out, k_out, pair_axis, interleaved, factor */
static PyObject* rope(PyObject* self, PyObject* const* a, Py_ssize_t count) {
    Tensor q, k, qo, ko, pos, freq;
    uint8_t axis[64];
    double factor;
    uint64_t stream;
    if (count != 9 || !look(a[0], &q, -1)) return no();
    const long dev = q.device;
    const int type = in_type(&q), n = q.dims, has_k = a[1] != Py_None;
    if (type < 0 || (!has_k && a[5] != Py_None)) return no();
    qo = q;
    if (a[4] != Py_None && (!look(a[4], &qo, dev) || qo.dtype != q.dtype || qo.dims != n ||
                            !same(&q, &qo, n)))
        return no();
    if (has_k) {
        if (!look(a[1], &k, dev) || k.dtype != q.dtype || k.dims != n || !same(&q, &k, n - 2))
            return no();
        ko = k;
        if (a[5] != Py_None && (!look(a[5], &ko, dev) || ko.dtype != q.dtype || ko.dims != n ||
                                !same(&k, &ko, n)))
            return no();
    }
    const int64_t qs = row_stride(&q), qos = row_stride(&qo), ks = has_k ? row_stride(&k) : 0,
                  kos = has_k ? row_stride(&ko) : 0;
    if (qs < 1 || qos < 1 || (has_k && (ks < 1 || kos < 1))) return no();
    if (!look(a[2], &pos, dev) || pos.dtype != i32 || !pos.packed || pos.dims < n - 2 ||
        pos.dims > n - 1 || !same(&pos, &q, n - 2) || !look(a[3], &freq, dev) ||
        freq.dtype != f32 || !freq.packed || freq.dims != 1 || freq.shape[0] > 64)
        return no();
    const int64_t axes = pos.dims == n - 1 ? pos.shape[n - 2] : 1, pairs = freq.shape[0];
    const uint8_t* table = NULL;
    if (a[6] != Py_None) {
        PyObject* seq = PySequence_Fast(a[6], "");
        if (!seq) return no();
        int ok = PySequence_Fast_GET_SIZE(seq) == pairs;
        for (int64_t i = 0; ok && i < pairs; ++i) {
            int64_t x;
            ok = whole(PySequence_Fast_GET_ITEM(seq, i), 0, axes - 1 < 255 ? axes - 1 : 255, &x);
            axis[i] = (uint8_t)x;
        }
        Py_DECREF(seq);
        if (!ok) return no();
        table = axis;
    } else if (axes > 1) {
        return no();
    }
    const int turn = PyObject_IsTrue(a[7]);
    if (turn < 0 || !number(a[8], &factor) || axes > 4 || q.shape[n - 2] > 1 << 16 ||
        (has_k && k.shape[n - 2] > 1 << 16) || !stream_of(dev, &stream))
        return no();
    const int64_t rows = n == 3 ? q.shape[0] : q.shape[0] * q.shape[1];
    RETURN_CALL(rope_(q.at, has_k ? k.at : NULL, qo.at, has_k ? ko.at : NULL, rows,
                      (int)q.shape[n - 2], has_k ? (int)k.shape[n - 2] : 0, D, type, qs, ks, qos, kos,
                      pos.at, (int)axes, freq.at, (int)pairs, table, turn, (float)factor, stream));
}

/* A page table, the pages' counts and a workspace. */
typedef struct {
    Tensor table, refs, ws;
    int64_t rows, width, pages;
    size_t bytes;
} Pages;
static int pages_of(PyObject* table, PyObject* refs, PyObject* ws, Pages* p) {
    if (!look(table, &p->table, -1)) return 0;
    const long dev = p->table.device;
    if (p->table.dtype != i32 || !p->table.packed || p->table.dims != 2 ||
        !look(refs, &p->refs, dev) || p->refs.dtype != i32 || !p->refs.packed || p->refs.dims != 1)
        return 0;
    p->rows = p->table.shape[0], p->width = p->table.shape[1], p->pages = p->refs.shape[0];
    p->bytes = space(ws, dev, &p->ws);
    return p->bytes > 0 && p->rows <= INT32_MAX && p->width <= INT32_MAX;
}

/* page_table, lens, refs, page, workspace */
static PyObject* resize(PyObject* self, PyObject* const* a, Py_ssize_t count) {
    Pages p;
    Tensor lens;
    int64_t page;
    uint64_t stream;
    if (count != 5 || !pages_of(a[0], a[2], a[4], &p) ||
        !array(a[1], &lens, p.table.device, i32, 1, p.rows, 0) || !whole(a[3], 1, 1 << 20, &page) ||
        !stream_of(p.table.device, &stream))
        return no();
    RETURN_CALL(resize_(p.table.at, lens.at, p.refs.at, (int)p.rows, (int)p.width, p.pages,
                        (int)page, p.ws.at, p.bytes, stream));
}

/* page_table, lens, refs, parent, page_table_out, lens_out, refs_out, src, dst, count, page,
 * workspace */
static PyObject* fork_pages(PyObject* self, PyObject* const* a, Py_ssize_t count) {
    Pages p;
    Tensor lens, parent, table_out, lens_out, refs_out, src, dst, n;
    int64_t page;
    uint64_t stream;
    if (count != 12 || !pages_of(a[0], a[2], a[11], &p)) return no();
    const long dev = p.table.device;
    if (!array(a[1], &lens, dev, i32, 1, p.rows, 0) ||
        !array(a[3], &parent, dev, i32, 1, p.rows, 0) ||
        !array(a[7], &src, dev, i32, 1, p.rows, 0) || !array(a[8], &dst, dev, i32, 1, p.rows, 0) ||
        !array(a[9], &n, dev, i32, 1, 1, 0) || !whole(a[10], 1, 1 << 20, &page))
        return no();
    table_out = p.table, lens_out = lens, refs_out = p.refs;
    if ((a[4] != Py_None && !array(a[4], &table_out, dev, i32, 2, p.rows, p.width)) ||
        (a[5] != Py_None && !array(a[5], &lens_out, dev, i32, 1, p.rows, 0)) ||
        (a[6] != Py_None && !array(a[6], &refs_out, dev, i32, 1, p.pages, 0)) ||
        !stream_of(dev, &stream))
        return no();
    RETURN_CALL(fork_(p.table.at, lens.at, p.refs.at, parent.at, table_out.at, lens_out.at,
                      refs_out.at, src.at, dst.at, n.at, (int)p.rows, (int)p.width, p.pages,
                      (int)page, p.ws.at, p.bytes, stream));
}

/* page_table, refs, page_table_out, refs_out, src, dst, count, workspace */
static PyObject* compact(PyObject* self, PyObject* const* a, Py_ssize_t count) {
    Pages p;
    Tensor table_out, refs_out, src, dst, n;
    uint64_t stream;
    if (count != 8 || !pages_of(a[0], a[1], a[7], &p)) return no();
    const long dev = p.table.device;
    if (!array(a[4], &src, dev, i32, 1, p.pages / 2, 0) ||
        !array(a[5], &dst, dev, i32, 1, p.pages / 2, 0) || !array(a[6], &n, dev, i32, 1, 1, 0))
        return no();
    table_out = p.table, refs_out = p.refs;
    if ((a[2] != Py_None && !array(a[2], &table_out, dev, i32, 2, p.rows, p.width)) ||
        (a[3] != Py_None && !array(a[3], &refs_out, dev, i32, 1, p.pages, 0)) ||
        !stream_of(dev, &stream))
        return no();
    RETURN_CALL(compact_(p.table.at, p.refs.at, table_out.at, refs_out.at, src.at, dst.at, n.at,
                         (int)p.rows, (int)p.width, p.pages, p.ws.at, p.bytes, stream));
}

/* caches (a list), src, dst, count */
static PyObject* copy(PyObject* self, PyObject* const* a, Py_ssize_t count) {
    Tensor first, t, src, dst, n;
    uint8_t* at[KDA_KV4_MAX_CACHES];
    uint64_t stream;
    if (count != 4 || !PyList_Check(a[0])) return no();
    const Py_ssize_t caches = PyList_GET_SIZE(a[0]);
    if (caches < 1 || caches > KDA_KV4_MAX_CACHES || !look(PyList_GET_ITEM(a[0], 0), &first, -1))
        return no();
    const long dev = first.device;
    for (Py_ssize_t i = 0; i < caches; ++i) {
        if (!look(PyList_GET_ITEM(a[0], i), &t, dev) || t.dtype != u8 || !t.packed || t.dims != 3 ||
            !same(&t, &first, 3))
            return no();
        at[i] = t.at;
    }
    if (first.shape[2] % KDA_KV4_TOKEN_BYTES || first.shape[2] / KDA_KV4_TOKEN_BYTES > 1 << 20 ||
        first.shape[1] > INT32_MAX || !look(a[1], &src, dev) || src.dims != 1 || !src.packed ||
        src.dtype != i32 || src.shape[0] > INT32_MAX ||
        !array(a[2], &dst, dev, i32, 1, src.shape[0], 0) || !array(a[3], &n, dev, i32, 1, 1, 0) ||
        !stream_of(dev, &stream))
        return no();
    RETURN_CALL(copy_(at, (int)caches, first.shape[0],
                      (int)(first.shape[2] / KDA_KV4_TOKEN_BYTES), (int)first.shape[1], src.at,
                      dst.at, n.at, (int)src.shape[0], stream));
}

/* setup(addresses of the seven functions, the types, raw_stream, current_device) */
static PyObject* setup(PyObject* self, PyObject* args) {
    unsigned long long f[7];
    PyObject *types[5], *rs, *cd;
    if (!PyArg_ParseTuple(args, "(KKKKKKK)(OOOOO)OO", f, f + 1, f + 2, f + 3, f + 4, f + 5, f + 6,
                          types, types + 1, types + 2, types + 3, types + 4, &rs, &cd))
        return NULL;
    lin_prefill_ = (void*)(uintptr_t)f[0];
    lin_decode_ = (void*)(uintptr_t)f[1];
    rope_ = (void*)(uintptr_t)f[2];
    resize_ = (void*)(uintptr_t)f[3];
    fork_ = (void*)(uintptr_t)f[4];
    compact_ = (void*)(uintptr_t)f[5];
    copy_ = (void*)(uintptr_t)f[6];
    PyObject** keep[] = {&bf16, &f16, &f32, &i32, &u8};
    for (int i = 0; i < 5; ++i) Py_XSETREF(*keep[i], Py_NewRef(types[i]));
    Py_XSETREF(raw_stream, Py_NewRef(rs));
    Py_XSETREF(current_device, Py_NewRef(cd));
    Py_RETURN_NONE;
}

#define FAST(name, fn) {name, (PyCFunction)(void (*)(void))fn, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, NULL},
    FAST("lin_prefill", lin_prefill), FAST("lin_decode", lin_decode), FAST("rope", rope),
    FAST("resize", resize), FAST("fork", fork_pages), FAST("compact", compact), FAST("copy", copy),
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "fast_calls", NULL, -1, methods};

PyMODINIT_FUNC PyInit_fast_calls(void) {
    PyObject** names[] = {&n_dtype, &n_shape, &n_get_device, &n_data_ptr, &n_stride};
    const char* text[] = {"dtype", "shape", "get_device", "data_ptr", "stride"};
    for (int i = 0; i < 5; ++i)
        if (!(*names[i] = PyUnicode_InternFromString(text[i]))) return NULL;
    return PyModule_Create(&module);
}
