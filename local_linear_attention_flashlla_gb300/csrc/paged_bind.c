/* Argument marshalling of the paged calls in C: what __init__.py does in Python, for calls whose tensors all lie as
 * the kernels take them.  A decode step's paged calls run for a few microseconds on the GPU, and reading their
 * tensors' attributes from Python took longer than that (10 us of a 17 us attention call; 3 us here).
 *
 * Each function returns 0 when the library call succeeded, and -1 or the library's status when anything is not as
 * expected; the caller then goes the general way in Python, which copies what has to be copied and raises what
 * has to be raised.  The C library's entry points are given as addresses, so this module links against nothing. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>
#include <string.h>

typedef int (*plan_fn)(const void*, const void*, int, int, void*, int, const void*, int, const void*, int, void*, void*,
                       void*, void*, void*, void*, void*);
typedef int (*append_fn)(int, const void*, const void*, const void*, void*, void*, int, int, int, int, int, long long,
                         long long, long long, void*);
typedef int (*attend_fn)(int, int, const void*, const void*, const void*, const void*, const void*, const void*,
                         const void*, void*, void*, int, int, int, int, int, int, int, int, int, long long, long long, long long,
                         float, int, void*, size_t, void*);

static plan_fn f_plan;
static append_fn f_append;
static attend_fn f_attend;
static PyObject *t_bf16, *t_fp32, *t_i32, *t_i64;                        /* torch dtypes (singletons) */
static PyObject *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_device;   /* attribute names */

typedef struct {
    PyObject* dtype;      /* borrowed: dtypes live as long as torch */
    long device, dim;
    long long shape[4], stride[4];
    uintptr_t ptr;
} Tensor;

static int numbers(PyObject* tuple, long long* out, long* count) {
    if (!tuple || !PyTuple_Check(tuple) || PyTuple_GET_SIZE(tuple) > 4) return 0;
    *count = (long)PyTuple_GET_SIZE(tuple);
    for (long i = 0; i < *count; ++i) {
        out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
        if (out[i] == -1 && PyErr_Occurred()) return 0;
    }
    return 1;
}

/* Reads a tensor; 0 if obj is none (no error is left set). */
static int read_tensor(PyObject* obj, Tensor* t) {
    long strides = 0;
    int ok = 0;
    PyObject *dtype = PyObject_GetAttr(obj, s_dtype), *shape = NULL, *stride = NULL, *dev = NULL, *ptr = NULL;
    if (dtype && (shape = PyObject_GetAttr(obj, s_shape)) && (stride = PyObject_CallMethodNoArgs(obj, s_stride)) &&
        (dev = PyObject_CallMethodNoArgs(obj, s_device)) && (ptr = PyObject_CallMethodNoArgs(obj, s_data_ptr))) {
        t->dtype = dtype;
        t->device = PyLong_AsLong(dev);
        t->ptr = (uintptr_t)PyLong_AsUnsignedLongLong(ptr);
        ok = numbers(shape, t->shape, &t->dim) && numbers(stride, t->stride, &strides) && strides == t->dim;
    }
    Py_XDECREF(dtype);
    Py_XDECREF(shape);
    Py_XDECREF(stride);
    Py_XDECREF(dev);
    Py_XDECREF(ptr);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        ok = 0;
    }
    return ok;
}

/* A contiguous vector of n (n < 0: any length) elements. */
static int vector(PyObject* obj, PyObject* dtype, long device, long long n, Tensor* t) {
    return read_tensor(obj, t) && t->dtype == dtype && t->device == device && t->dim == 1 &&
           (n < 0 || t->shape[0] == n) && (t->stride[0] == 1 || t->shape[0] <= 1);
}
/* A contiguous [rows, any] matrix. */
static int matrix(PyObject* obj, PyObject* dtype, long device, long long rows, Tensor* t) {
    return read_tensor(obj, t) && t->dtype == dtype && t->device == device && t->dim == 2 && t->shape[0] == rows &&
           (t->stride[1] == 1 || t->shape[1] == 1) && (t->stride[0] == t->shape[1] || rows == 1);
}
/* Two caches laid out alike; *page_stride their pages' distance. */
static int caches(PyObject* ko, PyObject* vo, Tensor* k, Tensor* v, long long* page_stride) {
    if (!read_tensor(ko, k) || !read_tensor(vo, v) || k->dim != 4 || v->dim != 4 || k->dtype != v->dtype ||
        k->device != v->device || k->device < 0 || (k->dtype != t_bf16 && k->dtype != t_fp32))
        return 0;
    for (int i = 0; i < 4; ++i)
        if (k->shape[i] != v->shape[i] || k->stride[i] != v->stride[i]) return 0;
    if (k->stride[3] != 1 || k->stride[2] != k->shape[3] || k->stride[1] != k->shape[2] * k->shape[3]) return 0;
    *page_stride = k->shape[0] > 1 ? k->stride[0] : k->shape[1] * k->stride[1];
    return 1;
}
/* [T, heads, d] token rows of the caches' type, heads packed, 16-byte token stride; *stride their distance. */
static int rows(PyObject* obj, const Tensor* cache, long long heads, Tensor* t, long long* stride) {
    const long long d = cache->shape[3], most = heads * d;
    if (t->dtype != cache->dtype || t->device != cache->device || t->dim != 3 || t->shape[1] != heads || t->shape[2] != d ||
        t->stride[2] != 1 || (t->stride[1] != d && heads != 1) || t->ptr % 16)
        return 0;
    *stride = t->shape[0] > 1 ? t->stride[0] : most;
    (void)obj;
    return *stride >= most && *stride * (cache->dtype == t_bf16 ? 2 : 4) % 16 == 0;
}

static int fits(long long x) { return x >= 0 && x <= 0x7fffffff; }

static uintptr_t pointer_of(PyObject* obj) {
    PyObject* p = PyObject_CallMethodNoArgs(obj, s_data_ptr);
    uintptr_t x = p ? (uintptr_t)PyLong_AsUnsignedLongLong(p) : 0;
    Py_XDECREF(p);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        x = 0;
    }
    return x;
}

#define P(x) ((void*)(x))

/* plan(device, ctx, new, table, free, count, page, T, kv, cu, slots, positions, granted, left, stream): the six
 * outputs are the caller's own, freshly allocated. */
static PyObject* plan(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Tensor ctx, fresh, table, pages, count;
    int status = -1;
    (void)self;
    if (n != 15) return PyLong_FromLong(-1);
    const long device = PyLong_AsLong(a[0]);
    const long long page = PyLong_AsLongLong(a[6]), T = PyLong_AsLongLong(a[7]);
    const uintptr_t stream = (uintptr_t)PyLong_AsUnsignedLongLong(a[14]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return PyLong_FromLong(-1);
    }
    if (vector(a[1], t_i32, device, -1, &ctx) && vector(a[2], t_i32, device, ctx.shape[0], &fresh) &&
        matrix(a[3], t_i32, device, ctx.shape[0], &table) && vector(a[4], t_i32, device, -1, &pages) &&
        vector(a[5], t_i32, device, 1, &count) && fits(ctx.shape[0]) && fits(table.shape[1]) && fits(pages.shape[0]) &&
        fits(page) && fits(T)) {
        uintptr_t out[6];
        for (int i = 0; i < 6; ++i) out[i] = pointer_of(a[8 + i]);
        Py_BEGIN_ALLOW_THREADS
        status = f_plan(P(ctx.ptr), P(fresh.ptr), (int)ctx.shape[0], (int)page, P(table.ptr), (int)table.shape[1],
                        P(pages.ptr), (int)pages.shape[0], P(count.ptr), (int)T, P(out[0]), P(out[1]), P(out[2]), P(out[3]),
                        P(out[4]), P(out[5]), P(stream));
        Py_END_ALLOW_THREADS
    }
    return PyLong_FromLong(status);
}

/* append(device, k_new, v_new, slots, k_cache, v_cache, stream) */
static PyObject* append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Tensor k, v, slots, kc, vc;
    long long ks, vs, ps;
    int status = -1;
    (void)self;
    if (n != 7) return PyLong_FromLong(-1);
    const long device = PyLong_AsLong(a[0]);
    const uintptr_t stream = (uintptr_t)PyLong_AsUnsignedLongLong(a[6]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return PyLong_FromLong(-1);
    }
    if (caches(a[4], a[5], &kc, &vc, &ps) && kc.device == device && read_tensor(a[1], &k) && read_tensor(a[2], &v) &&
        rows(a[1], &kc, kc.shape[1], &k, &ks) && rows(a[2], &kc, kc.shape[1], &v, &vs) && k.shape[0] == v.shape[0] &&
        vector(a[3], t_i64, device, k.shape[0], &slots) && fits(k.shape[0]) && fits(kc.shape[0]) && fits(kc.shape[1]) &&
        fits(kc.shape[2])) {
        Py_BEGIN_ALLOW_THREADS
        status = f_append(kc.dtype == t_bf16 ? 0 : 1, P(k.ptr), P(v.ptr), P(slots.ptr), P(kc.ptr), P(vc.ptr), (int)k.shape[0],
                          (int)kc.shape[1], (int)kc.shape[3], (int)kc.shape[2], (int)kc.shape[0], ks, vs, ps, P(stream));
        Py_END_ALLOW_THREADS
    }
    return PyLong_FromLong(status);
}

/* parallax(device, q, probe, k_cache, v_cache, table, cu_q, kv_lens, out, tau, max_new, causal, path, workspace,
 * workspace bytes, stream[, lse or None]) */
static PyObject* parallax(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Tensor q, r, kc, vc, table, cu, kv, out, lse;
    long long qs, rs, os, ps;
    int status = -1;
    (void)self;
    if (n != 16 && n != 17) return PyLong_FromLong(-1);
    const long device = PyLong_AsLong(a[0]);
    const double tau = PyFloat_AsDouble(a[9]);
    const long long max_new = PyLong_AsLongLong(a[10]);
    const int causal = PyObject_IsTrue(a[11]);
    const long path = PyLong_AsLong(a[12]);
    const uintptr_t ws = (uintptr_t)PyLong_AsUnsignedLongLong(a[13]), stream = (uintptr_t)PyLong_AsUnsignedLongLong(a[15]);
    const size_t ws_bytes = PyLong_AsSize_t(a[14]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return PyLong_FromLong(-1);
    }
    if (!caches(a[3], a[4], &kc, &vc, &ps) || kc.device != device || !read_tensor(a[1], &q) || q.dim != 3 ||
        !rows(a[1], &kc, q.shape[1], &q, &qs) || !read_tensor(a[2], &r) || !rows(a[2], &kc, q.shape[1], &r, &rs) ||
        r.shape[0] != q.shape[0] || !read_tensor(a[8], &out) || !rows(a[8], &kc, q.shape[1], &out, &os) ||
        out.shape[0] != q.shape[0] || os != q.shape[1] * q.shape[2] || !read_tensor(a[7], &kv) || kv.dim != 1)
        return PyLong_FromLong(-1);
    const long long S = kv.shape[0];
    lse.ptr = 0;
    if (n == 17 && a[16] != Py_None &&
        (!read_tensor(a[16], &lse) || lse.dtype != t_fp32 || lse.device != device || lse.dim != 2 || lse.shape[0] != q.shape[0] ||
         lse.shape[1] != q.shape[1] || lse.stride[1] != 1 || lse.stride[0] != q.shape[1]))
        return PyLong_FromLong(-1);
    if (vector(a[7], t_i32, device, S, &kv) && vector(a[6], t_i32, device, S + 1, &cu) && matrix(a[5], t_i32, device, S, &table) &&
        fits(q.shape[0]) && fits(q.shape[1]) && fits(S) && fits(table.shape[1]) && fits(kc.shape[0]) && fits(kc.shape[1]) &&
        fits(kc.shape[2]) && fits(max_new)) {
        Py_BEGIN_ALLOW_THREADS
        status = f_attend(kc.dtype == t_bf16 ? 0 : 1, (int)path, P(q.ptr), P(r.ptr), P(kc.ptr), P(vc.ptr), P(table.ptr),
                          P(cu.ptr), P(kv.ptr), P(out.ptr), P(lse.ptr), (int)q.shape[0], (int)S, (int)q.shape[1], (int)kc.shape[1],
                          (int)kc.shape[3], (int)kc.shape[2], (int)kc.shape[0], (int)table.shape[1], (int)max_new, qs, rs, ps,
                          (float)tau, causal, P(ws), ws_bytes, P(stream));
        Py_END_ALLOW_THREADS
    }
    return PyLong_FromLong(status);
}

/* init(plan, append, attend addresses, bfloat16, float32, int32, int64) */
static PyObject* init(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (n != 7) {
        PyErr_SetString(PyExc_TypeError, "init takes three addresses and four dtypes");
        return NULL;
    }
    f_plan = (plan_fn)(uintptr_t)PyLong_AsUnsignedLongLong(a[0]);
    f_append = (append_fn)(uintptr_t)PyLong_AsUnsignedLongLong(a[1]);
    f_attend = (attend_fn)(uintptr_t)PyLong_AsUnsignedLongLong(a[2]);
    if (PyErr_Occurred()) return NULL;
    t_bf16 = Py_NewRef(a[3]);
    t_fp32 = Py_NewRef(a[4]);
    t_i32 = Py_NewRef(a[5]);
    t_i64 = Py_NewRef(a[6]);
    Py_RETURN_NONE;
}

/* ------------------------------------------------- rotary positions and bounded caches (include/lla.h)
 * The entry points' arguments are written out once more here, as above. */
typedef struct {
    const void* x;
    const void* dy;
    void* out;
    const void* gain;
    void* dgain;
    long long x_stride[3], dy_stride[3], out_stride[3];
    int heads;
} rotary_rows;
enum { kRotaryMost = 4 };
typedef int (*rotary_fn)(int, const rotary_rows*, int, int, int, int, const void*, long long, const void*, int, int, float, float,
                         const void*, const void*, int, void*);
typedef int (*rotary_backward_fn)(int, int, const rotary_rows*, int, int, int, int, const void*, long long, const void*, int, int,
                                  float, float, const void*, const void*, int, void*, size_t, void*);
typedef int (*weigh_fn)(int, const void*, const void*, const void*, const void*, void*, void*, const void*, const void*, const void*,
                        const void*, const void*, int, int, int, int, int, int, int, int, int, long long, long long, float, float, int,
                        int, void*, size_t, void*);
typedef int (*evict_fn)(int, const void*, void*, const void*, void*, void*, void*, const void*, const void*, const void*, const void*,
                        int, int, int, int, int, int, long long, int, int, void*);
typedef int (*trim_fn)(const void*, const void*, int, int, const void*, int, void*, int, const void*, const void*, void*, void*, void*,
                       void*);
static rotary_fn f_rotary;
static rotary_backward_fn f_rotary_backward;
static weigh_fn f_weigh;
static evict_fn f_evict;
static trim_fn f_trim;

/* Item i of a tuple or list of `count`, or the object itself where it stands for one; NULL where there is none. */
static PyObject* item(PyObject* obj, Py_ssize_t i, Py_ssize_t count) {
    if (PyTuple_Check(obj)) return PyTuple_GET_SIZE(obj) == count ? PyTuple_GET_ITEM(obj, i) : NULL;
    if (PyList_Check(obj)) return PyList_GET_SIZE(obj) == count ? PyList_GET_ITEM(obj, i) : NULL;
    return count == 1 ? obj : NULL;
}
/* A contiguous tensor of n elements in `dim` dimensions. */
static int packed(PyObject* obj, PyObject* dtype, long device, const long long* shape, long dim, Tensor* t) {
    long long step = 1;
    if (!read_tensor(obj, t) || t->dtype != dtype || t->device != device || t->dim != dim) return 0;
    for (long i = dim - 1; i >= 0; --i) {
        if (t->shape[i] != shape[i] || (t->stride[i] != step && t->shape[i] > 1)) return 0;
        step *= t->shape[i];
    }
    return 1;
}
/* [T, heads, d] or [B, heads, n, d] rows, 16-byte aligned and strided; their strides of batch, head and position. */
static int head_rows(const Tensor* t, PyObject* dtype, long device, const Tensor* like, long long* stride) {
    const int ve = dtype == t_bf16 ? 8 : 4;
    if (t->dtype != dtype || t->device != device || t->dim != like->dim || t->ptr % 16) return 0;
    for (long i = 0; i < t->dim; ++i)
        if (t->shape[i] != like->shape[i] || (i + 1 < t->dim ? t->stride[i] % ve != 0 : t->stride[i] != 1)) return 0;
    stride[0] = t->dim == 4 ? t->stride[0] : 0;
    stride[1] = t->stride[1];
    stride[2] = t->dim == 4 ? t->stride[2] : t->stride[0];
    return 1;
}

typedef struct {
    rotary_rows rows[kRotaryMost];
    int dtype, dy_dtype, count, B, n, d, S;
    long long position_stride;
    uintptr_t positions, turns, cu, shift;
} Rotary;

/* What both directions take: x (or None), dy (or None in the forward pass), positions, turns, rot, gains, eps given, cu_q, shift, and
 * out: contiguous tensors that the caller made like x. */
static int rotary_args(Rotary* r, long device, PyObject* x, PyObject* dy, PyObject* positions, PyObject* turns, long rot, PyObject* gains,
                       int normalise, PyObject* cu, PyObject* shift, PyObject* out) {
    Tensor first, t, p;
    PyObject* like = x != Py_None ? x : dy;
    const Py_ssize_t count = PyTuple_Check(like) ? PyTuple_GET_SIZE(like) : PyList_Check(like) ? PyList_GET_SIZE(like) : 1;
    if (count < 1 || count > kRotaryMost || !item(like, 0, count) || !read_tensor(item(like, 0, count), &first) || first.device != device ||
        first.device < 0 || (first.dim != 3 && first.dim != 4))
        return 0;
    PyObject* dtype = first.dtype;
    PyObject* dy_dtype = dtype;
    if (dtype != t_bf16 && dtype != t_fp32) return 0;
    if (dy != Py_None) {
        if (x == Py_None) t = first;
        else if (!item(dy, 0, count) || !read_tensor(item(dy, 0, count), &t)) return 0;
        dy_dtype = t.dtype;
        if (dy_dtype != dtype && dy_dtype != t_fp32) return 0;
    }
    const int flat = first.dim == 3;
    const long long B = flat ? 1 : first.shape[0], n = flat ? first.shape[0] : first.shape[2], d = first.shape[first.dim - 1];
    if (!fits(B) || !fits(n) || !fits(d)) return 0;
    memset(r, 0, sizeof *r);
    for (Py_ssize_t i = 0; i < count; ++i) {
        rotary_rows* o = &r->rows[i];
        Tensor l = first;
        if (i > 0 && (!item(like, i, count) || !read_tensor(item(like, i, count), &l))) return 0;
        if (l.dim != first.dim || l.dtype != dtype || l.shape[l.dim - 1] != d ||
            (flat ? l.shape[0] != n : l.shape[0] != B || l.shape[2] != n) || !fits(l.shape[1]))
            return 0;
        o->heads = (int)l.shape[1];
        if (x != Py_None) {
            if (!head_rows(&l, dtype, device, &l, o->x_stride)) return 0;
            o->x = P(l.ptr);
        }
        if (dy != Py_None) {
            if (x == Py_None) t = l;
            else if (!item(dy, i, count) || !read_tensor(item(dy, i, count), &t)) return 0;
            if (!head_rows(&t, dy_dtype, device, &l, o->dy_stride)) return 0;
            o->dy = P(t.ptr);
        }
        const uintptr_t to = item(out, i, count) ? pointer_of(item(out, i, count)) : 0;
        if (!to) return 0;
        o->out = P(to);
        o->out_stride[0] = flat ? 0 : l.shape[1] * n * d;
        o->out_stride[1] = flat ? d : n * d;
        o->out_stride[2] = flat ? l.shape[1] * d : d;
        if (gains != Py_None) {
            PyObject* g = item(gains, i, count);
            if (!g) return 0;
            if (g != Py_None) {
                if (!normalise || !vector(g, t_fp32, device, d, &t)) return 0;
                o->gain = P(t.ptr);
            }
        }
    }
    const long long both[2] = {B, n};
    if (vector(positions, t_i32, device, n, &p)) r->position_stride = 0;
    else if (!flat && packed(positions, t_i32, device, both, 2, &p)) r->position_stride = n;
    else return 0;
    r->positions = p.ptr;
    if (!vector(turns, t_i64, device, rot / 2, &t)) return 0;
    r->turns = t.ptr;
    if ((cu == Py_None) != (shift == Py_None)) return 0;
    if (cu != Py_None) {
        if (!flat || !vector(shift, t_i32, device, -1, &t) || !fits(t.shape[0])) return 0;
        r->shift = t.ptr;
        r->S = (int)t.shape[0];
        if (!vector(cu, t_i32, device, r->S + 1, &t)) return 0;
        r->cu = t.ptr;
    }
    r->dtype = dtype == t_bf16 ? 0 : 1;
    r->dy_dtype = dy_dtype == t_bf16 ? 0 : 1;
    r->count = (int)count;
    r->B = (int)B;
    r->n = (int)n;
    r->d = (int)d;
    return 1;
}

/* rotary(device, x, positions, turns, rot, magnitude, gains, eps, interleaved, cu_q, shift, out, stream); eps None: no normalisation */
static PyObject* rotary(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Rotary r;
    int status = -1;
    (void)self;
    if (n != 13) return PyLong_FromLong(-1);
    const long device = PyLong_AsLong(a[0]), rot = PyLong_AsLong(a[4]);
    const double magnitude = PyFloat_AsDouble(a[5]), eps = a[7] == Py_None ? -1.0 : PyFloat_AsDouble(a[7]);
    const int interleaved = PyObject_IsTrue(a[8]);
    const uintptr_t stream = (uintptr_t)PyLong_AsUnsignedLongLong(a[12]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return PyLong_FromLong(-1);
    }
    if (rotary_args(&r, device, a[1], Py_None, a[2], a[3], rot, a[6], eps >= 0.0, a[9], a[10], a[11]) && (a[7] == Py_None || eps >= 0.0)) {
        Py_BEGIN_ALLOW_THREADS
        status = f_rotary(r.dtype, r.rows, r.count, r.B, r.n, r.d, P(r.positions), r.position_stride, P(r.turns), (int)rot, interleaved,
                          (float)magnitude, (float)eps, P(r.cu), P(r.shift), r.S, P(stream));
        Py_END_ALLOW_THREADS
    }
    return PyLong_FromLong(status);
}

/* rotary_backward(device, dy, x, positions, turns, rot, magnitude, gains, eps, interleaved, cu_q, shift, dx, dgains, workspace,
 * workspace bytes, stream) */
static PyObject* rotary_backward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Rotary r;
    int status = -1;
    (void)self;
    if (n != 17) return PyLong_FromLong(-1);
    const long device = PyLong_AsLong(a[0]), rot = PyLong_AsLong(a[5]);
    const double magnitude = PyFloat_AsDouble(a[6]), eps = a[8] == Py_None ? -1.0 : PyFloat_AsDouble(a[8]);
    const int interleaved = PyObject_IsTrue(a[9]);
    const uintptr_t ws = (uintptr_t)PyLong_AsUnsignedLongLong(a[14]), stream = (uintptr_t)PyLong_AsUnsignedLongLong(a[16]);
    const size_t ws_bytes = PyLong_AsSize_t(a[15]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return PyLong_FromLong(-1);
    }
    if (!rotary_args(&r, device, a[2], a[1], a[3], a[4], rot, a[7], eps >= 0.0, a[10], a[11], a[12]) || (a[8] != Py_None && eps < 0.0))
        return PyLong_FromLong(-1);
    for (int i = 0; i < r.count; ++i) {
        if (!r.rows[i].gain) continue;
        PyObject* g = item(a[13], i, r.count);               /* the caller's own, like the gain */
        const uintptr_t to = g ? pointer_of(g) : 0;
        if (!to) return PyLong_FromLong(-1);
        r.rows[i].dgain = P(to);
    }
    Py_BEGIN_ALLOW_THREADS
    status = f_rotary_backward(r.dtype, r.dy_dtype, r.rows, r.count, r.B, r.n, r.d, P(r.positions), r.position_stride, P(r.turns), (int)rot,
                               interleaved, (float)magnitude, (float)eps, P(r.cu), P(r.shift), r.S, P(ws), ws_bytes, P(stream));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
}

/* weigh(device, q, lse, k_cache, scores, out, positions or None, dropped or None, table, cu_q, kv_lens, tau, max_new, decay, last,
 * causal, workspace, workspace bytes, stream, granted or None) */
static PyObject* weigh(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Tensor q, lse, kc, vc, sc, so, pos, drop, table, cu, kv, ok;
    long long qs, ps;
    int status = -1;
    (void)self;
    if (n != 20) return PyLong_FromLong(-1);
    const long device = PyLong_AsLong(a[0]);
    const double tau = PyFloat_AsDouble(a[11]), decay = PyFloat_AsDouble(a[13]);
    const long long max_new = PyLong_AsLongLong(a[12]), last = PyLong_AsLongLong(a[14]);
    const int causal = PyObject_IsTrue(a[15]);
    const uintptr_t ws = (uintptr_t)PyLong_AsUnsignedLongLong(a[16]), stream = (uintptr_t)PyLong_AsUnsignedLongLong(a[18]);
    const size_t ws_bytes = PyLong_AsSize_t(a[17]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return PyLong_FromLong(-1);
    }
    if (!caches(a[3], a[3], &kc, &vc, &ps) || kc.device != device || !read_tensor(a[1], &q) || q.dim != 3 || !rows(a[1], &kc, q.shape[1], &q, &qs) ||
        !packed(a[2], t_fp32, device, q.shape, 2, &lse) || !packed(a[4], t_fp32, device, kc.shape, 3, &sc) ||
        !packed(a[5], t_fp32, device, kc.shape, 3, &so) || !vector(a[10], t_i32, device, -1, &kv))
        return PyLong_FromLong(-1);
    const long long S = kv.shape[0];
    pos.ptr = drop.ptr = ok.ptr = 0;
    if ((a[19] == Py_None || vector(a[19], t_i32, device, S, &ok)) && (a[6] == Py_None || packed(a[6], t_i32, device, kc.shape, 3, &pos)) && (a[7] == Py_None || vector(a[7], t_i32, device, S, &drop)) &&
        vector(a[9], t_i32, device, S + 1, &cu) && matrix(a[8], t_i32, device, S, &table) && fits(q.shape[0]) && fits(q.shape[1]) && fits(S) &&
        fits(table.shape[1]) && fits(kc.shape[0]) && fits(kc.shape[1]) && fits(kc.shape[2]) && fits(max_new) && fits(last)) {
        Py_BEGIN_ALLOW_THREADS
        status = f_weigh(kc.dtype == t_bf16 ? 0 : 1, P(q.ptr), P(lse.ptr), P(kc.ptr), P(sc.ptr), P(so.ptr), P(pos.ptr), P(drop.ptr), P(table.ptr),
                         P(cu.ptr), P(kv.ptr), P(ok.ptr), (int)q.shape[0], (int)S, (int)q.shape[1], (int)kc.shape[1], (int)kc.shape[3], (int)kc.shape[2],
                         (int)kc.shape[0], (int)table.shape[1], (int)max_new, qs, ps, (float)tau, (float)decay, (int)last, causal, P(ws),
                         ws_bytes, P(stream));
        Py_END_ALLOW_THREADS
    }
    return PyLong_FromLong(status);
}

/* evict(device, scores, scores_out, positions or None, positions_out or None, k_cache, v_cache, table, kv_lens, keep, dropped or None,
 * sinks, recent, stream) */
static PyObject* evict(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Tensor sc, so, pos, po, kc, vc, table, kv, keep, drop;
    long long ps;
    int status = -1;
    (void)self;
    if (n != 14) return PyLong_FromLong(-1);
    const long device = PyLong_AsLong(a[0]);
    const long long sinks = PyLong_AsLongLong(a[11]), recent = PyLong_AsLongLong(a[12]);
    const uintptr_t stream = (uintptr_t)PyLong_AsUnsignedLongLong(a[13]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return PyLong_FromLong(-1);
    }
    if (!caches(a[5], a[6], &kc, &vc, &ps) || kc.device != device || !vector(a[8], t_i32, device, -1, &kv)) return PyLong_FromLong(-1);
    const long long S = kv.shape[0];
    pos.ptr = po.ptr = drop.ptr = 0;
    if (packed(a[1], t_fp32, device, kc.shape, 3, &sc) && packed(a[2], t_fp32, device, kc.shape, 3, &so) &&
        (a[3] == Py_None || packed(a[3], t_i32, device, kc.shape, 3, &pos)) && (a[4] == Py_None || packed(a[4], t_i32, device, kc.shape, 3, &po)) &&
        matrix(a[7], t_i32, device, S, &table) && vector(a[9], t_i32, device, S, &keep) &&
        (a[10] == Py_None || vector(a[10], t_i32, device, S, &drop)) && fits(S) && fits(table.shape[1]) && fits(kc.shape[0]) &&
        fits(kc.shape[1]) && fits(kc.shape[2]) && fits(sinks) && fits(recent)) {
        Py_BEGIN_ALLOW_THREADS
        status = f_evict(kc.dtype == t_bf16 ? 0 : 1, P(sc.ptr), P(so.ptr), P(pos.ptr), P(po.ptr), P(kc.ptr), P(vc.ptr), P(table.ptr), P(kv.ptr),
                         P(keep.ptr), P(drop.ptr), (int)S, (int)kc.shape[1], (int)kc.shape[3], (int)kc.shape[2], (int)kc.shape[0],
                         (int)table.shape[1], ps, (int)sinks, (int)recent, P(stream));
        Py_END_ALLOW_THREADS
    }
    return PyLong_FromLong(status);
}

/* trim(device, kv_lens, keep, table, free, count, page, dropped or None, new_lens, new_dropped, left, stream) */
static PyObject* trim(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Tensor kv, keep, table, pages, count, drop, nl, nd, left;
    int status = -1;
    (void)self;
    if (n != 12) return PyLong_FromLong(-1);
    const long device = PyLong_AsLong(a[0]);
    const long long page = PyLong_AsLongLong(a[6]);
    const uintptr_t stream = (uintptr_t)PyLong_AsUnsignedLongLong(a[11]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return PyLong_FromLong(-1);
    }
    if (device < 0 || !vector(a[1], t_i32, device, -1, &kv)) return PyLong_FromLong(-1);
    const long long S = kv.shape[0];
    drop.ptr = 0;
    if (vector(a[2], t_i32, device, S, &keep) && matrix(a[3], t_i32, device, S, &table) && vector(a[4], t_i32, device, -1, &pages) &&
        vector(a[5], t_i32, device, 1, &count) && (a[7] == Py_None || vector(a[7], t_i32, device, S, &drop)) &&
        vector(a[8], t_i32, device, S, &nl) && vector(a[9], t_i32, device, S, &nd) && vector(a[10], t_i32, device, 1, &left) && fits(S) &&
        fits(table.shape[1]) && fits(pages.shape[0]) && fits(page)) {
        Py_BEGIN_ALLOW_THREADS
        status = f_trim(P(kv.ptr), P(keep.ptr), (int)S, (int)page, P(table.ptr), (int)table.shape[1], P(pages.ptr), (int)pages.shape[0],
                        P(count.ptr), P(drop.ptr), P(nl.ptr), P(nd.ptr), P(left.ptr), P(stream));
        Py_END_ALLOW_THREADS
    }
    return PyLong_FromLong(status);
}

/* init_bounded(rotary, rotary_backward, weigh, evict, trim addresses), after init */
static PyObject* init_bounded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "init_bounded takes five addresses");
        return NULL;
    }
    f_rotary = (rotary_fn)(uintptr_t)PyLong_AsUnsignedLongLong(a[0]);
    f_rotary_backward = (rotary_backward_fn)(uintptr_t)PyLong_AsUnsignedLongLong(a[1]);
    f_weigh = (weigh_fn)(uintptr_t)PyLong_AsUnsignedLongLong(a[2]);
    f_evict = (evict_fn)(uintptr_t)PyLong_AsUnsignedLongLong(a[3]);
    f_trim = (trim_fn)(uintptr_t)PyLong_AsUnsignedLongLong(a[4]);
    if (PyErr_Occurred()) return NULL;
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"rotary", (PyCFunction)(void (*)(void))rotary, METH_FASTCALL, NULL},
    {"rotary_backward", (PyCFunction)(void (*)(void))rotary_backward, METH_FASTCALL, NULL},
    {"weigh", (PyCFunction)(void (*)(void))weigh, METH_FASTCALL, NULL},
    {"evict", (PyCFunction)(void (*)(void))evict, METH_FASTCALL, NULL},
    {"trim", (PyCFunction)(void (*)(void))trim, METH_FASTCALL, NULL},
    {"init_bounded", (PyCFunction)(void (*)(void))init_bounded, METH_FASTCALL, NULL},
    {"init", (PyCFunction)(void (*)(void))init, METH_FASTCALL, NULL},
    {"plan", (PyCFunction)(void (*)(void))plan, METH_FASTCALL, NULL},
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, NULL},
    {"parallax", (PyCFunction)(void (*)(void))parallax, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL},
};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_bind", "Paged-call marshalling.", -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__paged_bind(void) {
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_device = PyUnicode_InternFromString("get_device");
    return PyModule_Create(&module);
}
