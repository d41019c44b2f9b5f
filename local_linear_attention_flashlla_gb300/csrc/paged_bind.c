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

typedef int (*plan_fn)(const void*, const void*, int, int, void*, int, const void*, int, const void*, int, void*, void*,
                       void*, void*, void*, void*, void*);
typedef int (*append_fn)(int, const void*, const void*, const void*, void*, void*, int, int, int, int, int, long long,
                         long long, long long, void*);
typedef int (*attend_fn)(int, int, const void*, const void*, const void*, const void*, const void*, const void*,
                         const void*, void*, int, int, int, int, int, int, int, int, int, long long, long long, long long,
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
 * workspace bytes, stream) */
static PyObject* parallax(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Tensor q, r, kc, vc, table, cu, kv, out;
    long long qs, rs, os, ps;
    int status = -1;
    (void)self;
    if (n != 16) return PyLong_FromLong(-1);
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
    if (vector(a[7], t_i32, device, S, &kv) && vector(a[6], t_i32, device, S + 1, &cu) && matrix(a[5], t_i32, device, S, &table) &&
        fits(q.shape[0]) && fits(q.shape[1]) && fits(S) && fits(table.shape[1]) && fits(kc.shape[0]) && fits(kc.shape[1]) &&
        fits(kc.shape[2]) && fits(max_new)) {
        Py_BEGIN_ALLOW_THREADS
        status = f_attend(kc.dtype == t_bf16 ? 0 : 1, (int)path, P(q.ptr), P(r.ptr), P(kc.ptr), P(vc.ptr), P(table.ptr),
                          P(cu.ptr), P(kv.ptr), P(out.ptr), (int)q.shape[0], (int)S, (int)q.shape[1], (int)kc.shape[1],
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

static PyMethodDef methods[] = {
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
