/* The feed-forward and attention operators' Python calls without ctypes: the same argument
 * marshalling as __init__.py's ctypes wrappers (integers, objects with
 * data_ptr(), None; streams as integers or objects with cuda_stream; names of
 * types and activations), at about 0.7 us a call instead of 3.3.  Nothing of
 * the library is linked in: bind() takes the entry points' addresses from the
 * library that load() has opened.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>
#include <string.h>

#include "tg_gemm.h"

static PyObject *s_data_ptr, *s_cuda_stream, *s_numel, *s_element_size;

static int64_t (*f_linear_ws)(int64_t, int64_t, int64_t, const void *, int64_t, const void *, int64_t,
                              tg_dtype);
static tg_status (*f_linear)(int64_t, int64_t, int64_t, const void *, int64_t, const void *, int64_t,
                             const float *, tg_activation, const void *, int64_t, void *, int64_t,
                             void *, int64_t, tg_dtype, void *, int64_t, void *);
static int64_t (*f_gated_ws)(int64_t, int64_t, int64_t, const void *, int64_t, const void *, int64_t,
                             const void *, int64_t, tg_dtype);
static tg_status (*f_gated)(int64_t, int64_t, int64_t, const void *, int64_t, const void *, int64_t,
                            const void *, int64_t, tg_activation, void *, int64_t, void *, int64_t,
                            void *, int64_t, tg_dtype, void *, int64_t, void *);
static tg_status (*f_norm)(int64_t, int64_t, const void *, int64_t, const float *, const float *, float,
                           void *, int64_t, float *, float *, tg_out_dtype, void *);
static int64_t (*f_norm_back_ws)(int64_t, int64_t);
static tg_status (*f_norm_back)(int64_t, int64_t, const void *, int64_t, const void *, int64_t,
                                const float *, const float *, const float *, void *, int64_t, float *,
                                float *, tg_out_dtype, void *, int64_t, void *);

static tg_status (*f_rotary)(int64_t, int64_t, int64_t, int64_t, const void *, int64_t, int64_t, void *,
                             int64_t, int64_t, int64_t, const int64_t *, const int64_t *,
                             const uint64_t *, tg_rotary_layout, float, tg_out_dtype, void *);
static tg_status (*f_rotary_back)(int64_t, int64_t, int64_t, int64_t, const void *, int64_t, int64_t,
                                  void *, int64_t, int64_t, const int64_t *, const uint64_t *,
                                  tg_rotary_layout, float, tg_out_dtype, void *);
static int64_t (*f_attn_ws)(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t,
                            tg_dtype);
static tg_status (*f_attn)(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, const void *, int64_t,
                           int64_t, const void *, int64_t, int64_t, const void *, int64_t, int64_t,
                           const int64_t *, const int64_t *, const int64_t *, const int64_t *, int64_t,
                           int64_t, int32_t, float, void *, int64_t, int64_t, float *, tg_dtype, void *,
                           int64_t, void *);
static int64_t (*f_attn_back_ws)(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t,
                                 tg_dtype);
static tg_status (*f_attn_back)(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, const void *,
                                int64_t, int64_t, const void *, int64_t, int64_t, const void *, int64_t,
                                int64_t, const void *, int64_t, int64_t, const void *, int64_t, int64_t,
                                const float *, const int64_t *, const int64_t *, const int64_t *,
                                const int64_t *, int64_t, int64_t, int32_t, float, void *, int64_t,
                                int64_t, void *, int64_t, int64_t, void *, int64_t, int64_t, tg_dtype,
                                void *, int64_t, void *);

static const struct {
    const char *name;
    void *slot;
} ENTRIES[] = {
    {"tg_linear_workspace_bytes", &f_linear_ws}, {"tg_linear", &f_linear},
    {"tg_gated_workspace_bytes", &f_gated_ws},   {"tg_gated", &f_gated},
    {"tg_layer_norm", &f_norm},                  {"tg_layer_norm_backward_workspace_bytes", &f_norm_back_ws},
    {"tg_layer_norm_backward", &f_norm_back},
    {"tg_rotary", &f_rotary},                    {"tg_rotary_backward", &f_rotary_back},
    {"tg_attention_workspace_bytes", &f_attn_ws}, {"tg_attention", &f_attn},
    {"tg_attention_backward_workspace_bytes", &f_attn_back_ws},
    {"tg_attention_backward", &f_attn_back},
};
#define N_ENTRIES (sizeof(ENTRIES) / sizeof(ENTRIES[0]))

/* Argument readers: `*ok` goes to 0, with a Python error set, on failure. */
static int64_t as_int(PyObject *o, int *ok) {
    int64_t v = 0;
    if (!*ok) return 0;
    if (PyLong_Check(o)) {
        v = PyLong_AsLongLong(o);
    } else {
        PyObject *i = PyNumber_Index(o);
        if (!i) {
            *ok = 0;
            return 0;
        }
        v = PyLong_AsLongLong(i);
        Py_DECREF(i);
    }
    if (v == -1 && PyErr_Occurred()) *ok = 0;
    return v;
}

static void *as_ptr(PyObject *o, int *ok) {
    void *p = NULL;
    if (!*ok || o == Py_None) return NULL;
    if (PyLong_Check(o)) {
        p = (void *)(uintptr_t)PyLong_AsUnsignedLongLong(o);
    } else {
        PyObject *v = PyObject_CallMethodNoArgs(o, s_data_ptr);
        if (!v) {
            if (PyErr_ExceptionMatches(PyExc_AttributeError)) {
                PyErr_Clear();
                PyErr_Format(PyExc_TypeError, "cannot pass %s as a pointer", Py_TYPE(o)->tp_name);
            }
            *ok = 0;
            return NULL;
        }
        p = (void *)(uintptr_t)PyLong_AsUnsignedLongLong(v);
        Py_DECREF(v);
    }
    if (PyErr_Occurred()) *ok = 0;
    return p;
}

static void *as_stream(PyObject *o, int *ok) {
    void *p = NULL;
    PyObject *v;
    if (!*ok || o == Py_None) return NULL;
    if (PyLong_Check(o)) {
        p = (void *)(uintptr_t)PyLong_AsUnsignedLongLong(o);
        if (PyErr_Occurred()) *ok = 0;
        return p;
    }
    v = PyObject_GetAttr(o, s_cuda_stream);
    if (!v) {
        if (PyErr_ExceptionMatches(PyExc_AttributeError)) {
            PyErr_Clear();
            PyErr_Format(PyExc_TypeError, "cannot pass %s as a stream", Py_TYPE(o)->tp_name);
        }
        *ok = 0;
        return NULL;
    }
    p = (void *)(uintptr_t)PyLong_AsUnsignedLongLong(v);
    Py_DECREF(v);
    if (PyErr_Occurred()) *ok = 0;
    return p;
}

/* A name from one of the package's tables (bind() brings them), or its code. */
static PyObject *t_dtypes, *t_acts, *t_outs;
static int as_code(PyObject *o, PyObject *names, int *ok) {
    if (!*ok) return 0;
    if (PyUnicode_Check(o)) {
        PyObject *v = PyDict_GetItemWithError(names, o);
        if (!v) {
            if (!PyErr_Occurred()) PyErr_SetObject(PyExc_KeyError, o);
            *ok = 0;
            return 0;
        }
        return (int)as_int(v, ok);
    }
    return (int)as_int(o, ok);
}
#define DTYPE(o) ((tg_dtype)as_code(o, t_dtypes, &ok))
#define ACT(o) ((tg_activation)as_code(o, t_acts, &ok))
#define OUT(o) ((tg_out_dtype)as_code(o, t_outs, &ok))
#define INT(o) as_int(o, &ok)
#define PTR(o) as_ptr(o, &ok)

/* A workspace: None, a tensor, or (pointer, bytes). */
static void *as_space(PyObject *o, int64_t *bytes, int *ok) {
    void *p;
    PyObject *n, *e;
    *bytes = 0;
    if (!*ok || o == Py_None) return NULL;
    if (PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 2) {
        p = as_ptr(PyTuple_GET_ITEM(o, 0), ok);
        *bytes = as_int(PyTuple_GET_ITEM(o, 1), ok);
        return p;
    }
    p = as_ptr(o, ok);
    if (!*ok) return NULL;
    n = PyObject_CallMethodNoArgs(o, s_numel);
    e = n ? PyObject_CallMethodNoArgs(o, s_element_size) : NULL;
    if (n && e) *bytes = as_int(n, ok) * as_int(e, ok);
    else *ok = 0;
    Py_XDECREF(n);
    Py_XDECREF(e);
    return p;
}

#define TAKE(count, what)                                                                        \
    int ok = 1;                                                                                  \
    if (n != (count)) {                                                                          \
        PyErr_Format(PyExc_TypeError, "%s: %zd arguments for %d", what, n, (count));             \
        return NULL;                                                                             \
    }

/* A launching call, without Python's lock while it runs. */
#define RUN(call)                            \
    {                                        \
        tg_status status;                    \
        if (!ok) return NULL;                \
        Py_BEGIN_ALLOW_THREADS               \
        status = call;                       \
        Py_END_ALLOW_THREADS                 \
        return PyLong_FromLong(status);      \
    }

static PyObject *py_linear_ws(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    TAKE(8, "tg_linear_workspace_bytes")
    const int64_t m = INT(a[0]), nn = INT(a[1]), k = INT(a[2]);
    const void *x = PTR(a[3]);
    const int64_t ldx = INT(a[4]);
    const void *w = PTR(a[5]);
    const int64_t ldw = INT(a[6]);
    const tg_dtype t = DTYPE(a[7]);
    return ok ? PyLong_FromLongLong(f_linear_ws(m, nn, k, x, ldx, w, ldw, t)) : NULL;
}

static PyObject *py_linear(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    TAKE(18, "tg_linear")
    int64_t bytes;
    const int64_t m = INT(a[0]), nn = INT(a[1]), k = INT(a[2]);
    const void *x = PTR(a[3]);
    const int64_t ldx = INT(a[4]);
    const void *w = PTR(a[5]);
    const int64_t ldw = INT(a[6]);
    const float *bias = PTR(a[7]);
    const tg_activation act = ACT(a[8]);
    const void *r = PTR(a[9]);
    const int64_t ldr = INT(a[10]);
    void *y = PTR(a[11]);
    const int64_t ldy = INT(a[12]);
    void *z = PTR(a[13]);
    const int64_t ldz = INT(a[14]);
    const tg_dtype t = DTYPE(a[15]);
    void *ws = as_space(a[16], &bytes, &ok);
    void *st = as_stream(a[17], &ok);
    RUN(f_linear(m, nn, k, x, ldx, w, ldw, bias, act, r, ldr, y, ldy, z, ldz, t, ws, bytes, st))
}

static PyObject *py_gated_ws(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    TAKE(10, "tg_gated_workspace_bytes")
    const int64_t m = INT(a[0]), nn = INT(a[1]), k = INT(a[2]);
    const void *x = PTR(a[3]);
    const int64_t ldx = INT(a[4]);
    const void *wg = PTR(a[5]);
    const int64_t ldwg = INT(a[6]);
    const void *wu = PTR(a[7]);
    const int64_t ldwu = INT(a[8]);
    const tg_dtype t = DTYPE(a[9]);
    return ok ? PyLong_FromLongLong(f_gated_ws(m, nn, k, x, ldx, wg, ldwg, wu, ldwu, t)) : NULL;
}

static PyObject *py_gated(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    TAKE(19, "tg_gated")
    int64_t bytes;
    const int64_t m = INT(a[0]), nn = INT(a[1]), k = INT(a[2]);
    const void *x = PTR(a[3]);
    const int64_t ldx = INT(a[4]);
    const void *wg = PTR(a[5]);
    const int64_t ldwg = INT(a[6]);
    const void *wu = PTR(a[7]);
    const int64_t ldwu = INT(a[8]);
    const tg_activation act = ACT(a[9]);
    void *h = PTR(a[10]);
    const int64_t ldh = INT(a[11]);
    void *g = PTR(a[12]);
    const int64_t ldg = INT(a[13]);
    void *u = PTR(a[14]);
    const int64_t ldu = INT(a[15]);
    const tg_dtype t = DTYPE(a[16]);
    void *ws = as_space(a[17], &bytes, &ok);
    void *st = as_stream(a[18], &ok);
    RUN(f_gated(m, nn, k, x, ldx, wg, ldwg, wu, ldwu, act, h, ldh, g, ldg, u, ldu, t, ws, bytes, st))
}

static PyObject *py_norm(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    TAKE(13, "tg_layer_norm")
    const int64_t m = INT(a[0]), nn = INT(a[1]);
    const void *x = PTR(a[2]);
    const int64_t ldx = INT(a[3]);
    const float *gamma = PTR(a[4]), *beta = PTR(a[5]);
    const double eps = ok ? PyFloat_AsDouble(a[6]) : 0.0;
    if (eps == -1.0 && PyErr_Occurred()) return NULL;
    void *y = PTR(a[7]);
    const int64_t ldy = INT(a[8]);
    float *mean = PTR(a[9]), *rstd = PTR(a[10]);
    const tg_out_dtype t = OUT(a[11]);
    void *st = as_stream(a[12], &ok);
    RUN(f_norm(m, nn, x, ldx, gamma, beta, (float)eps, y, ldy, mean, rstd, t, st))
}

static PyObject *py_norm_back_ws(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    TAKE(2, "tg_layer_norm_backward_workspace_bytes")
    const int64_t m = INT(a[0]), nn = INT(a[1]);
    return ok ? PyLong_FromLongLong(f_norm_back_ws(m, nn)) : NULL;
}

static PyObject *py_norm_back(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    TAKE(16, "tg_layer_norm_backward")
    int64_t bytes;
    const int64_t m = INT(a[0]), nn = INT(a[1]);
    const void *dy = PTR(a[2]);
    const int64_t lddy = INT(a[3]);
    const void *x = PTR(a[4]);
    const int64_t ldx = INT(a[5]);
    const float *gamma = PTR(a[6]), *mean = PTR(a[7]), *rstd = PTR(a[8]);
    void *dx = PTR(a[9]);
    const int64_t lddx = INT(a[10]);
    float *dgamma = PTR(a[11]), *dbeta = PTR(a[12]);
    const tg_out_dtype t = OUT(a[13]);
    void *ws = as_space(a[14], &bytes, &ok);
    void *st = as_stream(a[15], &ok);
    RUN(f_norm_back(m, nn, dy, lddy, x, ldx, gamma, mean, rstd, dx, lddx, dgamma, dbeta, t, ws, bytes, st))
}

static float as_float(PyObject *o, int *ok) {
    double v;
    if (!*ok) return 0.0f;
    v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) *ok = 0;
    return (float)v;
}
#define FLT(o) as_float(o, &ok)

static PyObject *py_rotary(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    TAKE(18, "tg_rotary")
    const int64_t tokens = INT(a[0]), heads = INT(a[1]), dim = INT(a[2]), rot = INT(a[3]);
    const void *x = PTR(a[4]);
    const int64_t ldx = INT(a[5]), hx = INT(a[6]);
    void *y = PTR(a[7]);
    const int64_t ldy = INT(a[8]), hy = INT(a[9]), rows = INT(a[10]);
    const int64_t *pos = PTR(a[11]), *to = PTR(a[12]);
    const uint64_t *steps = PTR(a[13]);
    const int layout = (int)INT(a[14]);
    const float amp = FLT(a[15]);
    const tg_out_dtype t = OUT(a[16]);
    void *st = as_stream(a[17], &ok);
    RUN(f_rotary(tokens, heads, dim, rot, x, ldx, hx, y, ldy, hy, rows, pos, to, steps,
                 (tg_rotary_layout)layout, amp, t, st))
}

static PyObject *py_rotary_back(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    TAKE(16, "tg_rotary_backward")
    const int64_t tokens = INT(a[0]), heads = INT(a[1]), dim = INT(a[2]), rot = INT(a[3]);
    const void *dy = PTR(a[4]);
    const int64_t lddy = INT(a[5]), hdy = INT(a[6]);
    void *dx = PTR(a[7]);
    const int64_t lddx = INT(a[8]), hdx = INT(a[9]);
    const int64_t *pos = PTR(a[10]);
    const uint64_t *steps = PTR(a[11]);
    const int layout = (int)INT(a[12]);
    const float amp = FLT(a[13]);
    const tg_out_dtype t = OUT(a[14]);
    void *st = as_stream(a[15], &ok);
    RUN(f_rotary_back(tokens, heads, dim, rot, dy, lddy, hdy, dx, lddx, hdx, pos, steps,
                      (tg_rotary_layout)layout, amp, t, st))
}

/* The sizes that the attention calls and queries begin with. */
#define SIZES                                                                                     \
    const int64_t seqs = INT(a[0]), q_rows = INT(a[1]), k_rows = INT(a[2]), heads = INT(a[3]),     \
                  kv = INT(a[4]), dim = INT(a[5]);

static PyObject *attn_ws(int64_t (*f)(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t,
                                      int64_t, tg_dtype),
                         const char *name, PyObject *const *a, Py_ssize_t n) {
    TAKE(9, name)
    SIZES
    const int64_t max_q = INT(a[6]), max_k = INT(a[7]);
    const tg_dtype t = DTYPE(a[8]);
    return ok ? PyLong_FromLongLong(f(seqs, q_rows, k_rows, heads, kv, dim, max_q, max_k, t)) : NULL;
}
static PyObject *py_attn_ws(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    return attn_ws(f_attn_ws, "tg_attention_workspace_bytes", a, n);
}
static PyObject *py_attn_back_ws(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    return attn_ws(f_attn_back_ws, "tg_attention_backward_workspace_bytes", a, n);
}

static PyObject *py_attn(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    TAKE(30, "tg_attention")
    int64_t bytes;
    SIZES
    const void *q = PTR(a[6]);
    const int64_t ldq = INT(a[7]), hq = INT(a[8]);
    const void *k = PTR(a[9]);
    const int64_t ldk = INT(a[10]), hk = INT(a[11]);
    const void *v = PTR(a[12]);
    const int64_t ldv = INT(a[13]), hv = INT(a[14]);
    const int64_t *qs = PTR(a[15]), *ql = PTR(a[16]), *ks = PTR(a[17]), *kl = PTR(a[18]);
    const int64_t max_q = INT(a[19]), max_k = INT(a[20]);
    const int32_t causal = (int32_t)INT(a[21]);
    const float scale = FLT(a[22]);
    void *o = PTR(a[23]);
    const int64_t ldo = INT(a[24]), ho = INT(a[25]);
    float *lse = PTR(a[26]);
    const tg_dtype t = DTYPE(a[27]);
    void *ws = as_space(a[28], &bytes, &ok);
    void *st = as_stream(a[29], &ok);
    RUN(f_attn(seqs, q_rows, k_rows, heads, kv, dim, q, ldq, hq, k, ldk, hk, v, ldv, hv, qs, ql, ks, kl,
               max_q, max_k, causal, scale, o, ldo, ho, lse, t, ws, bytes, st))
}

static PyObject *py_attn_back(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    TAKE(42, "tg_attention_backward")
    int64_t bytes;
    SIZES
    const void *in[5];
    void *out[3];
    int64_t ld[8], hd[8];
    for (int i = 0; i < 5; ++i) {
        in[i] = PTR(a[6 + 3 * i]);
        ld[i] = INT(a[7 + 3 * i]);
        hd[i] = INT(a[8 + 3 * i]);
    }
    const float *lse = PTR(a[21]);
    const int64_t *qs = PTR(a[22]), *ql = PTR(a[23]), *ks = PTR(a[24]), *kl = PTR(a[25]);
    const int64_t max_q = INT(a[26]), max_k = INT(a[27]);
    const int32_t causal = (int32_t)INT(a[28]);
    const float scale = FLT(a[29]);
    for (int i = 0; i < 3; ++i) {
        out[i] = PTR(a[30 + 3 * i]);
        ld[5 + i] = INT(a[31 + 3 * i]);
        hd[5 + i] = INT(a[32 + 3 * i]);
    }
    const tg_dtype t = DTYPE(a[39]);
    void *ws = as_space(a[40], &bytes, &ok);
    void *st = as_stream(a[41], &ok);
    RUN(f_attn_back(seqs, q_rows, k_rows, heads, kv, dim, in[0], ld[0], hd[0], in[1], ld[1], hd[1], in[2],
                    ld[2], hd[2], in[3], ld[3], hd[3], in[4], ld[4], hd[4], lse, qs, ql, ks, kl, max_q,
                    max_k, causal, scale, out[0], ld[5], hd[5], out[1], ld[6], hd[6], out[2], ld[7], hd[7],
                    t, ws, bytes, st))
}

/* bind({name: address}, dtypes, acts, outs): every entry point the calls above
 * use, and the {name: code} tables of their arguments. */
static PyObject *py_bind(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    PyObject *table;
    if (n != 4 || !PyDict_Check(a[0]) || !PyDict_Check(a[1]) || !PyDict_Check(a[2]) || !PyDict_Check(a[3])) {
        PyErr_SetString(PyExc_TypeError, "bind: four dictionaries");
        return NULL;
    }
    table = a[0];
    for (size_t i = 0; i < N_ENTRIES; ++i) {
        PyObject *v = PyDict_GetItemString(table, ENTRIES[i].name);
        void *p;
        if (!v) {
            PyErr_Format(PyExc_KeyError, "%s", ENTRIES[i].name);
            return NULL;
        }
        p = PyLong_AsVoidPtr(v);
        if (!p) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "NULL entry point");
            return NULL;
        }
        memcpy(ENTRIES[i].slot, &p, sizeof(p));
    }
    Py_INCREF(a[1]);
    Py_INCREF(a[2]);
    Py_INCREF(a[3]);
    Py_XSETREF(t_dtypes, a[1]);
    Py_XSETREF(t_acts, a[2]);
    Py_XSETREF(t_outs, a[3]);
    Py_RETURN_NONE;
}

#define FAST(name, f) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL}
static PyMethodDef METHODS[] = {
    FAST("bind", py_bind),
    FAST("tg_linear_workspace_bytes", py_linear_ws),
    FAST("tg_linear", py_linear),
    FAST("tg_gated_workspace_bytes", py_gated_ws),
    FAST("tg_gated", py_gated),
    FAST("tg_layer_norm", py_norm),
    FAST("tg_layer_norm_backward_workspace_bytes", py_norm_back_ws),
    FAST("tg_layer_norm_backward", py_norm_back),
    FAST("tg_rotary", py_rotary),
    FAST("tg_rotary_backward", py_rotary_back),
    FAST("tg_attention_workspace_bytes", py_attn_ws),
    FAST("tg_attention", py_attn),
    FAST("tg_attention_backward_workspace_bytes", py_attn_back_ws),
    FAST("tg_attention_backward", py_attn_back),
    {NULL, NULL, 0, NULL},
};
static struct PyModuleDef MODULE = {PyModuleDef_HEAD_INIT, "_tgcall", NULL, -1, METHODS,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__tgcall(void) {
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    s_numel = PyUnicode_InternFromString("numel");
    s_element_size = PyUnicode_InternFromString("element_size");
    if (!s_data_ptr || !s_cuda_stream || !s_numel || !s_element_size) return NULL;
    return PyModule_Create(&MODULE);
}
