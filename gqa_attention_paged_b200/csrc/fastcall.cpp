// fastcall.cpp -- the checks and the call of binding.py's hottest functions in one C function each.
//
// A decode step of a small batch runs for 5 to 10 us on the GPU; checking ten tensors in Python and
// marshalling twenty arguments through ctypes took another 9 to 12 on the host.  Here a call whose
// tensors are all as they should be (and its outputs and workspace given) goes straight to the
// library; anything else returns None, and binding.py takes its own path with its own errors.  No
// check is weaker than there.  Only the interpreter's C API is used: tensors are asked for their
// attributes, their layout in memory is not known here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <limits.h>
#include <stdint.h>

#include "gqa_paged.h"

namespace {

PyObject *g_tensor, *g_bf16, *g_u8, *g_e4m3, *g_f32, *g_i32, *g_i64;  // torch.Tensor and dtypes
PyObject *s_dtype, *s_shape, *s_stride, *s_get_device, *s_is_contiguous, *s_data_ptr;

decltype(&gqa_paged_decode) f_decode;
decltype(&gqa_paged_decode_partial) f_partial;
decltype(&gqa_paged_append_kv) f_append;
decltype(&gqa_paged_append_decode) f_append_decode;
decltype(&gqa_paged_write_kv) f_write;
decltype(&gqa_paged_read_kv) f_read;

struct Tensor {
    void *ptr = nullptr;
    int nd = 0;
    long long size[4] = {0, 0, 0, 0};
};

bool method_long(PyObject *t, PyObject *name, long long &v) {
    PyObject *r = PyObject_CallMethodNoArgs(t, name);
    if (!r) return false;
    v = PyLong_Check(r) ? PyLong_AsLongLong(r) : (PyErr_SetNone(PyExc_TypeError), -1);
    Py_DECREF(r);
    return !(v == -1 && PyErr_Occurred());
}

// A torch.Tensor of `dtype` on device `here` and, unless the caller looks at its strides, contiguous.
bool get(PyObject *t, PyObject *dtype, long here, Tensor &x, bool contiguous = true) {
    if (!PyObject_TypeCheck(t, reinterpret_cast<PyTypeObject *>(g_tensor))) return false;
    PyObject *d = PyObject_GetAttr(t, s_dtype);
    if (!d) return false;
    Py_DECREF(d);
    if (d != dtype) return false;
    long long dev;
    if (!method_long(t, s_get_device, dev) || dev != here) return false;
    if (contiguous) {
        PyObject *c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
        if (!c) return false;
        Py_DECREF(c);
        if (c != Py_True) return false;
    }
    PyObject *s = PyObject_GetAttr(t, s_shape);
    if (!s) return false;
    const bool tuple = PyTuple_Check(s) && PyTuple_GET_SIZE(s) <= 4;
    bool ok = tuple;
    x.nd = tuple ? (int)PyTuple_GET_SIZE(s) : 0;
    for (int i = 0; ok && i < x.nd; ++i) {
        PyObject *n = PyTuple_GET_ITEM(s, i);
        ok = PyLong_Check(n);
        if (ok) x.size[i] = PyLong_AsLongLong(n);
    }
    Py_DECREF(s);
    if (!ok) return false;
    PyObject *p = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!p) return false;
    x.ptr = PyLong_AsVoidPtr(p);
    Py_DECREF(p);
    return !PyErr_Occurred();
}

bool shaped(const Tensor &x, int nd, long long a, long long b = 0, long long c = 0) {
    const long long want[3] = {a, b, c};
    if (x.nd != nd) return false;
    for (int i = 0; i < nd; ++i)
        if (x.size[i] != want[i]) return false;
    return true;
}

bool to_int(PyObject *o, long long lo, long long hi, long long &v) {
    if (!PyLong_Check(o)) return false;
    v = PyLong_AsLongLong(o);
    return !(v == -1 && PyErr_Occurred()) && v >= lo && v <= hi;
}

// The pools, their scales, the page table and the lengths of a call.
struct Cache {
    Tensor k, v, ks, vs, table, lens;
    int kv_dtype, D, Hk, P, pages, B, pt_stride;

    bool get_all(PyObject *const *o, long here) {  // k, v, page_table, seq_lens, k_scale, v_scale
        PyObject *dt = PyObject_TypeCheck(o[0], reinterpret_cast<PyTypeObject *>(g_tensor)) ? PyObject_GetAttr(o[0], s_dtype) : nullptr;
        if (!dt) return false;
        Py_DECREF(dt);  // (the dtypes live as long as torch)
        if (dt != g_bf16 && dt != g_u8 && dt != g_e4m3) return false;
        if (!get(o[0], dt, here, k) || !get(o[1], dt, here, v) || k.nd != 4 || v.nd != 4) return false;
        for (int i = 0; i < 4; ++i)
            if (k.size[i] != v.size[i] || k.size[i] > INT_MAX) return false;
        pages = (int)k.size[0];
        Hk = (int)k.size[1];
        P = (int)k.size[2];
        D = (int)k.size[3];
        kv_dtype = dt == g_bf16 ? GQA_KV_BF16 : GQA_KV_FP8_E4M3;
        if (dt == g_u8 && (D == 36 || D == 72)) {
            kv_dtype = GQA_KV_FP4;
            D = D / 9 * 16;
        }
        if (!get(o[2], g_i32, here, table) || !get(o[3], g_i32, here, lens)) return false;
        if (table.nd != 2 || lens.nd != 1 || table.size[0] != lens.size[0]) return false;
        if (table.size[0] > INT_MAX || table.size[1] > INT_MAX) return false;
        B = (int)table.size[0];
        pt_stride = (int)table.size[1];
        for (int i = 0; i < 2; ++i) {
            Tensor &s = i ? vs : ks;
            if (o[4 + i] == Py_None) {
                if (kv_dtype == GQA_KV_FP8_E4M3) return false;
                continue;
            }
            if (kv_dtype == GQA_KV_BF16 || !get(o[4 + i], g_f32, here, s)) return false;
            if (kv_dtype == GQA_KV_FP4 ? !shaped(s, 1, Hk) : !shaped(s, 2, pages, Hk)) return false;
        }
        return true;
    }
    const float *k_scale() const { return static_cast<const float *>(ks.ptr); }
    const float *v_scale() const { return static_cast<const float *>(vs.ptr); }
    const int32_t *page_table() const { return static_cast<const int32_t *>(table.ptr); }
    const int32_t *seq_lens() const { return static_cast<const int32_t *>(lens.ptr); }
};

PyObject *no() {
    PyErr_Clear();
    Py_RETURN_NONE;
}

// The last two arguments of every function: the device the call is on and its raw stream.
bool tail(PyObject *const *o, long &here, cudaStream_t &stream) {
    long long h;
    if (!to_int(o[0], 0, INT_MAX, h) || !PyLong_Check(o[1])) return false;
    here = (long)h;
    stream = static_cast<cudaStream_t>(PyLong_AsVoidPtr(o[1]));
    return !PyErr_Occurred();
}

#define CALL(expr)              \
    int status;                 \
    Py_BEGIN_ALLOW_THREADS;     \
    status = (expr);            \
    Py_END_ALLOW_THREADS;       \
    return PyLong_FromLong(status)

// decode(partial, q, k, v, table, lens, k_scale, v_scale, scale, num_splits, pack, out, lse, ws, here, stream)
PyObject *decode(PyObject *, PyObject *const *o, Py_ssize_t n) {
    long here;
    cudaStream_t stream;
    Cache c;
    Tensor q, out, lse, ws;
    long long splits, pack;
    if (n != 16) return no();
    const bool partial = o[0] == Py_True;
    if (!tail(o + 14, here, stream) || !c.get_all(o + 2, here) || !get(o[1], g_bf16, here, q) || q.nd != 3) return no();
    if (q.size[0] != c.B || q.size[2] != c.D || q.size[1] > INT_MAX) return no();
    const double scale = PyFloat_AsDouble(o[8]);
    if (PyErr_Occurred() || !to_int(o[9], INT_MIN, INT_MAX, splits) || !to_int(o[10], 0, 1, pack)) return no();
    if (!get(o[11], partial ? g_f32 : g_bf16, here, out) || !shaped(out, 3, c.B, q.size[1], c.D)) return no();
    if (o[12] != Py_None && (!get(o[12], g_f32, here, lse) || !shaped(lse, 2, c.B, q.size[1]))) return no();
    if (!get(o[13], g_u8, here, ws) || ws.nd != 1) return no();
    float *lse_out = static_cast<float *>(lse.ptr);
    if (partial) {
        CALL(f_partial(q.ptr, c.k.ptr, c.v.ptr, c.k_scale(), c.v_scale(), c.kv_dtype, c.page_table(), c.pt_stride, c.seq_lens(),
                       c.B, (int)q.size[1], c.Hk, c.D, c.P, c.pages, (float)scale, (int)splits, (int)pack,
                       static_cast<float *>(out.ptr), lse_out, ws.ptr, (size_t)ws.size[0], stream));
    }
    CALL(f_decode(q.ptr, c.k.ptr, c.v.ptr, c.k_scale(), c.v_scale(), c.kv_dtype, c.page_table(), c.pt_stride, c.seq_lens(), c.B,
                  (int)q.size[1], c.Hk, c.D, c.P, c.pages, (float)scale, (int)splits, (int)pack, out.ptr, lse_out, ws.ptr,
                  (size_t)ws.size[0], stream));
}

// append_kv(k_new, v_new, k, v, table, lens, k_scale, v_scale, ws, here, stream)
PyObject *append_kv(PyObject *, PyObject *const *o, Py_ssize_t n) {
    long here;
    cudaStream_t stream;
    Cache c;
    Tensor kn, vn, ws;
    if (n != 11 || !tail(o + 9, here, stream) || !c.get_all(o + 2, here)) return no();
    if (!get(o[0], g_bf16, here, kn) || !shaped(kn, 3, c.B, c.Hk, c.D) || !get(o[1], g_bf16, here, vn) ||
        !shaped(vn, 3, c.B, c.Hk, c.D) || !get(o[8], g_u8, here, ws) || ws.nd != 1 || ws.size[0] < 256)
        return no();
    CALL(f_append(kn.ptr, vn.ptr, c.k.ptr, c.v.ptr, static_cast<float *>(c.ks.ptr), static_cast<float *>(c.vs.ptr), c.kv_dtype,
                  c.page_table(), c.pt_stride, c.seq_lens(), c.B, c.Hk, c.D, c.P, c.pages, ws.ptr, stream));
}

// append_decode(q, k_new, v_new, k, v, table, lens, k_scale, v_scale, scale, num_splits, pack, out, lse, ws, here, stream)
PyObject *append_decode(PyObject *, PyObject *const *o, Py_ssize_t n) {
    long here;
    cudaStream_t stream;
    Cache c;
    Tensor q, kn, vn, out, lse, ws;
    long long splits, pack;
    if (n != 17 || !tail(o + 15, here, stream) || !c.get_all(o + 3, here) || !get(o[0], g_bf16, here, q) || q.nd != 3) return no();
    if (q.size[0] != c.B || q.size[2] != c.D || q.size[1] > INT_MAX) return no();
    if (!get(o[1], g_bf16, here, kn) || !shaped(kn, 3, c.B, c.Hk, c.D) || !get(o[2], g_bf16, here, vn) ||
        !shaped(vn, 3, c.B, c.Hk, c.D))
        return no();
    const double scale = PyFloat_AsDouble(o[9]);
    if (PyErr_Occurred() || !to_int(o[10], INT_MIN, INT_MAX, splits) || !to_int(o[11], 0, 1, pack)) return no();
    if (!get(o[12], g_bf16, here, out) || !shaped(out, 3, c.B, q.size[1], c.D)) return no();
    if (o[13] != Py_None && (!get(o[13], g_f32, here, lse) || !shaped(lse, 2, c.B, q.size[1]))) return no();
    if (!get(o[14], g_u8, here, ws) || ws.nd != 1) return no();
    CALL(f_append_decode(q.ptr, kn.ptr, vn.ptr, c.k.ptr, c.v.ptr, static_cast<float *>(c.ks.ptr), static_cast<float *>(c.vs.ptr),
                         c.kv_dtype, c.page_table(), c.pt_stride, c.seq_lens(), c.B, (int)q.size[1], c.Hk, c.D, c.P, c.pages,
                         (float)scale, (int)splits, (int)pack, out.ptr, static_cast<float *>(lse.ptr), ws.ptr,
                         (size_t)ws.size[0], stream));
}

// bf16 rows [T][Hk][D], contiguous inside a row; elements from one row to the next.
bool get_rows(PyObject *o, long here, const Cache &c, Tensor &x, long long &stride) {
    if (!get(o, g_bf16, here, x, false) || x.nd != 3 || x.size[1] != c.Hk || x.size[2] != c.D) return false;
    PyObject *s = PyObject_CallMethodNoArgs(o, s_stride);
    if (!s) return false;
    long long st[3] = {0, 0, 0};
    bool ok = PyTuple_Check(s) && PyTuple_GET_SIZE(s) == 3;
    for (int i = 0; ok && i < 3; ++i) {
        PyObject *v = PyTuple_GET_ITEM(s, i);
        ok = PyLong_Check(v);
        if (ok) st[i] = PyLong_AsLongLong(v);
    }
    Py_DECREF(s);
    stride = x.size[0] > 1 ? st[0] : (long long)c.Hk * c.D;
    return ok && st[2] == 1 && (c.Hk == 1 || st[1] == c.D);
}

// write_kv(k_new, v_new, cu_q, k, v, table, lens, k_scale, v_scale, max_q_len, ws, here, stream)
PyObject *write_kv(PyObject *, PyObject *const *o, Py_ssize_t n) {
    long here;
    cudaStream_t stream;
    Cache c;
    Tensor kn, vn, cu, ws;
    long long ks, vs, max_q;
    if (n != 13 || !tail(o + 11, here, stream) || !c.get_all(o + 3, here)) return no();
    if (!get_rows(o[0], here, c, kn, ks) || !get_rows(o[1], here, c, vn, vs) || kn.size[0] != vn.size[0] ||
        kn.size[0] > INT_MAX || kn.size[0] == 0)
        return no();
    if (!get(o[2], g_i32, here, cu) || !shaped(cu, 1, (long long)c.B + 1) || !to_int(o[9], 0, INT_MAX, max_q) ||
        !get(o[10], g_u8, here, ws) || ws.nd != 1 || ws.size[0] < 256)
        return no();
    CALL(f_write(kn.ptr, vn.ptr, ks, vs, static_cast<const int32_t *>(cu.ptr), c.k.ptr, c.v.ptr, static_cast<float *>(c.ks.ptr),
                 static_cast<float *>(c.vs.ptr), c.kv_dtype, c.page_table(), c.pt_stride, c.seq_lens(), c.B, c.Hk, c.D, c.P,
                 c.pages, (int)kn.size[0], (int)max_q, ws.ptr, stream));
}

// read_kv(k, v, table, lens, k_scale, v_scale, starts, cu, total, paged, k_out, v_out, ws, here, stream)
PyObject *read_kv(PyObject *, PyObject *const *o, Py_ssize_t n) {
    long here;
    cudaStream_t stream;
    Cache c;
    Tensor starts, cu, ko, vo, ws;
    long long total, paged;
    if (n != 15 || !tail(o + 13, here, stream) || !c.get_all(o, here)) return no();
    if (o[6] != Py_None && (!get(o[6], g_i32, here, starts) || !shaped(starts, 1, c.B))) return no();
    if (!get(o[7], g_i64, here, cu) || !shaped(cu, 1, (long long)c.B + 1) || !to_int(o[8], 1, LLONG_MAX, total) ||
        !to_int(o[9], 0, 1, paged))
        return no();
    for (int i = 0; i < 2; ++i) {
        Tensor &x = i ? vo : ko;
        if (!get(o[10 + i], g_bf16, here, x)) return no();
        if (paged) {
            if (x.nd != 4 || x.size[0] != total || x.size[1] != c.Hk || x.size[2] != c.P || x.size[3] != c.D) return no();
        } else if (!shaped(x, 3, total, c.Hk, c.D)) {
            return no();
        }
    }
    if (!get(o[12], g_u8, here, ws) || ws.nd != 1 || ws.size[0] < 256) return no();
    CALL(f_read(c.k.ptr, c.v.ptr, c.k_scale(), c.v_scale(), c.kv_dtype, c.page_table(), c.pt_stride,
                static_cast<const int32_t *>(starts.ptr), c.seq_lens(), static_cast<const int64_t *>(cu.ptr), c.B, c.Hk, c.D,
                c.P, c.pages, total, (int)paged, ko.ptr, vo.ptr, ws.ptr, stream));
}

// init(torch.Tensor, bfloat16, uint8, float8_e4m3fn, float32, int32, int64, addresses of decode, decode_partial,
// append_kv, append_decode, write_kv, read_kv)
PyObject *init(PyObject *, PyObject *const *o, Py_ssize_t n) {
    if (n != 13 || !PyType_Check(o[0])) {
        PyErr_SetString(PyExc_TypeError, "init(Tensor, 6 dtypes, 6 addresses)");
        return nullptr;
    }
    PyObject **keep[7] = {&g_tensor, &g_bf16, &g_u8, &g_e4m3, &g_f32, &g_i32, &g_i64};
    for (int i = 0; i < 7; ++i) {
        Py_INCREF(o[i]);
        Py_XSETREF(*keep[i], o[i]);
    }
    void *f[6];
    for (int i = 0; i < 6; ++i) {
        f[i] = PyLong_AsVoidPtr(o[7 + i]);
        if (!f[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
            return nullptr;
        }
    }
    f_decode = reinterpret_cast<decltype(f_decode)>(f[0]);
    f_partial = reinterpret_cast<decltype(f_partial)>(f[1]);
    f_append = reinterpret_cast<decltype(f_append)>(f[2]);
    f_append_decode = reinterpret_cast<decltype(f_append_decode)>(f[3]);
    f_write = reinterpret_cast<decltype(f_write)>(f[4]);
    f_read = reinterpret_cast<decltype(f_read)>(f[5]);
    Py_RETURN_NONE;
}

#define FN(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FN(init), FN(decode), FN(append_kv), FN(append_decode), FN(write_kv), FN(read_kv), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() {
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    return PyModule_Create(&module);
}
