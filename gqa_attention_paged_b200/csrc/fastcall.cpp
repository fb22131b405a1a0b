// fastcall.cpp -- the checks and the call of binding.py's hottest functions in one C function each.
//
// A decode step of a small batch runs for 5 to 10 us on the GPU; checking ten tensors in Python and
// marshalling twenty arguments through ctypes took another 9 to 12 on the host.  Here a call whose
// tensors are all as they should be (and its outputs and workspace given) goes straight to the
// library; anything else returns None, and binding.py takes its own path with its own errors.  No
// check is weaker than there.  A tensor's address, sizes and type come from DLPack's C exchange
// table, which torch.Tensor publishes for such callers (tens of nanoseconds a tensor, where five
// attributes by way of the interpreter are 260).
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <limits.h>
#include <stdint.h>

#include <ATen/dlpack.h>

#include "gqa_paged.h"

namespace {

PyTypeObject *g_tensor;  // torch.Tensor
const DLPackExchangeAPI *g_api;

// Element types by DLPack's (code, bits).
constexpr int type_key(int code, int bits) { return code * 256 + bits; }
constexpr int kBf16 = type_key(kDLBfloat, 16), kU8 = type_key(kDLUInt, 8), kE4m3 = type_key(kDLFloat8_e4m3fn, 8);
constexpr int kF32 = type_key(kDLFloat, 32), kI32 = type_key(kDLInt, 32), kI64 = type_key(kDLInt, 64);

decltype(&gqa_paged_decode) f_decode;
decltype(&gqa_paged_decode_partial) f_partial;
decltype(&gqa_paged_append_kv) f_append;
decltype(&gqa_paged_append_decode) f_append_decode;
decltype(&gqa_paged_write_kv) f_write;
decltype(&gqa_paged_read_kv) f_read;

struct Tensor {
    void *ptr = nullptr;
    int nd = 0, type = -1;
    long long size[4] = {0, 0, 0, 0}, stride[4] = {0, 0, 0, 0};
};

// A CUDA torch.Tensor on device `here` of at most four dimensions; `type` < 0: of any type.
bool look(PyObject *t, int type, long here, Tensor &x) {
    if (Py_TYPE(t) != g_tensor) return false;  // (subclasses take Python's way)
    DLTensor d;
    if (g_api->dltensor_from_py_object_no_sync(t, &d) != 0) return false;
    x.type = d.dtype.lanes == 1 ? type_key(d.dtype.code, d.dtype.bits) : -1;
    if (d.device.device_type != kDLCUDA || d.device.device_id != here || d.ndim > 4 || (type >= 0 && x.type != type)) return false;
    x.ptr = static_cast<char *>(d.data) + d.byte_offset;
    x.nd = d.ndim;
    long long dense = 1;
    for (int i = d.ndim - 1; i >= 0; --i) {
        x.size[i] = d.shape[i];
        x.stride[i] = d.strides ? d.strides[i] : dense;
        dense *= d.shape[i];
    }
    return true;
}

bool dense(const Tensor &x) {
    long long want = 1, count = 1;
    for (int i = 0; i < x.nd; ++i) count *= x.size[i];
    if (count == 0) return true;
    for (int i = x.nd - 1; i >= 0; --i) {
        if (x.size[i] != 1 && x.stride[i] != want) return false;
        want *= x.size[i];
    }
    return true;
}

bool get(PyObject *t, int type, long here, Tensor &x) { return look(t, type, here, x) && dense(x); }

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
        if (!get(o[0], -1, here, k) || (k.type != kBf16 && k.type != kU8 && k.type != kE4m3)) return false;
        if (!get(o[1], k.type, here, v) || k.nd != 4 || v.nd != 4) return false;
        for (int i = 0; i < 4; ++i)
            if (k.size[i] != v.size[i] || k.size[i] > INT_MAX) return false;
        pages = (int)k.size[0];
        Hk = (int)k.size[1];
        P = (int)k.size[2];
        D = (int)k.size[3];
        kv_dtype = k.type == kBf16 ? GQA_KV_BF16 : GQA_KV_FP8_E4M3;
        if (k.type == kU8 && (D == 36 || D == 72)) {
            kv_dtype = GQA_KV_FP4;
            D = D / 9 * 16;
        }
        if (!get(o[2], kI32, here, table) || !get(o[3], kI32, here, lens)) return false;
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
            if (kv_dtype == GQA_KV_BF16 || !get(o[4 + i], kF32, here, s)) return false;
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

// The last two arguments of every function: the current device, and the stream as a number or None
// for the current one.
bool tail(PyObject *const *o, long &here, cudaStream_t &stream) {
    long long h;
    if (!g_api || !to_int(o[0], 0, INT_MAX, h)) return false;
    here = (long)h;
    void *s = nullptr;
    if (o[1] == Py_None) {
        if (g_api->current_work_stream(kDLCUDA, (int32_t)h, &s) != 0) return false;
    } else {
        if (!PyLong_Check(o[1])) return false;
        s = PyLong_AsVoidPtr(o[1]);
    }
    stream = static_cast<cudaStream_t>(s);
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
    if (!tail(o + 14, here, stream) || !c.get_all(o + 2, here) || !get(o[1], kBf16, here, q) || q.nd != 3) return no();
    if (q.size[0] != c.B || q.size[2] != c.D || q.size[1] > INT_MAX) return no();
    const double scale = PyFloat_AsDouble(o[8]);
    if (PyErr_Occurred() || !to_int(o[9], INT_MIN, INT_MAX, splits) || !to_int(o[10], 0, 1, pack)) return no();
    if (!get(o[11], partial ? kF32 : kBf16, here, out) || !shaped(out, 3, c.B, q.size[1], c.D)) return no();
    if (o[12] != Py_None && (!get(o[12], kF32, here, lse) || !shaped(lse, 2, c.B, q.size[1]))) return no();
    if (!get(o[13], kU8, here, ws) || ws.nd != 1) return no();
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
    if (!get(o[0], kBf16, here, kn) || !shaped(kn, 3, c.B, c.Hk, c.D) || !get(o[1], kBf16, here, vn) ||
        !shaped(vn, 3, c.B, c.Hk, c.D) || !get(o[8], kU8, here, ws) || ws.nd != 1 || ws.size[0] < 256)
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
    if (n != 17 || !tail(o + 15, here, stream) || !c.get_all(o + 3, here) || !get(o[0], kBf16, here, q) || q.nd != 3) return no();
    if (q.size[0] != c.B || q.size[2] != c.D || q.size[1] > INT_MAX) return no();
    if (!get(o[1], kBf16, here, kn) || !shaped(kn, 3, c.B, c.Hk, c.D) || !get(o[2], kBf16, here, vn) ||
        !shaped(vn, 3, c.B, c.Hk, c.D))
        return no();
    const double scale = PyFloat_AsDouble(o[9]);
    if (PyErr_Occurred() || !to_int(o[10], INT_MIN, INT_MAX, splits) || !to_int(o[11], 0, 1, pack)) return no();
    if (!get(o[12], kBf16, here, out) || !shaped(out, 3, c.B, q.size[1], c.D)) return no();
    if (o[13] != Py_None && (!get(o[13], kF32, here, lse) || !shaped(lse, 2, c.B, q.size[1]))) return no();
    if (!get(o[14], kU8, here, ws) || ws.nd != 1) return no();
    CALL(f_append_decode(q.ptr, kn.ptr, vn.ptr, c.k.ptr, c.v.ptr, static_cast<float *>(c.ks.ptr), static_cast<float *>(c.vs.ptr),
                         c.kv_dtype, c.page_table(), c.pt_stride, c.seq_lens(), c.B, (int)q.size[1], c.Hk, c.D, c.P, c.pages,
                         (float)scale, (int)splits, (int)pack, out.ptr, static_cast<float *>(lse.ptr), ws.ptr,
                         (size_t)ws.size[0], stream));
}

// bf16 rows [T][Hk][D], contiguous inside a row; elements from one row to the next.
bool get_rows(PyObject *o, long here, const Cache &c, Tensor &x, long long &stride) {
    if (!look(o, kBf16, here, x) || x.nd != 3 || x.size[1] != c.Hk || x.size[2] != c.D) return false;
    stride = x.size[0] > 1 ? x.stride[0] : (long long)c.Hk * c.D;
    return x.stride[2] == 1 && (c.Hk == 1 || x.stride[1] == c.D);
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
    if (!get(o[2], kI32, here, cu) || !shaped(cu, 1, (long long)c.B + 1) || !to_int(o[9], 0, INT_MAX, max_q) ||
        !get(o[10], kU8, here, ws) || ws.nd != 1 || ws.size[0] < 256)
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
    if (o[6] != Py_None && (!get(o[6], kI32, here, starts) || !shaped(starts, 1, c.B))) return no();
    if (!get(o[7], kI64, here, cu) || !shaped(cu, 1, (long long)c.B + 1) || !to_int(o[8], 1, LLONG_MAX, total) ||
        !to_int(o[9], 0, 1, paged))
        return no();
    for (int i = 0; i < 2; ++i) {
        Tensor &x = i ? vo : ko;
        if (!get(o[10 + i], kBf16, here, x)) return no();
        if (paged) {
            if (x.nd != 4 || x.size[0] != total || x.size[1] != c.Hk || x.size[2] != c.P || x.size[3] != c.D) return no();
        } else if (!shaped(x, 3, total, c.Hk, c.D)) {
            return no();
        }
    }
    if (!get(o[12], kU8, here, ws) || ws.nd != 1 || ws.size[0] < 256) return no();
    CALL(f_read(c.k.ptr, c.v.ptr, c.k_scale(), c.v_scale(), c.kv_dtype, c.page_table(), c.pt_stride,
                static_cast<const int32_t *>(starts.ptr), c.seq_lens(), static_cast<const int64_t *>(cu.ptr), c.B, c.Hk, c.D,
                c.P, c.pages, total, (int)paged, ko.ptr, vo.ptr, ws.ptr, stream));
}

// init(torch.Tensor, addresses of decode, decode_partial, append_kv, append_decode, write_kv, read_kv): whether
// torch has the exchange table; without it every call below returns None.
PyObject *init(PyObject *, PyObject *const *o, Py_ssize_t n) {
    if (n != 7 || !PyType_Check(o[0])) {
        PyErr_SetString(PyExc_TypeError, "init(Tensor, 6 addresses)");
        return nullptr;
    }
    void *f[6];
    for (int i = 0; i < 6; ++i) {
        f[i] = PyLong_AsVoidPtr(o[1 + i]);
        if (!f[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
            return nullptr;
        }
    }
    g_api = nullptr;
    PyObject *capsule = PyObject_GetAttrString(o[0], "__dlpack_c_exchange_api__");
    if (capsule && PyCapsule_IsValid(capsule, "dlpack_exchange_api")) {
        const auto *api = static_cast<const DLPackExchangeAPI *>(PyCapsule_GetPointer(capsule, "dlpack_exchange_api"));
        if (api && api->header.version.major == DLPACK_MAJOR_VERSION && api->dltensor_from_py_object_no_sync &&
            api->current_work_stream)
            g_api = api;  // (lives as long as torch)
    }
    Py_XDECREF(capsule);
    PyErr_Clear();
    g_tensor = reinterpret_cast<PyTypeObject *>(o[0]);
    Py_INCREF(o[0]);
    f_decode = reinterpret_cast<decltype(f_decode)>(f[0]);
    f_partial = reinterpret_cast<decltype(f_partial)>(f[1]);
    f_append = reinterpret_cast<decltype(f_append)>(f[2]);
    f_append_decode = reinterpret_cast<decltype(f_append_decode)>(f[3]);
    f_write = reinterpret_cast<decltype(f_write)>(f[4]);
    f_read = reinterpret_cast<decltype(f_read)>(f[5]);
    return PyBool_FromLong(g_api != nullptr);
}

#define FN(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FN(init), FN(decode), FN(append_kv), FN(append_decode), FN(write_kv), FN(read_kv), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() {
    return PyModule_Create(&module);
}
