// Python entry points of the decoder-layer operators (CPython API, no torch headers):
// reads types, shapes and strides from the tensors, checks them and calls the C ABI of
// moehost.h, whose addresses bind() receives.  In Python the same checks and the
// marshalling took 5 to 7 us of a call's 8 to 10; here they take about 2.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <type_traits>

#include "moehost.h"

namespace {

// ---- what bind() receives ------------------------------------------------------

PyObject* g_error = nullptr;       // MoeError(code, where)
PyObject* g_raw_stream = nullptr;  // torch: device index -> cudaStream_t of the current stream
PyObject* g_current = nullptr;     // torch: index of the current device
enum { kBf16, kF16, kF32, kE4m3, kI32, kI64, kTypes };
PyObject* g_types[kTypes];  // torch dtypes in that order; the first four are moehost.h's codes

decltype(&moe_add_rms_norm) f_norm = nullptr;
decltype(&moe_kv_append) f_append = nullptr;
decltype(&moe_kv_attend) f_attend = nullptr;
decltype(&moe_linear) f_linear = nullptr;
decltype(&moe_quant_e4m3) f_quant = nullptr;
decltype(&moe_kv_append_axes) f_append_axes = nullptr;
decltype(&moe_linear_blocks) f_linear_blocks = nullptr;

PyObject *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_get_device, *s_device_index, *s_cuda_stream, *s_call;

// ---- errors ---------------------------------------------------------------------

void raise(int code, const char* where, const char* what, const char* why) {
    char text[256];
    if (what) snprintf(text, sizeof text, "%s: %s %s", where, what, why);
    else snprintf(text, sizeof text, "%s", where);
    PyObject* e = PyObject_CallFunction(g_error, "is", code, text);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
}
// One call of an entry point: its name, and the GPU that its tensors are on (-1 before the first).
// The library launches on the current device, whatever memory it is given, so that this GPU has
// to be the current one and every tensor's: anything else is refused before the launch.
struct Call {
    const char* name;
    int device = -1;
};
bool refuse(const Call& c, const char* what, const char* why) {
    raise(MOE_ERR_INVALID_ARG, c.name, what, why);
    return false;
}
PyObject* finish(int code, const char* where) {
    if (code != MOE_OK) {
        raise(code, where, nullptr, nullptr);
        return nullptr;
    }
    Py_RETURN_NONE;
}

// ---- tensors --------------------------------------------------------------------

constexpr int kDims = 4;
struct Tensor {
    void* ptr = nullptr;
    int type = -1, dims = 0;
    int64_t shape[kDims] = {}, stride[kDims] = {};
};

bool read_sizes(PyObject* seq, int64_t (&out)[kDims], int& n) {
    if (!seq) return false;
    bool ok = PyTuple_Check(seq);
    if (ok) {
        n = (int)PyTuple_GET_SIZE(seq);
        ok = n <= kDims;
        for (int i = 0; ok && i < n; ++i) out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(seq, i));
        if (!ok) n = kDims + 1;  // more dimensions than any argument has
    } else {
        PyErr_SetString(PyExc_TypeError, "a tensor was expected");
    }
    Py_DECREF(seq);
    return (ok || n > kDims) && !PyErr_Occurred();
}

// An integer that a call of torch's gave (and which is let go of here); false with an exception set.
bool small_int(PyObject* o, int& v) {
    if (!o) return false;
    v = (int)PyLong_AsLong(o);
    Py_DECREF(o);
    return !PyErr_Occurred();
}

bool on_device(Call& c, int device, const char* name) {
    if (device < 0) return refuse(c, name, "is not on a GPU");
    if (c.device < 0) {
        int now = -1;
        if (!small_int(PyObject_CallNoArgs(g_current), now)) return false;
        if (device != now) return refuse(c, name, "is not on the current GPU");
        c.device = device;
    }
    return device == c.device || refuse(c, name, "is on another GPU than the call's other tensors");
}

// Fills t from a CUDA tensor of one of the known types; false with an exception set.
bool read(PyObject* o, Tensor& t, Call& where, const char* name) {
    PyObject* d = PyObject_GetAttr(o, s_dtype);
    if (!d) return false;
    for (int i = 0; i < kTypes; ++i)
        if (d == g_types[i]) t.type = i;
    Py_DECREF(d);
    if (t.type < 0) return refuse(where, name, "has a type that the call does not take");
    int n = 0, device = -1;  // -1: a CPU tensor
    if (!small_int(PyObject_CallMethodNoArgs(o, s_get_device), device) || !on_device(where, device, name)) return false;
    if (!read_sizes(PyObject_GetAttr(o, s_shape), t.shape, t.dims) ||
        !read_sizes(PyObject_CallMethodNoArgs(o, s_stride), t.stride, n))
        return false;
    PyObject* p = PyObject_CallMethodNoArgs(o, s_data_ptr);
    if (!p) return false;
    t.ptr = PyLong_AsVoidPtr(p);
    Py_DECREF(p);
    return !PyErr_Occurred();
}

bool given(PyObject* o) { return o && o != Py_None; }

// A matrix [rows, cols] of any of the element types with contiguous rows.
bool matrix(PyObject* o, Tensor& t, int64_t rows, int64_t cols, Call& where, const char* name) {
    if (!read(o, t, where, name)) return false;
    if (t.type > kE4m3) return refuse(where, name, "has a type that the call does not take");
    if (t.dims != 2 || (rows >= 0 && (t.shape[0] != rows || t.shape[1] != cols)))
        return refuse(where, name, "has another shape than the call's other tensors need");
    if (t.stride[1] != 1 && t.shape[1] > 1) return refuse(where, name, "is not contiguous in its last dimension");
    return true;
}

// A contiguous vector of n elements; type < 0: any of the element types.
bool vector(PyObject* o, Tensor& t, int64_t n, int type, Call& where, const char* name) {
    if (!read(o, t, where, name)) return false;
    if (type >= 0 ? t.type != type : t.type > kE4m3) return refuse(where, name, "has a type that the call does not take");
    if (t.dims != 1 || t.shape[0] != n || (n > 1 && t.stride[0] != 1))
        return refuse(where, name, "is not a contiguous vector of the call's length");
    return true;
}

// fp32 [rows, blocks], contiguous in its last dimension.
bool scales(PyObject* o, Tensor& t, int64_t rows, int64_t blocks, Call& where, const char* name) {
    if (!matrix(o, t, rows, blocks, where, name)) return false;
    return t.type == kF32 || refuse(where, name, "has a type that the call does not take");
}

// [rows, heads, dim] of one type, contiguous in its last dimension.
bool heads(PyObject* o, Tensor& t, int64_t rows, int64_t n, int64_t dim, int type, Call& where, const char* name) {
    if (!read(o, t, where, name)) return false;
    if (t.type > kE4m3 || (type >= 0 && t.type != type)) return refuse(where, name, "has a type that the call does not take");
    if (t.dims != 3 || (rows >= 0 && t.shape[0] != rows) || t.shape[1] != n || t.shape[2] != dim)
        return refuse(where, name, "has another shape than the call's other tensors need");
    if (t.stride[2] != 1) return refuse(where, name, "is not contiguous in its last dimension");
    return true;
}

// ---- other arguments --------------------------------------------------------------

// cudaStream_t: a torch stream of the call's device, an integer, or None for torch's current
// stream of that device.
bool stream_of(PyObject* o, Call& c, void*& out) {
    PyObject* r;
    if (!given(o)) {
        PyObject* d = PyLong_FromLong(c.device);
        if (!d) return false;
        r = PyObject_CallOneArg(g_raw_stream, d);
        Py_DECREF(d);
    } else if (PyLong_Check(o)) {
        r = Py_NewRef(o);
    } else {
        int device = -1;
        if (!small_int(PyObject_GetAttr(o, s_device_index), device) || !on_device(c, device, "stream")) return false;
        r = PyObject_GetAttr(o, s_cuda_stream);
    }
    if (!r) return false;
    out = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    return !PyErr_Occurred();
}

// Positional and keyword arguments into slots by name; the first `needed` have to be there.
template <int N>
bool arguments(PyObject* const* args, Py_ssize_t n, PyObject* kw, const char* where, PyObject* (&names)[N], int needed,
               PyObject* (&out)[N]) {
    if (n > N) {
        PyErr_Format(PyExc_TypeError, "%s takes at most %d arguments", where, N);
        return false;
    }
    for (int i = 0; i < N; ++i) out[i] = i < n ? args[i] : nullptr;
    const Py_ssize_t k = kw ? PyTuple_GET_SIZE(kw) : 0;
    for (Py_ssize_t i = 0; i < k; ++i) {
        PyObject* key = PyTuple_GET_ITEM(kw, i);
        int at = -1;
        for (int j = 0; j < N && at < 0; ++j)
            if (key == names[j]) at = j;
        for (int j = 0; j < N && at < 0; ++j)  // a name that was not interned
            if (PyUnicode_Compare(key, names[j]) == 0) at = j;
        if (at < 0 || out[at]) {
            PyErr_Format(PyExc_TypeError, "%s: argument %R is unknown or given twice", where, key);
            return false;
        }
        out[at] = args[n + i];
    }
    for (int i = 0; i < needed; ++i)
        if (!out[i]) {
            PyErr_Format(PyExc_TypeError, "%s: argument %R is missing", where, names[i]);
            return false;
        }
    return true;
}

bool number(PyObject* o, double& v) {
    if (given(o)) v = PyFloat_AsDouble(o);
    return !PyErr_Occurred();
}
bool integer(PyObject* o, int& v) {
    if (given(o)) {
        const long x = PyLong_AsLong(o);
        if (PyErr_Occurred()) return false;
        v = x < INT32_MIN ? INT32_MIN : (x > INT32_MAX ? INT32_MAX : (int)x);
    }
    return true;
}

// The axis of each of `pairs` pairs: bytes, or any sequence of small integers.
constexpr int kMaxPairs = 128;
bool axis_list(PyObject* o, uint8_t (&out)[kMaxPairs], int64_t pairs, const Call& w) {
    if (PyBytes_Check(o) && PyBytes_GET_SIZE(o) == pairs && pairs <= kMaxPairs) {
        memcpy(out, PyBytes_AS_STRING(o), (size_t)pairs);
        return true;
    }
    PyObject* s = PySequence_Fast(o, "axes: a sequence was expected");
    if (!s) return false;
    bool ok = PySequence_Fast_GET_SIZE(s) == pairs && pairs <= kMaxPairs;
    for (int64_t i = 0; ok && i < pairs; ++i) {
        const long a = PyLong_AsLong(PySequence_Fast_GET_ITEM(s, i));
        ok = a >= 0 && a < 256 && !PyErr_Occurred();
        if (ok) out[i] = (uint8_t)a;
    }
    Py_DECREF(s);
    return ok || (!PyErr_Occurred() && refuse(w, "axes", "do not give each pair of the table an axis"));
}

// handle, q_heads, kv_heads, head_dim and device of a KvCache
struct Cache {
    moe_kv* kv = nullptr;
    int64_t q_heads = 0, kv_heads = 0, dim = 0;
};
bool cache_of(PyObject* o, Cache& c, Call& where) {
    PyObject* t = PyObject_GetAttr(o, s_call);
    if (!t) return false;
    const bool ok = PyTuple_Check(t) && PyTuple_GET_SIZE(t) == 5;
    int device = -1;
    if (ok) {
        c.kv = static_cast<moe_kv*>(PyLong_AsVoidPtr(PyTuple_GET_ITEM(t, 0)));
        c.q_heads = PyLong_AsLongLong(PyTuple_GET_ITEM(t, 1));
        c.kv_heads = PyLong_AsLongLong(PyTuple_GET_ITEM(t, 2));
        c.dim = PyLong_AsLongLong(PyTuple_GET_ITEM(t, 3));
        device = (int)PyLong_AsLong(PyTuple_GET_ITEM(t, 4));
    }
    Py_DECREF(t);
    if (!ok) return refuse(where, "the cache", "is closed");
    return !PyErr_Occurred() && on_device(where, device, "the cache");
}

// ---- the operators ------------------------------------------------------------------

PyObject* n_norm[8];
PyObject* py_norm(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    Call w{"moe_add_rms_norm"};
    PyObject* v[8];  // x, weight, y, residual, sum_out, scale, eps, stream
    if (!arguments(args, n, kw, w.name, n_norm, 3, v)) return nullptr;
    Tensor x, y, wt, r, s, sc;
    double eps = 1e-6;
    void* st = nullptr;
    if (!matrix(v[0], x, -1, 0, w, "x")) return nullptr;
    const int64_t T = x.shape[0], H = x.shape[1];
    if (!matrix(v[2], y, T, H, w, "y")) return nullptr;
    if (given(v[1]) && !vector(v[1], wt, H, -1, w, "weight")) return nullptr;
    if (given(v[3]) && !matrix(v[3], r, T, H, w, "residual")) return nullptr;
    if (given(v[4]) && !matrix(v[4], s, T, H, w, "sum_out")) return nullptr;
    if (given(v[3]) && given(v[4]) && r.type != s.type) return refuse(w, "sum_out", "has another type than residual"), nullptr;
    if (given(v[5]) && !vector(v[5], sc, T, kF32, w, "scale")) return nullptr;
    if (!number(v[6], eps) || !stream_of(v[7], w, st)) return nullptr;
    if (T > INT32_MAX || H > INT32_MAX) return refuse(w, "x", "is too large"), nullptr;
    return finish(f_norm(x.ptr, x.type, x.stride[0], r.ptr, given(v[3]) ? r.type : s.type, r.stride[0], wt.ptr, wt.type,
                         (float)eps, (int)T, (int)H, s.ptr, s.stride[0], y.ptr, y.type, y.stride[0],
                         static_cast<float*>(sc.ptr), st),
                  w.name);
}

PyObject* n_quant[4];
PyObject* py_quant(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    Call w{"moe_quant_e4m3"};
    PyObject* v[4];  // x, y, scale, stream
    if (!arguments(args, n, kw, w.name, n_quant, 3, v)) return nullptr;
    Tensor x, y, sc;
    void* st = nullptr;
    if (!matrix(v[0], x, -1, 0, w, "x")) return nullptr;
    const int64_t T = x.shape[0], K = x.shape[1];
    if (x.type == kE4m3) return refuse(w, "x", "has a type that the call does not take"), nullptr;
    if (!matrix(v[1], y, T, K, w, "y")) return nullptr;
    if (y.type != kE4m3) return refuse(w, "y", "has a type that the call does not take"), nullptr;
    if (!scales(v[2], sc, T, (K + 127) / 128, w, "scale") || !stream_of(v[3], w, st)) return nullptr;
    if (T > INT32_MAX || K > INT32_MAX) return refuse(w, "x", "is too large"), nullptr;
    return finish(f_quant(x.ptr, x.type, x.stride[0], (int)T, (int)K, y.ptr, y.stride[0], static_cast<float*>(sc.ptr),
                          sc.stride[0], st),
                  w.name);
}

PyObject* n_append[11];
PyObject* py_append(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    Call w{"moe_kv_append"};
    PyObject* v[11];  // kv, q, k, v, positions, slots, cos_sin, q_out, interleaved, stream, axes
    if (!arguments(args, n, kw, w.name, n_append, 8, v)) return nullptr;
    Cache c;
    Tensor q, k, x, o, pos, slots, cs;
    void* st = nullptr;
    if (!cache_of(v[0], c, w) || !heads(v[1], q, -1, c.q_heads, c.dim, -1, w, "q")) return nullptr;
    const int64_t T = q.shape[0];
    if (!heads(v[2], k, T, c.kv_heads, c.dim, q.type, w, "k") || !heads(v[3], x, T, c.kv_heads, c.dim, q.type, w, "v") ||
        !heads(v[7], o, T, c.q_heads, c.dim, q.type, w, "q_out") || !vector(v[5], slots, T, kI64, w, "slots"))
        return nullptr;
    if (given(v[6])) {
        if (!matrix(v[6], cs, -1, 0, w, "cos_sin")) return nullptr;
        if (cs.type != kF32 || (cs.stride[0] != cs.shape[1] && cs.shape[0] > 1) || cs.shape[0] > INT32_MAX)
            return refuse(w, "cos_sin", "is not a contiguous fp32 table"), nullptr;
        if (!given(v[10]) && !vector(v[4], pos, T, kI32, w, "positions")) return nullptr;
    }
    const int turn = given(v[8]) ? PyObject_IsTrue(v[8]) : 0;
    if (turn < 0) return nullptr;
    uint8_t axis[kMaxPairs];
    if (given(v[10])) {
        if (!given(v[6])) return refuse(w, "axes", "are given without cos_sin"), nullptr;
        if (!read(v[4], pos, w, "positions")) return nullptr;
        if (pos.type != kI32 || pos.dims != 2 || pos.shape[1] != T || (T > 1 && pos.stride[1] != 1))
            return refuse(w, "positions", "is not an int32 [axes, T] with contiguous rows"), nullptr;
        if (pos.shape[0] > INT32_MAX) return refuse(w, "positions", "is too large"), nullptr;
        if (!axis_list(v[10], axis, cs.shape[1] / 2, w)) return nullptr;
    }
    if (!stream_of(v[9], w, st)) return nullptr;
    if (T > INT32_MAX || cs.shape[1] > 1024) return refuse(w, "q or cos_sin", "is too large"), nullptr;
    if (given(v[10]))
        return finish(f_append_axes(c.kv, q.type, q.ptr, q.stride[0], q.stride[1], k.ptr, k.stride[0], k.stride[1], x.ptr,
                                    x.stride[0], x.stride[1], static_cast<int32_t*>(pos.ptr), pos.stride[0],
                                    (int)pos.shape[0], axis, static_cast<int64_t*>(slots.ptr),
                                    static_cast<float*>(cs.ptr), (int)cs.shape[0], (int)cs.shape[1], turn, (int)T, o.ptr,
                                    o.stride[0], o.stride[1], st),
                      w.name);
    return finish(f_append(c.kv, q.type, q.ptr, q.stride[0], q.stride[1], k.ptr, k.stride[0], k.stride[1], x.ptr,
                           x.stride[0], x.stride[1], static_cast<int32_t*>(pos.ptr), static_cast<int64_t*>(slots.ptr),
                           static_cast<float*>(cs.ptr), (int)cs.shape[0], (int)cs.shape[1], turn, (int)T, o.ptr,
                           o.stride[0], o.stride[1], st),
                  w.name);
}

PyObject* n_attend[9];
PyObject* py_attend(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    Call w{"moe_kv_attend"};
    PyObject* v[9];  // kv, q, page_table, lengths, out, scale, window, lse, stream
    if (!arguments(args, n, kw, w.name, n_attend, 5, v)) return nullptr;
    Cache c;
    Tensor q, o, table, len, lse;
    int window = 0;
    void* st = nullptr;
    if (!cache_of(v[0], c, w) || !heads(v[1], q, -1, c.q_heads, c.dim, -1, w, "q")) return nullptr;
    const int64_t B = q.shape[0];
    if (!heads(v[4], o, B, c.q_heads, c.dim, q.type, w, "out") || !vector(v[3], len, B, kI32, w, "lengths") ||
        !read(v[2], table, w, "page_table"))
        return nullptr;
    if (table.type != kI32 || table.dims != 2 || table.shape[0] != B || table.shape[1] > INT32_MAX ||
        (table.shape[1] > 1 && table.stride[1] != 1))
        return refuse(w, "page_table", "is not an int32 [B, max_pages] with contiguous rows"), nullptr;
    if (given(v[7])) {
        if (!read(v[7], lse, w, "lse")) return nullptr;
        if (lse.type != kF32 || lse.dims != 2 || lse.shape[0] != B || lse.shape[1] != c.q_heads ||
            (c.q_heads > 1 && lse.stride[1] != 1) || (B > 1 && lse.stride[0] != c.q_heads))
            return refuse(w, "lse", "is not a contiguous fp32 [B, q_heads]"), nullptr;
    }
    double scale = given(v[5]) ? 0.0 : 1.0;
    if (given(v[5])) {
        if (!number(v[5], scale)) return nullptr;
    } else {
        scale = 1.0 / __builtin_sqrt((double)c.dim);
    }
    if (!integer(v[6], window) || !stream_of(v[8], w, st)) return nullptr;
    if (B > INT32_MAX) return refuse(w, "q", "is too large"), nullptr;
    return finish(f_attend(c.kv, q.ptr, q.type, q.stride[0], q.stride[1], static_cast<int32_t*>(table.ptr),
                           table.stride[0], (int)table.shape[1], static_cast<int32_t*>(len.ptr), (int)B, (float)scale,
                           window, o.ptr, o.stride[0], o.stride[1], static_cast<float*>(lse.ptr), st),
                  w.name);
}

PyObject* g_acts[4];  // "none", "relu", "silu", "gelu"

// What moe_linear and moe_linear_blocks take alike, read and checked.
struct Product {
    Tensor x, w, y, bias, residual, status;
    int64_t T = 0, N = 0, K = 0;
    int act = MOE_ACT_NONE;
    void* stream = nullptr;
    bool read_all(PyObject* px, PyObject* pw, PyObject* py, PyObject* pb, PyObject* pact, PyObject* pr, PyObject* pstatus,
                  PyObject* pstream, Call& f) {
        if (!matrix(px, x, -1, 0, f, "x") || !matrix(pw, w, -1, 0, f, "w")) return false;
        T = x.shape[0], K = x.shape[1], N = w.shape[0];
        if (w.shape[1] != K || w.type != x.type) return refuse(f, "w", "is not [N, K] of x's type");
        if (!matrix(py, y, T, N, f, "y")) return false;
        if (given(pb) && !vector(pb, bias, N, -1, f, "bias")) return false;
        if (given(pact)) {
            act = -1;
            for (int i = 0; i < 4; ++i)
                if (pact == g_acts[i] || (PyUnicode_Check(pact) && PyUnicode_Compare(pact, g_acts[i]) == 0)) act = i;
            if (act < 0) return refuse(f, "act", "is not none, relu, silu or gelu");
        }
        if (given(pr)) {
            if (!matrix(pr, residual, T, N, f, "residual")) return false;
            if (residual.type != y.type) return refuse(f, "residual", "has another type than y");
        }
        if (given(pstatus) && !vector(pstatus, status, 1, kI32, f, "status")) return false;
        if (!stream_of(pstream, f, stream)) return false;
        return (T <= INT32_MAX && N <= INT32_MAX && K <= INT32_MAX) || refuse(f, "x or w", "is too large");
    }
};

PyObject* n_linear[10];
PyObject* py_linear(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    Call f{"moe_linear"};
    PyObject* v[10];  // x, w, y, bias, act, residual, x_scale, w_scale, status, stream
    if (!arguments(args, n, kw, f.name, n_linear, 3, v)) return nullptr;
    Product p;
    Tensor xs, ws;
    if (!p.read_all(v[0], v[1], v[2], v[3], v[4], v[5], v[8], v[9], f)) return nullptr;
    if (given(v[6]) && !vector(v[6], xs, p.T, kF32, f, "x_scale")) return nullptr;
    if (given(v[7]) && !vector(v[7], ws, p.N, kF32, f, "w_scale")) return nullptr;
    return finish(f_linear(p.x.ptr, p.x.stride[0], p.w.ptr, p.w.stride[0], p.x.type, (int)p.T, (int)p.N, (int)p.K,
                           static_cast<float*>(xs.ptr), static_cast<float*>(ws.ptr), p.bias.ptr, p.bias.type, p.act,
                           p.residual.ptr, p.residual.stride[0], p.y.ptr, p.y.type, p.y.stride[0],
                           static_cast<int*>(p.status.ptr), p.stream),
                  f.name);
}

PyObject* n_linear_blocks[10];
PyObject* py_linear_blocks(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    Call f{"moe_linear_blocks"};
    PyObject* v[10];  // x, w, y, x_scale, w_scale, bias, act, residual, status, stream
    if (!arguments(args, n, kw, f.name, n_linear_blocks, 5, v)) return nullptr;
    Product p;
    Tensor xs, ws;
    if (!p.read_all(v[0], v[1], v[2], v[5], v[6], v[7], v[8], v[9], f)) return nullptr;
    if (p.x.type != kE4m3) return refuse(f, "x", "has a type that the call does not take"), nullptr;
    const int64_t G = (p.K + 127) / 128;
    if (!scales(v[3], xs, p.T, G, f, "x_scale") || !scales(v[4], ws, (p.N + 127) / 128, G, f, "w_scale")) return nullptr;
    return finish(f_linear_blocks(p.x.ptr, p.x.stride[0], p.w.ptr, p.w.stride[0], (int)p.T, (int)p.N, (int)p.K,
                                  static_cast<float*>(xs.ptr), xs.stride[0], static_cast<float*>(ws.ptr), ws.stride[0],
                                  p.bias.ptr, p.bias.type, p.act, p.residual.ptr, p.residual.stride[0], p.y.ptr, p.y.type,
                                  p.y.stride[0], static_cast<int*>(p.status.ptr), p.stream),
                  f.name);
}

// bind(MoeError, raw_stream, current_device, (six dtypes), (the first addresses, in the order below))
PyObject* py_bind(PyObject*, PyObject* args) {
    PyObject *error, *raw, *current, *types, *addr;
    if (!PyArg_ParseTuple(args, "OOOO!O!", &error, &raw, &current, &PyTuple_Type, &types, &PyTuple_Type, &addr))
        return nullptr;
    constexpr int kCalls = 7;
    const Py_ssize_t calls = PyTuple_GET_SIZE(addr);
    if (PyTuple_GET_SIZE(types) != kTypes || calls > kCalls) {
        PyErr_SetString(PyExc_ValueError, "six types and at most seven addresses");
        return nullptr;
    }
    void* p[kCalls];
    for (Py_ssize_t i = 0; i < calls; ++i) p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(addr, i));
    if (PyErr_Occurred()) return nullptr;
    g_error = Py_NewRef(error);
    g_raw_stream = Py_NewRef(raw);
    g_current = Py_NewRef(current);
    for (int i = 0; i < kTypes; ++i) g_types[i] = Py_NewRef(PyTuple_GET_ITEM(types, i));
    auto take = [&](int i, auto& f) {  // those not given stay as they were
        if (i < calls) f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(p[i]);
    };
    take(0, f_norm), take(1, f_append), take(2, f_attend), take(3, f_linear);
    take(4, f_quant), take(5, f_append_axes), take(6, f_linear_blocks);
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL | METH_KEYWORDS

PyMethodDef methods[] = {
    {"bind", py_bind, METH_VARARGS, "What the entry points call and raise."},
    {"moe_add_rms_norm", FAST(py_norm),
     "moe_add_rms_norm(x, weight, y, residual=None, sum_out=None, scale=None, eps=1e-6, stream=None)\n--\n\n"
     "s = x + residual; sum_out = s; y = s * rsqrt(mean(s^2) + eps) * weight, row by row.\n\n"
     "x [T, H]; residual and sum_out [T, H] of one type (each may be None); weight [H] or\n"
     "None; y [T, H].  A float8_e4m3fn y holds y / scale[t], scale [T] fp32 being the\n"
     "row's largest |y| / 448.  sum_out may be residual or x; y may be x."},
    {"moe_kv_append", FAST(py_append),
     "moe_kv_append(kv, q, k, v, positions, slots, cos_sin, q_out, interleaved=False, stream=None, axes=None)\n--\n\n"
     "Rotates q and k by position, writes q to q_out and k, v to their cache slots.\n\n"
     "q, q_out [T, q_heads, head_dim]; k, v [T, kv_heads, head_dim], strided views of a\n"
     "fused projection's rows among them; positions int32 [T]; slots int64 [T] (page *\n"
     "page_size + entry, negative: not appended); cos_sin fp32 [positions, rot_dim]\n"
     "(cosines, then sines), or None for no rotation.  interleaved pairs (2i, 2i + 1)\n"
     "instead of (i, i + rot_dim / 2).  q_out may be q.\n\n"
     "axes (bytes or a sequence of rot_dim / 2 small integers): pair i is turned by\n"
     "positions[axes[i]], positions being int32 [n_axes, T], at most four axes.  A cache\n"
     "with scales of blocks: the tokens that share a block follow one another, with\n"
     "none between them that goes elsewhere or nowhere (else kv.status() tells)."},
    {"moe_quant_e4m3", FAST(py_quant),
     "moe_quant_e4m3(x, y, scale, stream=None)\n--\n\n"
     "y = x / scale in float8_e4m3fn, scale the largest |x| / 448 of each 128 elements.\n\n"
     "x [T, K] bfloat16, float16 or float32; y [T, K] float8_e4m3fn; scale fp32\n"
     "[T, ceil(K / 128)].  None of the three shares memory with another."},
    {"moe_kv_attend", FAST(py_attend),
     "moe_kv_attend(kv, q, page_table, lengths, out, scale=None, window=0, lse=None, stream=None)\n--\n\n"
     "Attention of one query token per sequence over the cache.\n\n"
     "q, out [B, q_heads, head_dim] bfloat16 or float16, not the same memory; page_table int32 [B, max_pages]\n"
     "(an expanded single row fits); lengths int32 [B]; scale defaults to\n"
     "head_dim ** -0.5; window: only the last `window` tokens count (0: all); lse fp32\n"
     "[B, q_heads] receives the log of the softmax sums."},
    {"moe_linear", FAST(py_linear),
     "moe_linear(x, w, y, bias=None, act='none', residual=None, x_scale=None, w_scale=None, status=None, "
     "stream=None)\n--\n\n"
     "y = act(x w^T [* x_scale[t] * w_scale[n]] + bias) + residual.\n\n"
     "x [T, K] and w [N, K] of one type: bfloat16, float16, or float8_e4m3fn with\n"
     "x_scale fp32 [T] and w_scale fp32 [N]; y [T, N] bfloat16, float16 or float32;\n"
     "bias [N]; residual [T, N] of y's type (may be y); act 'none', 'relu', 'silu' or\n"
     "'gelu' (exact); status int32 [1], set to MOE_ERR_TIMEOUT if a device wait ran out."},
    {"moe_linear_blocks", FAST(py_linear_blocks),
     "moe_linear_blocks(x, w, y, x_scale, w_scale, bias=None, act='none', residual=None, status=None, "
     "stream=None)\n--\n\n"
     "y = act(sum over blocks g of 128 elements of K of x_scale[t, g] * w_scale[n // 128, g] *\n"
     "(x w^T of block g) + bias) + residual.\n\n"
     "x [T, K] and w [N, K] float8_e4m3fn; x_scale fp32 [T, ceil(K / 128)]; w_scale fp32\n"
     "[ceil(N / 128), ceil(K / 128)]; the rest as moe_linear."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_decoder_ops", "Entry points of the decoder-layer operators.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

template <int N>
bool intern(PyObject* (&out)[N], const char* const (&names)[N]) {
    for (int i = 0; i < N; ++i)
        if (!(out[i] = PyUnicode_InternFromString(names[i]))) return false;
    return true;
}

}  // namespace

PyMODINIT_FUNC PyInit__decoder_ops() {
    PyObject* attr[8];
    if (!intern(attr, {"dtype", "shape", "stride", "data_ptr", "get_device", "device_index", "cuda_stream", "_call"}) ||
        !intern(n_norm, {"x", "weight", "y", "residual", "sum_out", "scale", "eps", "stream"}) ||
        !intern(n_append, {"kv", "q", "k", "v", "positions", "slots", "cos_sin", "q_out", "interleaved", "stream",
                           "axes"}) ||
        !intern(n_quant, {"x", "y", "scale", "stream"}) ||
        !intern(n_linear_blocks,
                {"x", "w", "y", "x_scale", "w_scale", "bias", "act", "residual", "status", "stream"}) ||
        !intern(n_attend, {"kv", "q", "page_table", "lengths", "out", "scale", "window", "lse", "stream"}) ||
        !intern(n_linear, {"x", "w", "y", "bias", "act", "residual", "x_scale", "w_scale", "status", "stream"}) ||
        !intern(g_acts, {"none", "relu", "silu", "gelu"}))
        return nullptr;
    s_dtype = attr[0], s_shape = attr[1], s_stride = attr[2], s_data_ptr = attr[3];
    s_get_device = attr[4], s_device_index = attr[5], s_cuda_stream = attr[6], s_call = attr[7];
    return PyModule_Create(&module);
}
