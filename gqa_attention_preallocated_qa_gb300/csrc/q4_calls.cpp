// q4_calls.cpp -- the Python side of the 4-bit and 8-bit caches' calls that are made
// once per layer and token: argument marshalling only, for binding.py.
//
// A decode step of a short cache takes 2.5 us on the GPU, and a call through
// ctypes with its conversions took the host 2.2 us beside the launch itself.
// Here tensors (anything with data_ptr()), addresses and None become pointers,
// and sequences of ints or int32 buffers become int32 arrays, without a Python
// object in between.  binding.py hands over the addresses of the library's
// functions, so this module links against nothing.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>
#include <type_traits>
#include <vector>

namespace {

PyObject *g_data_ptr = nullptr, *g_cuda_stream = nullptr;  // attribute names
PyObject *g_current_stream = nullptr;                      // callable: torch's current stream as a handle

using Fn = void (*)();
enum {
    kAppend, kRead, kPrefill, kDecode, kDecodeDevice,
    kQ8Append, kQ8Read, kQ8Prefill, kQ8Decode, kQ8DecodeDevice, kQ8Sparse, kQ8SparseDevice,
    kCount
};
Fn g_fn[kCount] = {};

// A device pointer from a tensor, an address or None.
bool pointer(PyObject *x, void *&p) {
    if (x == Py_None) {
        p = nullptr;
        return true;
    }
    PyObject *v = nullptr;
    if (!PyLong_Check(x)) {
        v = PyObject_CallMethodNoArgs(x, g_data_ptr);
        if (!v) return false;
        x = v;
    }
    p = PyLong_AsVoidPtr(x);
    Py_XDECREF(v);
    return !(p == nullptr && PyErr_Occurred());
}

// A stream handle from a handle, a torch stream or None (the current one).
bool stream(PyObject *x, void *&p) {
    PyObject *v = nullptr;
    if (x == Py_None) {
        v = PyObject_CallNoArgs(g_current_stream);
        if (!v) return false;
        x = v;
        if (x == Py_None) {  // no device: the legacy stream
            Py_DECREF(v);
            p = nullptr;
            return true;
        }
    } else if (!PyLong_Check(x)) {
        v = PyObject_GetAttr(x, g_cuda_stream);
        if (!v) return false;
        x = v;
    }
    p = PyLong_AsVoidPtr(x);
    Py_XDECREF(v);
    return !(p == nullptr && PyErr_Occurred());
}

bool small_int(PyObject *x, int &v) {
    const long n = PyLong_AsLong(x);
    if (n == -1 && PyErr_Occurred()) return false;
    if (n < INT32_MIN || n > INT32_MAX) {
        PyErr_SetString(PyExc_OverflowError, "value does not fit 32 bits");
        return false;
    }
    v = static_cast<int>(n);
    return true;
}

// int32 values of a sequence of ints or of a contiguous buffer of them.
class Ints {
  public:
    bool take(PyObject *x) {
        try {
            return taken(x);
        } catch (...) {  // a sequence that does not fit memory
            PyErr_NoMemory();
            return false;
        }
    }
    const int32_t *data() const { return v_.data(); }
    int size() const { return static_cast<int>(v_.size()); }

  private:
    bool taken(PyObject *x) {
        if (PyList_Check(x) || PyTuple_Check(x)) return items(x);
        if (PyObject_CheckBuffer(x)) {
            Py_buffer b;
            if (PyObject_GetBuffer(x, &b, PyBUF_CONTIG_RO | PyBUF_FORMAT) == 0) {
                const char *f = b.format ? b.format : "B";
                const char kind = f[0] == '<' || f[0] == '=' || f[0] == '@' ? f[1] : f[0];
                const bool ok = b.itemsize == 4 && (kind == 'i' || kind == 'l');
                if (ok) {
                    const int32_t *v = static_cast<const int32_t *>(b.buf);
                    v_.assign(v, v + b.len / 4);
                }
                PyBuffer_Release(&b);
                if (ok) return true;
            } else {
                PyErr_Clear();
            }
        }
        PyObject *s = PySequence_Fast(x, "positions are a sequence of ints");
        if (!s) return false;
        bool ok = false;
        try {
            ok = items(s);
        } catch (...) {
            PyErr_NoMemory();
        }
        Py_DECREF(s);
        return ok;
    }
    bool items(PyObject *s) {
        const Py_ssize_t n = PySequence_Fast_GET_SIZE(s);
        v_.resize(static_cast<size_t>(n));
        for (Py_ssize_t i = 0; i < n; ++i)
            if (!small_int(PySequence_Fast_GET_ITEM(s, i), v_[i])) return false;
        return true;
    }
    std::vector<int32_t> v_;
};

bool wants(const char *what, Py_ssize_t got, Py_ssize_t n) {
    if (got == n) return true;
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments (got %zd)", what, n, got);
    return false;
}

// (cache, layer, start, ntok, N pointers, stream)
template <int N, class Call>
PyObject *ranged(const char *what, PyObject *const *a, Py_ssize_t n, Call &&call) {
    void *cache, *p[N], *s;
    int layer;
    Ints start, ntok;
    if (!wants(what, n, N + 5) || !pointer(a[0], cache) || !small_int(a[1], layer) || !start.take(a[2]) ||
        !ntok.take(a[3]))
        return nullptr;
    if (start.size() != ntok.size()) {
        PyErr_SetString(PyExc_ValueError, "start and ntok need one entry per sequence");
        return nullptr;
    }
    for (int i = 0; i < N; ++i)
        if (!pointer(a[4 + i], p[i])) return nullptr;
    if (!stream(a[4 + N], s)) return nullptr;
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = call(cache, layer, start.size(), start.data(), ntok.data(), p, s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return ranged<4>("append", a, n, [](void *c, int l, int b, const int32_t *s, const int32_t *t, void **p, void *st) {
        using F = int (*)(void *, int, int, const int32_t *, const int32_t *, void *, void *, void *, void *, void *);
        return reinterpret_cast<F>(g_fn[kAppend])(c, l, b, s, t, p[0], p[1], p[2], p[3], st);
    });
}

// K and V rows: a read, or the 8-bit cache's append.
template <int kFn>
PyObject *rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return ranged<2>(kFn == kQ8Append ? "append" : "read", a, n,
                     [](void *c, int l, int b, const int32_t *s, const int32_t *t, void **p, void *st) {
        using F = int (*)(void *, int, int, const int32_t *, const int32_t *, void *, void *, void *);
        return reinterpret_cast<F>(g_fn[kFn])(c, l, b, s, t, p[0], p[1], st);
    });
}
constexpr auto read = rows<kRead>;
constexpr auto q8_read = rows<kQ8Read>;
constexpr auto q8_append = rows<kQ8Append>;

template <int kFn>
PyObject *prefills(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return ranged<6>("prefill", a, n, [](void *c, int l, int b, const int32_t *s, const int32_t *t, void **p, void *st) {
        using F = int (*)(void *, int, int, const int32_t *, const int32_t *, void *, void *, void *, void *, void *,
                          void *, void *);
        return reinterpret_cast<F>(g_fn[kFn])(c, l, b, s, t, p[0], p[1], p[2], p[3], p[4], p[5], st);
    });
}
constexpr auto prefill = prefills<kPrefill>;
constexpr auto q8_prefill = prefills<kQ8Prefill>;

using Step = int (*)(void *, int, int, const int32_t *, void *, void *, void *, void *, void *, void *, void *, void *,
                     void *);
using SparseStep = int (*)(void *, int, int, const int32_t *, int, void *, void *, void *, void *, void *, void *, void *,
                           void *, void *, void *);

int step(int fn, void *cache, int layer, int batch, const int32_t *pos, int, void **p, void *s, Step) {
    return reinterpret_cast<Step>(g_fn[fn])(cache, layer, batch, pos, p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], s);
}
int step(int fn, void *cache, int layer, int batch, const int32_t *pos, int n_blocks, void **p, void *s, SparseStep) {
    return reinterpret_cast<SparseStep>(g_fn[fn])(cache, layer, batch, pos, n_blocks, p[0], p[1], p[2], p[3], p[4], p[5],
                                                  p[6], p[7], p[8], s);
}

// (cache, layer, positions, [n_blocks,] 8 or 9 pointers, stream)
template <int kFn, class F>
PyObject *steps(PyObject *, PyObject *const *a, Py_ssize_t n) {
    constexpr bool sparse = std::is_same<F, SparseStep>::value;
    constexpr int N = sparse ? 9 : 8, P = sparse ? 4 : 3;
    void *cache, *p[N], *s;
    int layer, n_blocks = 0;
    Ints pos;
    if (!wants(sparse ? "sparse" : "decode", n, P + N + 1) || !pointer(a[0], cache) || !small_int(a[1], layer) ||
        !pos.take(a[2]) || (sparse && !small_int(a[3], n_blocks)))
        return nullptr;
    for (int i = 0; i < N; ++i)
        if (!pointer(a[P + i], p[i])) return nullptr;
    if (!stream(a[P + N], s)) return nullptr;
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = step(kFn, cache, layer, pos.size(), pos.data(), n_blocks, p, s, F());
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}
constexpr auto decode = steps<kDecode, Step>;
constexpr auto q8_decode = steps<kQ8Decode, Step>;
constexpr auto q8_sparse = steps<kQ8Sparse, SparseStep>;

// (cache, layer, batch, positions, [n_blocks,] 8 or 9 pointers, stream)
template <int kFn, class F>
PyObject *device_steps(PyObject *, PyObject *const *a, Py_ssize_t n) {
    constexpr bool sparse = std::is_same<F, SparseStep>::value;
    constexpr int N = sparse ? 9 : 8, P = sparse ? 5 : 4;
    void *cache, *pos, *p[N], *s;
    int layer, batch, n_blocks = 0;
    if (!wants(sparse ? "sparse_device" : "decode_device", n, P + N + 1) || !pointer(a[0], cache) ||
        !small_int(a[1], layer) || !small_int(a[2], batch) || !pointer(a[3], pos) ||
        (sparse && !small_int(a[4], n_blocks)))
        return nullptr;
    for (int i = 0; i < N; ++i)
        if (!pointer(a[P + i], p[i])) return nullptr;
    if (!stream(a[P + N], s)) return nullptr;
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = step(kFn, cache, layer, batch, static_cast<const int32_t *>(pos), n_blocks, p, s, F());
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}
constexpr auto decode_device = device_steps<kDecodeDevice, Step>;
constexpr auto q8_decode_device = device_steps<kQ8DecodeDevice, Step>;
constexpr auto q8_sparse_device = device_steps<kQ8SparseDevice, SparseStep>;

// (addresses of the library's functions in the order of the enum; current-stream callable)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!wants("bind", n, kCount + 1)) return nullptr;
    for (int i = 0; i < kCount; ++i) {
        void *p;
        if (!pointer(a[i], p)) return nullptr;
        g_fn[i] = reinterpret_cast<Fn>(p);
    }
    Py_INCREF(a[kCount]);
    Py_XSETREF(g_current_stream, a[kCount]);
    Py_RETURN_NONE;
}

#define QA_FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {QA_FAST(append),    QA_FAST(read),             QA_FAST(prefill),
                           QA_FAST(decode),    QA_FAST(decode_device),    QA_FAST(q8_append),
                           QA_FAST(q8_read),   QA_FAST(q8_prefill),       QA_FAST(q8_decode),
                           QA_FAST(q8_sparse), QA_FAST(q8_decode_device), QA_FAST(q8_sparse_device),
                           QA_FAST(bind),      {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_q4calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__q4calls() {
    g_data_ptr = PyUnicode_InternFromString("data_ptr");
    g_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    if (!g_data_ptr || !g_cuda_stream) return nullptr;
    return PyModule_Create(&g_module);
}
