// q4_calls.cpp -- the Python side of the 4-bit cache's calls that are made once
// per layer and token: argument marshalling only, for binding.py.
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
#include <vector>

namespace {

PyObject *g_data_ptr = nullptr, *g_cuda_stream = nullptr;  // attribute names
PyObject *g_current_stream = nullptr;                      // callable: torch's current stream as a handle

using Fn = void (*)();
enum { kAppend, kRead, kPrefill, kDecode, kDecodeDevice, kCount };
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

PyObject *read(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return ranged<2>("read", a, n, [](void *c, int l, int b, const int32_t *s, const int32_t *t, void **p, void *st) {
        using F = int (*)(void *, int, int, const int32_t *, const int32_t *, void *, void *, void *);
        return reinterpret_cast<F>(g_fn[kRead])(c, l, b, s, t, p[0], p[1], st);
    });
}

PyObject *prefill(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return ranged<6>("prefill", a, n, [](void *c, int l, int b, const int32_t *s, const int32_t *t, void **p, void *st) {
        using F = int (*)(void *, int, int, const int32_t *, const int32_t *, void *, void *, void *, void *, void *,
                          void *, void *);
        return reinterpret_cast<F>(g_fn[kPrefill])(c, l, b, s, t, p[0], p[1], p[2], p[3], p[4], p[5], st);
    });
}

using Step = int (*)(void *, int, int, const int32_t *, void *, void *, void *, void *, void *, void *, void *, void *,
                     void *);

// (cache, layer, positions, 8 pointers, stream)
PyObject *decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
    void *cache, *p[8], *s;
    int layer;
    Ints pos;
    if (!wants("decode", n, 12) || !pointer(a[0], cache) || !small_int(a[1], layer) || !pos.take(a[2])) return nullptr;
    for (int i = 0; i < 8; ++i)
        if (!pointer(a[3 + i], p[i])) return nullptr;
    if (!stream(a[11], s)) return nullptr;
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = reinterpret_cast<Step>(g_fn[kDecode])(cache, layer, pos.size(), pos.data(), p[0], p[1], p[2], p[3], p[4], p[5],
                                               p[6], p[7], s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

// (cache, layer, batch, 9 pointers, stream)
PyObject *decode_device(PyObject *, PyObject *const *a, Py_ssize_t n) {
    void *cache, *p[9], *s;
    int layer, batch;
    if (!wants("decode_device", n, 13) || !pointer(a[0], cache) || !small_int(a[1], layer) || !small_int(a[2], batch))
        return nullptr;
    for (int i = 0; i < 9; ++i)
        if (!pointer(a[3 + i], p[i])) return nullptr;
    if (!stream(a[12], s)) return nullptr;
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = reinterpret_cast<Step>(g_fn[kDecodeDevice])(cache, layer, batch, static_cast<const int32_t *>(p[0]), p[1], p[2],
                                                     p[3], p[4], p[5], p[6], p[7], p[8], s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

// (addresses of append, read, prefill, decode, decode_device; current-stream callable)
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
PyMethodDef g_methods[] = {QA_FAST(append), QA_FAST(read),          QA_FAST(prefill),
                           QA_FAST(decode), QA_FAST(decode_device), QA_FAST(bind),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_q4calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__q4calls() {
    g_data_ptr = PyUnicode_InternFromString("data_ptr");
    g_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    if (!g_data_ptr || !g_cuda_stream) return nullptr;
    return PyModule_Create(&g_module);
}
