// Host half of the Python binding: the checks of a tensor argument and the
// calls of the C entry points, without the interpreter's cost for each of
// their steps.  An attention call checks 12 tensors and passes 30 arguments:
// 0.75 us a tensor and 2.3 us for the call from Python, 0.1 and 0.5 us here.
// Calls that end in a few microseconds of GPU work are bound by this time.
//
//   need(t, name, dtypes, shape=None)   nothing, if t is a contiguous GPU
//       tensor of one of the dtypes and of this shape (None: any); otherwise
//       whatever the function given to explain() raises for the same arguments
//   cache(t, dtypes, heads, d)   pages, page size and stride of a paged cache
//   rows(t, dtypes, tail)   rows, their stride and the sizes and strides of the
//       last `tail` dimensions of a GPU tensor whose leading ones are one
//   on_device(index, ...)   whether all tensors given are on that GPU
//   gdn_*(arguments of the C entry point)   its status; a pointer is an int,
//       None or a tensor
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gdn_tree.h"

namespace {

PyObject *g_explain = nullptr;

// f(), or `failed` with the Python exception set that its C++ exception stands
// for.  Sizes, strides and addresses raise for tensors whose metadata is not
// plain (symbolic sizes, subclasses that answer in Python, no storage), and no
// C++ exception may cross the interpreter's frames.
template <typename R, typename F>
R guarded(R failed, F f) {
    try {
        return f();
    } catch (python_error &e) {
        if (!PyErr_Occurred()) e.restore();
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "a C++ exception");
    }
    return failed;
}

bool known_dtype(const at::Tensor &x, PyObject *dtypes) {
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(dtypes); ++i) {
        PyObject *d = PyTuple_GET_ITEM(dtypes, i);
        if (THPDtype_Check(d) &&
            reinterpret_cast<THPDtype *>(d)->scalar_type == x.scalar_type())
            return true;
    }
    return false;
}

bool plain(PyObject *t, PyObject *dtypes, PyObject *shape) {
    if (!THPVariable_Check(t) || !PyTuple_Check(dtypes)) return false;
    const at::Tensor &x = THPVariable_Unpack(t);
    if (!x.is_cuda() || !x.is_contiguous() || !known_dtype(x, dtypes)) return false;
    if (shape == Py_None) return true;
    if (!PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != x.dim()) return false;
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(shape); ++i) {
        const long long n = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
        if (n == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            return false;
        }
        if (n != x.size(i)) return false;
    }
    return true;
}

// false as well where the tensor's metadata raises: the function given to
// explain() asks the same of it, and lets its exception through
bool suits(PyObject *t, PyObject *dtypes, PyObject *shape) {
    const bool ok = guarded(false, [&] { return plain(t, dtypes, shape); });
    if (!ok) PyErr_Clear();
    return ok;
}

// cache(t, dtypes, heads, d): (pages, tokens a page, elements between pages)
// of a cache [pages][heads][page][d] on the GPU whose pages are contiguous (the
// stride of a dimension of one says nothing),
// or None (also where its metadata raises, as above)
PyObject *cache(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 4) {
        PyErr_SetString(PyExc_TypeError, "cache(t, dtypes, heads, d)");
        return nullptr;
    }
    const long long heads = PyLong_AsLongLong(args[2]), d = PyLong_AsLongLong(args[3]);
    if (PyErr_Occurred()) return nullptr;
    if (!THPVariable_Check(args[0]) || !PyTuple_Check(args[1])) Py_RETURN_NONE;
    const at::Tensor &x = THPVariable_Unpack(args[0]);
    long long pages = 0, page = 0, stride = 0;
    const bool ok = guarded(false, [&] {
        if (!x.is_cuda() || !known_dtype(x, args[1]) || x.dim() != 4 || x.size(1) != heads ||
            x.size(3) != d)
            return false;
        const long long dense[4] = {0, x.size(2) * d, d, 1};
        for (int i = 1; i < 4; ++i)
            if (x.size(i) != 1 && x.stride(i) != dense[i]) return false;
        pages = x.size(0), page = x.size(2);
        stride = pages > 1 ? (long long)x.stride(0) : heads * page * d;
        return true;
    });
    if (ok) return Py_BuildValue("LLL", pages, page, stride);
    PyErr_Clear();
    Py_RETURN_NONE;
}

// rows(t, dtypes, tail): of a tensor [...][heads][d] (tail 2) or [...][d] (tail 1)
// on the GPU whose d elements are adjacent and whose leading dimensions can be
// walked with one stride, the numbers (rows, row stride, heads, head stride, d)
// or (rows, row stride, d); None otherwise (also where its metadata raises).
// The stride of a single row or head says nothing: a dense one is given.
PyObject *rows(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 3) {
        PyErr_SetString(PyExc_TypeError, "rows(t, dtypes, tail)");
        return nullptr;
    }
    const long long tail = PyLong_AsLongLong(args[2]);
    if (PyErr_Occurred()) return nullptr;
    if (!THPVariable_Check(args[0]) || !PyTuple_Check(args[1]) || tail < 1 || tail > 2)
        Py_RETURN_NONE;
    const at::Tensor &x = THPVariable_Unpack(args[0]);
    long long count = 1, stride = 0, heads = 1, head = 0, d = 0;
    const bool ok = guarded(false, [&] {
        if (!x.is_cuda() || !known_dtype(x, args[1]) || x.dim() < tail) return false;
        int64_t i = x.dim() - 1;
        d = x.size(i);
        if (d > 1 && x.stride(i) != 1) return false;
        if (tail == 2) {
            --i;
            heads = x.size(i);
            head = heads > 1 ? (long long)x.stride(i) : d;
        }
        stride = tail == 2 ? heads * head : d;
        bool first = true;
        for (--i; i >= 0; --i) {
            const long long size = x.size(i);
            if (size == 1) continue;
            if (first) stride = x.stride(i);
            else if (x.stride(i) != stride * count) return false;
            first = false;
            count *= size;
        }
        return true;
    });
    if (!ok) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    return tail == 2 ? Py_BuildValue("LLLLL", count, stride, heads, head, d)
                     : Py_BuildValue("LLL", count, stride, d);
}

// on_device(index, t, ...): whether every argument that is a tensor is on it
PyObject *on_device(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n < 1) {
        PyErr_SetString(PyExc_TypeError, "on_device(index, ...)");
        return nullptr;
    }
    const long long index = PyLong_AsLongLong(args[0]);
    if (PyErr_Occurred()) return nullptr;
    const bool ok = guarded(false, [&] {
        for (Py_ssize_t i = 1; i < n; ++i)
            if (THPVariable_Check(args[i]) && THPVariable_Unpack(args[i]).get_device() != index)
                return false;
        return true;
    });
    if (PyErr_Occurred()) return nullptr;
    return PyBool_FromLong(ok);
}

PyObject *need(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n < 3 || n > 4) {
        PyErr_SetString(PyExc_TypeError, "need(t, name, dtypes, shape=None)");
        return nullptr;
    }
    if (suits(args[0], args[2], n == 4 ? args[3] : Py_None)) Py_RETURN_NONE;
    if (!g_explain) {
        PyErr_SetString(PyExc_RuntimeError, "explain() has not been called");
        return nullptr;
    }
    return PyObject_Vectorcall(g_explain, args, (size_t)n, nullptr);
}

PyObject *explain(PyObject *, PyObject *f) {
    Py_INCREF(f);
    Py_XSETREF(g_explain, f);
    Py_RETURN_NONE;
}

// one argument of an entry point; false with an exception set
template <typename T>
bool read(PyObject *o, T &x) {
    if constexpr (std::is_pointer_v<T>) {
        void *p = nullptr;
        if (o == Py_None) p = nullptr;
        else if (THPVariable_Check(o)) p = THPVariable_Unpack(o).data_ptr();
        else p = PyLong_AsVoidPtr(o);
        x = static_cast<T>(p);
    } else if constexpr (std::is_same_v<T, float>) {
        x = static_cast<float>(PyFloat_AsDouble(o));
    } else {
        const long long v = PyLong_AsLongLong(o);
        if (sizeof(T) == 4 && (v < INT32_MIN || v > INT32_MAX) && !PyErr_Occurred()) {
            PyErr_SetString(PyExc_OverflowError, "argument does not fit 32 bits");
            return false;
        }
        x = static_cast<T>(v);
    }
    return !PyErr_Occurred();
}

template <typename R, typename... A, size_t... I>
PyObject *call(R (*fn)(A...), PyObject *const *args, std::index_sequence<I...>) {
    std::tuple<A...> v;
    if (!(... && read(args[I], std::get<I>(v)))) return nullptr;
    R r;
    Py_BEGIN_ALLOW_THREADS
    r = fn(std::get<I>(v)...);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(static_cast<long>(r));
}

template <auto F>
struct Entry;
template <typename R, typename... A, R (*F)(A...)>
struct Entry<F> {
    static PyObject *run(PyObject *, PyObject *const *args, Py_ssize_t n) {
        if (n != (Py_ssize_t)sizeof...(A)) {
            PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", n,
                         (Py_ssize_t)sizeof...(A));
            return nullptr;
        }
        return guarded((PyObject *)nullptr,
                       [&] { return call(F, args, std::index_sequence_for<A...>{}); });
    }
};

#define ENTRY(name) \
    {#name, (PyCFunction)(void (*)(void))Entry<&name>::run, METH_FASTCALL, nullptr}

PyMethodDef g_methods[] = {
    {"need", (PyCFunction)(void (*)(void))need, METH_FASTCALL, nullptr},
    {"cache", (PyCFunction)(void (*)(void))cache, METH_FASTCALL, nullptr},
    {"rows", (PyCFunction)(void (*)(void))rows, METH_FASTCALL, nullptr},
    {"on_device", (PyCFunction)(void (*)(void))on_device, METH_FASTCALL, nullptr},
    {"explain", explain, METH_O, nullptr},
    ENTRY(gdn_prefill),
    ENTRY(gdn_step),
    ENTRY(gdn_tree_attention),
    ENTRY(gdn_page_fork),
    ENTRY(gdn_page_extend),
    ENTRY(gdn_page_free),
    ENTRY(gdn_page_compact),
    ENTRY(gdn_page_copy),
    ENTRY(gdn_kv_commit),
    ENTRY(gdn_rope),
    ENTRY(gdn_qk_norm_rope),
    ENTRY(gdn_kv_append),
    ENTRY(gdn_count_prompt),
    ENTRY(gdn_count_commit),
    ENTRY(gdn_adjust_logits),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
    PyObject *m = PyModule_Create(&g_module);
    // the header that the calls above were compiled with
    if (m && PyModule_AddIntConstant(m, "ABI_VERSION", GDN_TREE_ABI_VERSION) < 0) Py_CLEAR(m);
    return m;
}
