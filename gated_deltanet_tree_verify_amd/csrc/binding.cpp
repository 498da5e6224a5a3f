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
//   heads_call, append_call, ..   checks and call of an operator in one
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

// Rows of a tensor [...][heads][d] (tail 2) or [...][d] (tail 1) whose d elements
// are adjacent and whose leading dimensions can be walked with one stride.  The
// stride of a single row or head says nothing: a dense one is given.
struct Rows {
    int64_t count = 1, stride = 0, heads = 1, head = 0, d = 0;
};

bool walk(const at::Tensor &x, int64_t tail, Rows &r) {
    if (x.dim() < tail) return false;
    r = Rows{};
    int64_t i = x.dim() - 1;
    r.d = x.size(i);
    if (r.d > 1 && x.stride(i) != 1) return false;
    if (tail == 2) {
        --i;
        r.heads = x.size(i);
        r.head = r.heads > 1 ? x.stride(i) : r.d;
    }
    r.stride = tail == 2 ? r.heads * r.head : r.d;
    bool first = true;
    for (--i; i >= 0; --i) {
        const int64_t size = x.size(i);
        if (size == 1) continue;
        if (size == 0) {             // no rows: their strides say nothing
            r.count = 0;
            return true;
        }
        if (first) r.stride = x.stride(i);
        else if (x.stride(i) != r.stride * r.count) return false;
        first = false;
        r.count *= size;
    }
    return true;
}

// rows(t, dtypes, tail): the numbers (rows, row stride, heads, head stride, d) or
// (rows, row stride, d) of a GPU tensor that has them; None otherwise (also
// where its metadata raises)
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
    Rows r;
    const bool ok = guarded(
        false, [&] { return x.is_cuda() && known_dtype(x, args[1]) && walk(x, tail, r); });
    if (!ok) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    typedef long long L;
    return tail == 2 ? Py_BuildValue("LLLLL", (L)r.count, (L)r.stride, (L)r.heads, (L)r.head, (L)r.d)
                     : Py_BuildValue("LLL", (L)r.count, (L)r.stride, (L)r.d);
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

// ---------------------------------------------------------------------------
// Whole calls.  heads_call, append_call, count_*_call and logits_call check the
// arguments of an operator and call its entry point: 0.7 to 1.2 us instead of 2
// to 6 for the same steps in Python.  They know the usual case alone, outputs
// given and everything in order: for anything else they return None, having
// done nothing, and the Python function goes through its own checks, which say
// what is wrong, or do what is left to do.
// ---------------------------------------------------------------------------
PyObject *g_get_device = nullptr, *g_get_stream = nullptr;

// streams(get_device, get_stream): torch's functions for the current ones
PyObject *streams(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 2) {
        PyErr_SetString(PyExc_TypeError, "streams(get_device, get_stream)");
        return nullptr;
    }
    Py_INCREF(args[0]);
    Py_INCREF(args[1]);
    Py_XSETREF(g_get_device, args[0]);
    Py_XSETREF(g_get_stream, args[1]);
    Py_RETURN_NONE;
}

// The arguments of a call, one after the other; `ok` is false from the first
// one on that is not as it should be.
class Arguments {
public:
    bool ok = true;
    int64_t device = -1;
    void *stream = nullptr;

    // the stream that the call runs on, of the current device
    void where(PyObject *o) {
        if (!g_get_device || !g_get_stream) return fail();
        PyObject *d = PyObject_CallNoArgs(g_get_device);
        if (!d) return fail();
        device = PyLong_AsLongLong(d);
        PyObject *s = nullptr;
        if (o == Py_None) s = PyObject_CallOneArg(g_get_stream, d);
        else if (PyLong_Check(o)) s = Py_NewRef(o);
        else s = PyObject_GetAttrString(o, "cuda_stream");
        Py_DECREF(d);
        if (!s) return fail();
        stream = PyLong_AsVoidPtr(s);
        Py_DECREF(s);
        if (PyErr_Occurred()) fail();
    }
    const at::Tensor *tensor(PyObject *o) {
        if (!ok || !THPVariable_Check(o)) return nothing();
        const at::Tensor &x = THPVariable_Unpack(o);
        return x.is_cuda() && x.get_device() == device ? &x : nothing();
    }
    // a contiguous tensor of a type, and of these sizes
    const at::Tensor *plain(PyObject *o, at::ScalarType t) {
        const at::Tensor *x = tensor(o);
        return x && x->scalar_type() == t && x->is_contiguous() ? x : nothing();
    }
    const at::Tensor *plain(PyObject *o, at::ScalarType t, at::IntArrayRef sizes) {
        const at::Tensor *x = plain(o, t);
        return x && x->sizes() == sizes ? x : nothing();
    }
    const at::Tensor *plain_or_none(PyObject *o, at::ScalarType t, at::IntArrayRef sizes) {
        return o == Py_None ? nullptr : plain(o, t, sizes);
    }
    // rows of a tensor of a type
    const at::Tensor *walked(PyObject *o, at::ScalarType t, int64_t tail, Rows &r) {
        const at::Tensor *x = tensor(o);
        return x && x->scalar_type() == t && walk(*x, tail, r) ? x : nothing();
    }
    long long integer(PyObject *o) {
        const long long v = PyLong_Check(o) ? PyLong_AsLongLong(o) : -1;
        if (!PyLong_Check(o) || v < 0 || PyErr_Occurred()) fail();
        return v;
    }
    float number(PyObject *o) {
        const double v = PyFloat_Check(o) || PyLong_Check(o) ? PyFloat_AsDouble(o) : 0;
        if (!(PyFloat_Check(o) || PyLong_Check(o)) || PyErr_Occurred()) fail();
        return static_cast<float>(v);
    }
    void check(bool good) {
        if (!good) fail();
    }

private:
    void fail() {
        ok = false;
        PyErr_Clear();
    }
    const at::Tensor *nothing() {
        ok = false;
        return nullptr;
    }
};

bool narrow(int64_t x) { return x >= 0 && x <= INT32_MAX; }

template <typename T = void>
T *data(const at::Tensor *x) {
    return x ? static_cast<T *>(x->data_ptr()) : nullptr;
}

bool element_type(at::ScalarType t, gdn_dtype &out) {
    if (t == at::kBFloat16) out = GDN_DTYPE_BF16;
    else if (t == at::kHalf) out = GDN_DTYPE_F16;
    else if (t == at::kFloat) out = GDN_DTYPE_F32;
    else return false;
    return true;
}

// weights [d] or [heads][d] of the heads' type or fp32; the stride of a head
const at::Tensor *norm_weight(Arguments &in, PyObject *o, at::ScalarType t, int64_t heads, int64_t d,
                              int64_t &head) {
    head = 0;
    if (o == Py_None) return nullptr;
    const at::Tensor *w = in.tensor(o);
    if (!w || (w->scalar_type() != t && w->scalar_type() != at::kFloat) || !w->is_contiguous()) {
        in.check(false);
        return nullptr;
    }
    if (w->dim() == 2) {
        head = d;
        in.check(w->size(0) == heads && w->size(1) == d);
    } else {
        in.check(w->dim() == 1 && w->size(0) == d);
    }
    return w;
}

bool same_lead(const at::Tensor &x, const at::Tensor &y) {
    if (x.dim() != y.dim()) return false;
    for (int64_t i = 0; i + 2 < x.dim(); ++i)
        if (x.size(i) != y.size(i)) return false;
    return true;
}

template <typename F>
PyObject *whole_call(PyObject *const *args, Py_ssize_t n, Py_ssize_t expected, F f) {
    if (n != expected) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", n, expected);
        return nullptr;
    }
    int status = 0;
    const bool done = guarded(false, [&] { return f(args, status); });
    if (done) return PyLong_FromLong(status);
    PyErr_Clear();
    Py_RETURN_NONE;
}

// fn(x...) while other threads may have the interpreter.  The arguments are
// formed before that: a tensor without storage raises for its address.
template <typename... P, typename... A>
int unlocked(gdn_status (*fn)(P...), A... x) {
    gdn_status status;
    Py_BEGIN_ALLOW_THREADS
    status = fn(x...);
    Py_END_ALLOW_THREADS
    return status;
}

// (norm, q, k, q_weight, k_weight, pos, base, inv_freq, eps, offset, layout,
// scale, q_out, k_out, stream); norm 0: gdn_rope
bool run_heads(PyObject *const *o, int &status) {
    Arguments in;
    in.where(o[14]);
    const long long norm = in.integer(o[0]), layout = in.integer(o[10]);
    const float eps = in.number(o[8]), offset = in.number(o[9]), scale = in.number(o[11]);
    const at::Tensor *q = in.tensor(o[1]);
    if (!q) return false;
    const at::ScalarType t = q->scalar_type();
    gdn_dtype dtype;
    Rows rq, rk, oq, ok;
    if (!element_type(t, dtype) || !walk(*q, 2, rq)) return false;
    const at::Tensor *k = o[2] == Py_None ? nullptr : in.walked(o[2], t, 2, rk), *k_out = nullptr;
    const at::Tensor *q_out = in.walked(o[12], t, 2, oq);
    if (!in.ok || q_out->sizes() != q->sizes()) return false;
    rk.heads = k ? rk.heads : 0;
    if (k) {
        k_out = in.walked(o[13], t, 2, ok);
        if (!in.ok || k_out->sizes() != k->sizes() || !same_lead(*q, *k) || rk.d != rq.d) return false;
    } else if (o[13] != Py_None) {
        return false;
    }
    const at::Tensor *f = o[7] == Py_None ? nullptr : in.plain(o[7], at::kFloat);
    if (!in.ok || (f && (f->dim() != 1 || 2 * f->size(0) > rq.d))) return false;
    const int64_t rot = f ? 2 * f->size(0) : 0;
    const at::Tensor *pos = nullptr, *base = nullptr;
    int64_t base_rows = 1;
    if (rot > 0) {
        const at::IntArrayRef lead = q->sizes().slice(0, q->dim() - 2);
        pos = in.plain(o[5], at::kInt, lead);
        base = in.plain_or_none(o[6], at::kInt, lead.slice(0, lead.empty() ? 0 : 1));
        if (!in.ok) return false;
        if (base) base_rows = rq.count / (base->numel() > 0 ? base->numel() : 1);
        if (base_rows < 1) base_rows = 1;
    } else if (norm == 0 || o[5] != Py_None || o[6] != Py_None) {
        return false;
    }
    int64_t wq_head, wk_head;
    const at::Tensor *wq = norm_weight(in, o[3], t, rq.heads, rq.d, wq_head);
    const at::Tensor *wk = norm_weight(in, o[4], t, rk.heads, rq.d, wk_head);
    if (!in.ok || (norm == 0 && (wq || wk)) ||
        (wq && wk && wq->scalar_type() != wk->scalar_type()) || !narrow(rq.count) ||
        !narrow(rq.heads) || !narrow(rk.heads) || !narrow(rq.d) || layout > 1 || norm > 2)
        return false;
    const bool wide = wq ? wq->scalar_type() == at::kFloat : wk && wk->scalar_type() == at::kFloat;
    status = unlocked(
        gdn_qk_norm_rope, data(q), rq.stride, rq.head, data(k), rk.stride, rk.head, dtype,
        static_cast<gdn_norm>(norm), eps, offset, data(wq), wq_head, data(wk), wk_head, wide ? GDN_DTYPE_F32 : dtype,
        data<int32_t>(pos), data<int32_t>(base), (int)base_rows, data<float>(f), (int)rot,
        static_cast<gdn_rope_layout>(layout), scale, data(q_out), oq.stride, oq.head, data(k_out),
        ok.stride, ok.head, (int)rq.count, (int)rq.heads, (int)rk.heads, (int)rq.d, in.stream);
    return true;
}

// pages, tokens a page and elements between pages of a cache [pages][heads][page][d]
bool cache_shape(const at::Tensor &x, int64_t heads, int64_t d, int64_t (&out)[3]) {
    if (x.dim() != 4 || x.size(1) != heads || x.size(3) != d) return false;
    const int64_t dense[4] = {0, x.size(2) * d, d, 1};
    for (int i = 1; i < 4; ++i)
        if (x.size(i) != 1 && x.stride(i) != dense[i]) return false;
    out[0] = x.size(0), out[1] = x.size(2);
    out[2] = out[0] > 1 ? x.stride(0) : heads * out[1] * d;
    return true;
}

// (k_cache, v_cache, table, dst, begin, k, v, cu, inv_freq, layout, scale, pos,
// norm, eps, offset, k_weight, q, q_weight, q_out, k_out, status, stream)
bool run_append(PyObject *const *o, int &status) {
    Arguments in;
    in.where(o[21]);
    const long long layout = in.integer(o[9]), norm = in.integer(o[12]);
    const float scale = in.number(o[10]), eps = in.number(o[13]), offset = in.number(o[14]);
    const at::Tensor *k = in.tensor(o[5]);
    if (!k) return false;
    const at::ScalarType t = k->scalar_type();
    gdn_dtype dtype;
    Rows rk, rv, rq, oq, ok;
    if (!element_type(t, dtype) || !walk(*k, 2, rk)) return false;
    const at::Tensor *v = in.walked(o[6], t, 2, rv);
    const at::Tensor *kc = in.tensor(o[0]), *vc = in.tensor(o[1]);
    int64_t page[3], other[3];
    if (!in.ok || v->sizes() != k->sizes() || kc->scalar_type() != t || vc->scalar_type() != t ||
        !cache_shape(*kc, rk.heads, rk.d, page) || !cache_shape(*vc, rk.heads, rk.d, other) ||
        page[0] != other[0] || page[1] != other[1] || page[2] != other[2])
        return false;
    const at::Tensor *table = in.plain(o[2], at::kInt);
    const at::Tensor *cu = o[7] == Py_None ? nullptr : in.plain(o[7], at::kInt);
    if (!in.ok || table->dim() != 2 || (cu && (cu->dim() != 1 || cu->size(0) < 1))) return false;
    const int64_t m = cu ? cu->size(0) - 1 : rk.count;
    const at::Tensor *dst = in.plain(o[3], at::kInt, {m}), *begin = in.plain(o[4], at::kInt, {m});
    const at::Tensor *q = nullptr, *q_out = nullptr, *k_out = nullptr;
    rq.heads = 0;
    if (o[16] != Py_None) {
        q = in.walked(o[16], t, 2, rq);
        q_out = in.walked(o[18], t, 2, oq);
        if (!in.ok || !same_lead(*q, *k) || rq.d != rk.d || q_out->sizes() != q->sizes()) return false;
    } else if (o[18] != Py_None || o[17] != Py_None) {
        return false;
    }
    if (o[19] != Py_None) {
        k_out = in.walked(o[19], t, 2, ok);
        if (!in.ok || k_out->sizes() != k->sizes()) return false;
    }
    const at::Tensor *f = o[8] == Py_None ? nullptr : in.plain(o[8], at::kFloat);
    if (!in.ok || (f && (f->dim() != 1 || 2 * f->size(0) > rk.d))) return false;
    const int64_t rot = f ? 2 * f->size(0) : 0;
    const at::Tensor *pos =
        in.plain_or_none(o[11], at::kInt, k->sizes().slice(0, k->dim() - 2));
    const at::Tensor *st = in.plain_or_none(o[20], at::kInt, {m});
    int64_t wq_head, wk_head;
    const at::Tensor *wq = norm_weight(in, o[17], t, rq.heads, rk.d, wq_head);
    const at::Tensor *wk = norm_weight(in, o[15], t, rk.heads, rk.d, wk_head);
    if (!in.ok || (pos && rot == 0) || (norm == 0 && (wq || wk)) ||
        (wq && wk && wq->scalar_type() != wk->scalar_type()) || layout > 1 || norm > 2)
        return false;
    for (int64_t x : {m, rk.count, rq.heads, rk.heads, rk.d, table->size(0), table->size(1), page[0],
                      page[1]})
        if (!narrow(x)) return false;
    const bool wide = wq ? wq->scalar_type() == at::kFloat : wk && wk->scalar_type() == at::kFloat;
    status = unlocked(
        gdn_kv_append, data(kc), data(vc), page[2], data<int32_t>(table), data<int32_t>(dst),
        data<int32_t>(begin), data<int32_t>(cu), data(q), rq.stride, rq.head, data(k), rk.stride, rk.head, data(v),
        rv.stride, rv.head, dtype, static_cast<gdn_norm>(norm), eps, offset, data(wq), wq_head,
        data(wk), wk_head, wide ? GDN_DTYPE_F32 : dtype, data<int32_t>(pos), data<float>(f), (int)rot,
        static_cast<gdn_rope_layout>(layout), scale, data(q_out), oq.stride, oq.head, data(k_out),
        ok.stride, ok.head, (int)m, (int)rk.count, (int)rq.heads, (int)rk.heads, (int)rk.d,
        (int)table->size(0), (int)table->size(1), (int)page[0], (int)page[1], data<int32_t>(st),
        in.stream);
    return true;
}

// (counts, slot, cu, tokens, status, stream)
bool run_count_prompt(PyObject *const *o, int &status) {
    Arguments in;
    in.where(o[5]);
    Rows r;
    const at::Tensor *counts = in.walked(o[0], at::kShort, 1, r), *slot = in.plain(o[1], at::kInt);
    if (!in.ok || counts->dim() != 2 || slot->dim() != 1) return false;
    const int64_t m = slot->size(0);
    const at::Tensor *cu = in.plain(o[2], at::kInt, {m + 1}), *tokens = in.plain(o[3], at::kInt);
    const at::Tensor *st = in.plain_or_none(o[4], at::kInt, {m});
    if (!in.ok || !narrow(m) || !narrow(tokens->numel()) || !narrow(r.count) || !narrow(r.d))
        return false;
    status = unlocked(
        gdn_count_prompt, data<int16_t>(counts), r.stride, data<int32_t>(slot), data<int32_t>(cu),
        data<int32_t>(tokens), (int)m, (int)tokens->numel(), (int)r.count, (int)r.d,
        data<int32_t>(st), in.stream);
    return true;
}

// (counts, slot, tokens, path, add, status, stream)
bool run_count_commit(PyObject *const *o, int &status) {
    Arguments in;
    in.where(o[6]);
    Rows r;
    const at::Tensor *counts = in.walked(o[0], at::kShort, 1, r), *slot = in.plain(o[1], at::kInt);
    if (!in.ok || counts->dim() != 2 || slot->dim() != 1) return false;
    const int64_t m = slot->size(0);
    const at::Tensor *tokens = in.plain(o[2], at::kInt), *path = in.plain(o[3], at::kInt);
    const at::Tensor *add = in.plain(o[4], at::kInt, {m});
    const at::Tensor *st = in.plain_or_none(o[5], at::kInt, {m});
    if (!in.ok || tokens->dim() != 2 || tokens->size(0) != m || path->dim() != 2 ||
        path->size(0) != m || !narrow(m) || !narrow(tokens->size(1)) || !narrow(path->size(1)) ||
        !narrow(r.count) || !narrow(r.d))
        return false;
    status = unlocked(
        gdn_count_commit, data<int16_t>(counts), r.stride, data<int32_t>(slot),
        data<int32_t>(tokens), data<int32_t>(path), data<int32_t>(add), (int)m,
        (int)tokens->size(1), (int)path->size(1), (int)r.count, (int)r.d, data<int32_t>(st),
        in.stream);
    return true;
}

// (logits, counts, slot, tokens, parent, repetition, presence, frequency,
// bias_tok, bias, mask, out, best, status, stream, workspace)
bool run_logits(PyObject *const *o, int &status) {
    Arguments in;
    in.where(o[14]);
    const at::Tensor *z = in.tensor(o[0]);
    if (!z || z->dim() != 3) return false;
    const at::ScalarType t = z->scalar_type();
    gdn_dtype dtype, out_dtype;
    Rows rz, rc, ro;
    if (!element_type(t, dtype) || !walk(*z, 1, rz)) return false;
    out_dtype = dtype;
    const int64_t batch = z->size(0), n = z->size(1), words = (rz.d + 31) / 32;
    const at::Tensor *counts = nullptr, *slot = nullptr;
    if (o[1] != Py_None) {
        counts = in.walked(o[1], at::kShort, 1, rc);
        slot = in.plain_or_none(o[2], at::kInt, {batch});
        if (!in.ok || counts->dim() != 2 || rc.d != rz.d) return false;
    } else if (o[2] != Py_None) {
        return false;
    }
    if ((o[3] == Py_None) != (o[4] == Py_None) || (o[8] == Py_None) != (o[9] == Py_None)) return false;
    const at::Tensor *tokens = in.plain_or_none(o[3], at::kInt, {batch, n});
    const at::Tensor *parent = in.plain_or_none(o[4], at::kInt, {batch, n});
    const at::Tensor *penalty[3];
    for (int i = 0; i < 3; ++i) penalty[i] = in.plain_or_none(o[5 + i], at::kFloat, {batch});
    const at::Tensor *bias_tok = nullptr, *bias = nullptr, *mask = nullptr, *out = nullptr;
    int64_t biases = 0, mask_rows = 0;
    if (o[8] != Py_None) {
        bias_tok = in.plain(o[8], at::kInt);
        if (!in.ok || bias_tok->dim() != 2 || bias_tok->size(0) != batch) return false;
        biases = bias_tok->size(1);
        bias = in.plain(o[9], at::kFloat, bias_tok->sizes());
    }
    if (o[10] != Py_None) {
        mask = in.plain(o[10], at::kInt);
        if (!in.ok || mask->dim() != 3 || mask->size(0) != batch || mask->size(2) != words)
            return false;
        mask_rows = mask->size(1);
        if (mask_rows != 1 && mask_rows != n) return false;
    }
    if (o[11] != Py_None) {
        out = in.tensor(o[11]);
        if (!out || (out->scalar_type() != t && out->scalar_type() != at::kFloat) ||
            !walk(*out, 1, ro) || out->sizes() != z->sizes() ||
            !element_type(out->scalar_type(), out_dtype))
            return false;
    }
    const at::Tensor *best = in.plain(o[12], at::kInt, {batch, n});
    const at::Tensor *st = in.plain_or_none(o[13], at::kInt, {batch});
    const at::Tensor *room = in.plain(o[15], at::kByte);
    if (!in.ok) return false;
    for (int64_t x : {batch, n, rz.d, rc.count, biases})
        if (!narrow(x)) return false;
    status = unlocked(
        gdn_adjust_logits, data(z), dtype, rz.stride, data<int16_t>(counts), rc.stride,
        data<int32_t>(slot), (int)rc.count, data<int32_t>(tokens), data<int32_t>(parent), data<float>(penalty[0]),
        data<float>(penalty[1]), data<float>(penalty[2]), data<int32_t>(bias_tok), data<float>(bias),
        (int)biases, data<int32_t>(mask), (int)mask_rows, data(out), out_dtype, ro.stride,
        data<int32_t>(best), (int)batch, (int)n, (int)rz.d, data(room), room->numel(),
        data<int32_t>(st), in.stream);
    return true;
}

#define WHOLE(name, run, count)                                                       \
    PyObject *name(PyObject *, PyObject *const *args, Py_ssize_t n) {                 \
        return whole_call(args, n, count, run);                                       \
    }
WHOLE(heads_call, run_heads, 15)
WHOLE(append_call, run_append, 22)
WHOLE(count_prompt_call, run_count_prompt, 6)
WHOLE(count_commit_call, run_count_commit, 7)
WHOLE(logits_call, run_logits, 16)

#define FASTCALL(name) \
    {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}

PyMethodDef g_methods[] = {
    FASTCALL(streams),
    FASTCALL(heads_call),
    FASTCALL(append_call),
    FASTCALL(count_prompt_call),
    FASTCALL(count_commit_call),
    FASTCALL(logits_call),
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
