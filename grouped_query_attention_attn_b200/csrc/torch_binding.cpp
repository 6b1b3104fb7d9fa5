// torch_binding.cpp -- the tensor-level calls of the paged 8-bit cache as a CPython
// extension.
//
// A serving step makes these calls once per layer or token, and their kernels take
// a few microseconds: checking seven tensors and marshalling twenty arguments in
// Python takes longer than that.  The functions here check the tensors, allocate
// outputs and workspace, and call the C entry points of libgqa.so on the current
// stream; api.py holds the signatures, defaults and documentation.  They raise
// what api.py's other calls raise: TypeError, ValueError (also for a bad or small
// workspace), NotImplementedError for unsupported shapes, RuntimeError otherwise.
// The library is not linked: bind() receives the addresses of its entry points.
#include <Python.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <cmath>

#include "gqa.h"

namespace {

decltype(&gqa_decode8) f_decode8;
decltype(&gqa_decode8_workspace_size) f_decode8_workspace_size;
decltype(&gqa_cache8_append) f_cache8_append;
decltype(&gqa_cache8_read) f_cache8_read;
decltype(&gqa_cache8_copy) f_cache8_copy;
decltype(&gqa_pages_resize) f_pages_resize;
decltype(&gqa_pages_fork) f_pages_fork;
decltype(&gqa_pages_compact) f_pages_compact;
decltype(&gqa_pages_workspace_size) f_pages_workspace_size;
decltype(&gqa_last_error) f_last_error;

const at::ScalarType kBf16 = at::kBFloat16, kInt = at::kInt, kFloat = at::kFloat;

[[noreturn]] void raise_shape(const char *what, const at::Tensor &t) {
    TORCH_CHECK_VALUE(false, what, ", got shape ", t.sizes());
}

// A contiguous CUDA tensor of one type and number of dimensions, on device dev
// (-1: not known yet, set here).
const at::Tensor &need(PyObject *o, const char *name, at::ScalarType type, int64_t dim, int &dev) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a torch.Tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor");
    TORCH_CHECK_VALUE(t.scalar_type() == type, name, " must be ", type, ", got ", t.scalar_type());
    TORCH_CHECK_VALUE(t.dim() == dim, name, " must have ", dim, " dims, got shape ", t.sizes());
    TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
    for (const int64_t n : t.sizes()) TORCH_CHECK_VALUE(n <= INT_MAX, name, " is too large: ", t.sizes());
    const int at = t.get_device();
    if (dev < 0) dev = at;
    TORCH_CHECK_VALUE(at == dev, "tensors on cuda:", dev, " and cuda:", at, ": one device is needed");
    return t;
}

struct Cache {
    const at::Tensor *k, *v, *ks, *vs;
    int kind, n_pages, Hkv, page, d, block;

    Cache(PyObject *o, int &dev) {
        TORCH_CHECK_TYPE(PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 4,
                         "the cache must be a Cache8 (k, v, k_scale, v_scale)");
        PyObject *first = PyTuple_GET_ITEM(o, 0);
        TORCH_CHECK_TYPE(THPVariable_Check(first), "cache.k must be a torch.Tensor");
        const at::ScalarType type = THPVariable_Unpack(first).scalar_type();
        TORCH_CHECK_VALUE(type == at::kFloat8_e4m3fn || type == at::kChar,
                          "the cache must be torch.float8_e4m3fn or torch.int8, got ", type);
        kind = type == at::kChar ? GQA_INT8 : GQA_E4M3;
        k = &need(first, "cache.k", type, 4, dev);
        v = &need(PyTuple_GET_ITEM(o, 1), "cache.v", type, 4, dev);
        ks = &need(PyTuple_GET_ITEM(o, 2), "cache.k_scale", kFloat, 3, dev);
        vs = &need(PyTuple_GET_ITEM(o, 3), "cache.v_scale", kFloat, 3, dev);
        const auto s = k->sizes(), n = ks->sizes();
        TORCH_CHECK_VALUE(v->sizes() == s && vs->sizes() == n && n[0] == s[0] && n[1] == s[1] && n[2] >= 1 &&
                              s[2] % n[2] == 0,
                          "cache shape mismatch: k ", s, ", v ", v->sizes(), ", k_scale ", n, ", v_scale ",
                          vs->sizes());
        n_pages = static_cast<int>(s[0]);
        Hkv = static_cast<int>(s[1]);
        page = static_cast<int>(s[2]);
        d = static_cast<int>(s[3]);
        block = static_cast<int>(s[2] / n[2]);
    }
};

struct Table {
    const at::Tensor *t;
    int B, M;

    Table(PyObject *o, int &dev) : t(&need(o, "table", kInt, 2, dev)) {
        B = static_cast<int>(t->size(0));
        M = static_cast<int>(t->size(1));
    }
    const at::Tensor &vector(PyObject *o, const char *name, int &dev) const {
        const at::Tensor &x = need(o, name, kInt, 1, dev);
        TORCH_CHECK_VALUE(x.size(0) == B, name, " must have ", B, " entries, one per table row, got ",
                          x.size(0));
        return x;
    }
};

template <class T>
T *ptr(const at::Tensor &t) {
    return static_cast<T *>(t.data_ptr());
}

int as_int(PyObject *o, const char *name) {
    int overflow = 0;
    const long long x = PyLong_AsLongLongAndOverflow(o, &overflow);
    if (x == -1 && PyErr_Occurred()) throw python_error();
    TORCH_CHECK_VALUE(!overflow && x >= INT_MIN && x <= INT_MAX, name, " is out of range");
    return static_cast<int>(x);
}

double as_double(PyObject *o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw python_error();
    return x;
}

// torch.empty on device dev, without the dispatcher.
at::Tensor empty_on(at::IntArrayRef shape, at::ScalarType type, int dev) {
    return at::Tensor(at::detail::empty_cuda(
        shape, type, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt));
}

at::Tensor workspace_of(PyObject *o, size_t need_bytes, int &dev) {
    if (o != Py_None) return need(o, "workspace", at::kByte, 1, dev);
    return empty_on({static_cast<int64_t>(need_bytes)}, at::kByte, dev);
}

// Runs call(stream) with dev current and the GIL released; raises on a non-zero status.
template <class F>
void run(const char *what, int dev, F &&call) {
    const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev)));
    const auto stream = reinterpret_cast<gqa_stream_t>(
        c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
    int rc;
    std::string why;
    Py_BEGIN_ALLOW_THREADS
    rc = call(stream);
    if (rc != GQA_OK) why = f_last_error();          // of this thread
    Py_END_ALLOW_THREADS
    if (rc == GQA_OK) return;
    TORCH_CHECK_VALUE(rc != GQA_ERR_INVALID_ARG && rc != GQA_ERR_WORKSPACE, what, ": ", why, " (status ", rc, ")");
    TORCH_CHECK_NOT_IMPLEMENTED(rc != GQA_ERR_UNSUPPORTED, what, ": ", why, " (status ", rc, ")");
    TORCH_CHECK(false, what, ": ", why, " (status ", rc, ")");
}

void check_count(const char *name, Py_ssize_t n, Py_ssize_t want) {
    TORCH_CHECK_TYPE(n == want, name, " takes ", want, " arguments, got ", n);
    TORCH_CHECK(f_last_error != nullptr, "the library is not bound");
}

PyObject *same(PyObject *o) {
    Py_INCREF(o);
    return o;
}

// (q, cache, table, seqlens, scale, workspace, out, window, sinks, rope_theta)
PyObject *decode8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count("decode8", n, 10);
    int dev = -1;
    const Cache c(a[1], dev);
    const Table t(a[2], dev);
    const at::Tensor &lens = t.vector(a[3], "seqlens", dev), &q = need(a[0], "q", kBf16, 3, dev);
    if (q.size(0) != t.B || q.size(2) != c.d) raise_shape("q must be [B, Hq, d] as the table and cache", q);
    const int Hq = static_cast<int>(q.size(1)), sinks = as_int(a[8], "sinks");
    int window = 0;
    if (a[7] != Py_None) {
        window = as_int(a[7], "window");
        TORCH_CHECK_VALUE(window >= 1, "window=", window, " must be >= 1");
    }
    float theta = 0.0f;
    if (a[9] != Py_None) {
        theta = static_cast<float>(as_double(a[9]));
        TORCH_CHECK_VALUE(theta > 0.0f, "rope_theta=", theta, " must be > 0");
    }
    const float scale = a[4] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(c.d)))
                                        : static_cast<float>(as_double(a[4]));
    at::Tensor o;
    if (a[6] == Py_None) {
        o = empty_on(q.sizes(), kBf16, dev);
    } else {
        o = need(a[6], "out", kBf16, 3, dev);
        if (o.sizes() != q.sizes()) raise_shape("out must have q's shape", o);
    }
    const long long Lmax = static_cast<long long>(t.M) * c.page;
    const at::Tensor ws = workspace_of(
        a[5], f_decode8_workspace_size(t.B, Hq, c.Hkv, c.d, static_cast<int>(std::min<long long>(Lmax, INT_MAX))),
        dev);
    run("gqa_decode8", dev, [&](gqa_stream_t s) {
        return f_decode8(q.data_ptr(), c.k->data_ptr(), c.v->data_ptr(), ptr<float>(*c.ks), ptr<float>(*c.vs),
                         ptr<int32_t>(*t.t), ptr<int32_t>(lens), o.data_ptr(), c.kind, t.B, Hq, c.Hkv, c.d, t.M,
                         c.n_pages, c.page, c.block, window, sinks, scale, theta, ws.data_ptr(),
                         static_cast<size_t>(ws.numel()), s);
    });
    return a[6] == Py_None ? THPVariable_Wrap(std::move(o)) : same(a[6]);
    END_HANDLE_TH_ERRORS
}

// (cache, table, seqlens, k, v, counts)
PyObject *cache8_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count("cache8_append_", n, 6);
    int dev = -1;
    const Cache c(a[0], dev);
    const Table t(a[1], dev);
    const at::Tensor &lens = t.vector(a[2], "seqlens", dev);
    const at::Tensor &k = need(a[3], "k", kBf16, 4, dev), &v = need(a[4], "v", kBf16, 4, dev);
    const int32_t *counts = a[5] == Py_None ? nullptr : ptr<int32_t>(t.vector(a[5], "counts", dev));
    if (k.size(0) != t.B || k.size(2) != c.Hkv || k.size(3) != c.d)
        raise_shape("k must be [B, T, Hkv, d] as the table and cache", k);
    if (v.sizes() != k.sizes()) raise_shape("v must have k's shape", v);
    run("gqa_cache8_append", dev, [&](gqa_stream_t s) {
        return f_cache8_append(c.k->data_ptr(), c.v->data_ptr(), ptr<float>(*c.ks), ptr<float>(*c.vs),
                               ptr<int32_t>(*t.t), ptr<int32_t>(lens), counts, k.data_ptr(), v.data_ptr(), c.kind,
                               t.B, static_cast<int>(k.size(1)), t.M, c.n_pages, c.Hkv, c.page, c.d, c.block, s);
    });
    return same(a[0]);
    END_HANDLE_TH_ERRORS
}

// (cache, table, seqlens, T, out)
PyObject *cache8_read(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count("cache8_read", n, 5);
    int dev = -1;
    const Cache c(a[0], dev);
    const Table t(a[1], dev);
    const at::Tensor &lens = t.vector(a[2], "seqlens", dev);
    const int T = as_int(a[3], "T");
    TORCH_CHECK_VALUE(T >= 0, "T=", T, " must be >= 0");
    const int64_t shape[4] = {t.B, T, c.Hkv, c.d};
    at::Tensor x[2];
    if (a[4] != Py_None)
        TORCH_CHECK_TYPE(PyTuple_Check(a[4]) || PyList_Check(a[4]), "out must be a pair of tensors");
    for (int i = 0; i < 2; ++i) {
        if (a[4] == Py_None) {
            x[i] = empty_on(shape, kBf16, dev);
            continue;
        }
        TORCH_CHECK_TYPE(PySequence_Size(a[4]) == 2, "out must be a pair of tensors");
        PyObject *o = PyTuple_Check(a[4]) ? PyTuple_GET_ITEM(a[4], i) : PyList_GET_ITEM(a[4], i);
        x[i] = need(o, i ? "out[1]" : "out[0]", kBf16, 4, dev);
        if (x[i].sizes() != at::IntArrayRef(shape)) raise_shape("out must hold tensors [B, T, Hkv, d]", x[i]);
    }
    run("gqa_cache8_read", dev, [&](gqa_stream_t s) {
        return f_cache8_read(c.k->data_ptr(), c.v->data_ptr(), ptr<float>(*c.ks), ptr<float>(*c.vs),
                             ptr<int32_t>(*t.t), ptr<int32_t>(lens), x[0].data_ptr(), x[1].data_ptr(), c.kind, t.B,
                             T, t.M, c.n_pages, c.Hkv, c.page, c.d, c.block, s);
    });
    PyObject *k = THPVariable_Wrap(std::move(x[0])), *v = THPVariable_Wrap(std::move(x[1]));
    PyObject *r = PyTuple_Pack(2, k, v);
    Py_XDECREF(k);
    Py_XDECREF(v);
    return r;
    END_HANDLE_TH_ERRORS
}

// (cache, moves)
PyObject *cache8_copy(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count("cache8_copy_", n, 2);
    int dev = -1;
    const Cache c(a[0], dev);
    const at::Tensor &m = need(a[1], "moves", kInt, 2, dev);
    if (m.size(0) < 1 || m.size(1) != 3) raise_shape("moves must be [1 + cap, 3]", m);
    run("gqa_cache8_copy", dev, [&](gqa_stream_t s) {
        return f_cache8_copy(c.k->data_ptr(), c.v->data_ptr(), ptr<float>(*c.ks), ptr<float>(*c.vs),
                             ptr<int32_t>(m), static_cast<int>(m.size(0) - 1), c.n_pages, c.Hkv, c.page, c.d,
                             c.block, s);
    });
    return same(a[0]);
    END_HANDLE_TH_ERRORS
}

// (table, refs, lengths, page, workspace)
PyObject *pages_resize(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count("pages_resize_", n, 5);
    int dev = -1;
    const Table t(a[0], dev);
    const at::Tensor &refs = need(a[1], "refs", kInt, 1, dev), &lens = t.vector(a[2], "lengths", dev);
    const int n_pages = static_cast<int>(refs.size(0)), page = as_int(a[3], "page");
    const at::Tensor ws = workspace_of(a[4], f_pages_workspace_size(t.B, t.M, n_pages), dev);
    run("gqa_pages_resize", dev, [&](gqa_stream_t s) {
        return f_pages_resize(ptr<int32_t>(*t.t), ptr<int32_t>(refs), ptr<int32_t>(lens), t.B, t.M, n_pages, page,
                              ws.data_ptr(), static_cast<size_t>(ws.numel()), s);
    });
    return same(a[0]);
    END_HANDLE_TH_ERRORS
}

// (table, refs, seqlens, parents, page, workspace)
PyObject *pages_fork(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count("pages_fork_", n, 6);
    int dev = -1;
    const Table t(a[0], dev);
    const at::Tensor &refs = need(a[1], "refs", kInt, 1, dev), &lens = t.vector(a[2], "seqlens", dev);
    const at::Tensor &parents = t.vector(a[3], "parents", dev);
    const int n_pages = static_cast<int>(refs.size(0)), page = as_int(a[4], "page");
    const at::Tensor ws = workspace_of(a[5], f_pages_workspace_size(t.B, t.M, n_pages), dev);
    at::Tensor moves = empty_on({1 + static_cast<int64_t>(t.B), 3}, kInt, dev);
    run("gqa_pages_fork", dev, [&](gqa_stream_t s) {
        return f_pages_fork(ptr<int32_t>(*t.t), ptr<int32_t>(refs), ptr<int32_t>(lens), ptr<int32_t>(parents),
                            ptr<int32_t>(moves), t.B, t.M, n_pages, page, ws.data_ptr(),
                            static_cast<size_t>(ws.numel()), s);
    });
    return THPVariable_Wrap(std::move(moves));
    END_HANDLE_TH_ERRORS
}

// (table, refs, page, workspace)
PyObject *pages_compact(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count("pages_compact_", n, 4);
    int dev = -1;
    const Table t(a[0], dev);
    const at::Tensor &refs = need(a[1], "refs", kInt, 1, dev);
    const int n_pages = static_cast<int>(refs.size(0)), page = as_int(a[2], "page");
    const at::Tensor ws = workspace_of(a[3], f_pages_workspace_size(t.B, t.M, n_pages), dev);
    at::Tensor moves = empty_on({1 + static_cast<int64_t>(n_pages / 2), 3}, kInt, dev);
    run("gqa_pages_compact", dev, [&](gqa_stream_t s) {
        return f_pages_compact(ptr<int32_t>(*t.t), ptr<int32_t>(refs), ptr<int32_t>(moves), t.B, t.M, n_pages, page,
                               ws.data_ptr(), static_cast<size_t>(ws.numel()), s);
    });
    return THPVariable_Wrap(std::move(moves));
    END_HANDLE_TH_ERRORS
}

// bind(lookup): lookup(name) gives the address of an entry point.
PyObject *bind(PyObject *, PyObject *lookup) {
    HANDLE_TH_ERRORS
    auto set = [&](auto &f, const char *name) {
        PyObject *x = PyObject_CallFunction(lookup, "s", name);
        if (!x) throw python_error();
        void *p = PyLong_AsVoidPtr(x);
        Py_DECREF(x);
        if (!p && PyErr_Occurred()) throw python_error();
        TORCH_CHECK(p != nullptr, name, " has no address");
        f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(p);
    };
    set(f_decode8, "gqa_decode8");
    set(f_decode8_workspace_size, "gqa_decode8_workspace_size");
    set(f_cache8_append, "gqa_cache8_append");
    set(f_cache8_read, "gqa_cache8_read");
    set(f_cache8_copy, "gqa_cache8_copy");
    set(f_pages_resize, "gqa_pages_resize");
    set(f_pages_fork, "gqa_pages_fork");
    set(f_pages_compact, "gqa_pages_compact");
    set(f_pages_workspace_size, "gqa_pages_workspace_size");
    set(f_last_error, "gqa_last_error");
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

using Fast = PyObject *(*)(PyObject *, PyObject *const *, Py_ssize_t);
PyMethodDef entry(const char *name, Fast f) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {
    entry("decode8", decode8),           entry("cache8_append_", cache8_append),
    entry("cache8_read", cache8_read),   entry("cache8_copy_", cache8_copy),
    entry("pages_resize_", pages_resize), entry("pages_fork_", pages_fork),
    entry("pages_compact_", pages_compact), {"bind", bind, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the torch and Python it was compiled against (build.py looks for it in the file)
PyMODINIT_FUNC PyInit__torch_binding() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", GQA_BUILT_FOR) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
