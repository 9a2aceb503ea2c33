// The ordinary calls of the 8-bit operators, without the interpreter between their checks: matrices and
// vectors as they mostly are, on the current device, with outputs made here.  Every other call (given
// outputs, wrong arguments, other devices, empty matrices) is left to the checks of w8.py: a function here
// returns None for it, before anything is queued.  What fails behind the checks (no memory for an output, an
// error of the runtime, which may come with a kernel already queued) is raised here, as w8.py raises it.
//
// The interpreter's lock is released while outputs are allocated and the library is called, which may wait (for
// memory, for room in a queue): other threads run meanwhile.
//
// A call on few rows is over sooner on the GPU (2 to 7 us) than the interpreter has checked its arguments, made
// its outputs and passed it on (one row, calls one behind the other): quant8 7.5 us there and 4.6 here, dequant8 6.6
// and 3.7, rmsnorm8 with a residual 10 and 5.4, gemm8 8.4 and 4.2.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "qamw_w8.h"

namespace {

using at::Tensor;

struct Entry {
    decltype(&qamw_quant8) quant8;
    decltype(&qamw_dequant8) dequant8;
    decltype(&qamw_rmsnorm8) rmsnorm8;
    decltype(&qamw_gemm8_workspace) gemm8_workspace;
    decltype(&qamw_gemm8) gemm8;
} lib;

struct Skip {};     // not an ordinary call
struct Raised {};   // a Python error is set

PyObject* failed = nullptr;   // failed(return code, function) raises

// The answer of the library: done, or a refusal, before anything was queued (w8.py gives its reason), or an
// error of the runtime.
void check(int rc, const char* name) {
    if (rc == QAMW_OK) return;
    if (rc == QAMW_ERR_ARG || rc == QAMW_ERR_UNSUPPORTED || rc == QAMW_ERR_WORKSPACE) throw Skip{};
    Py_XDECREF(PyObject_CallFunction(failed, "is", rc, name));
    throw Raised{};
}

const Tensor& tensor(PyObject* o) {
    if (!THPVariable_CheckExact(o)) throw Skip{};
    return THPVariable_Unpack(o);
}

void on(const Tensor& t, int device) {
    if (!t.is_cuda() || t.get_device() != device || t.layout() != at::kStrided) throw Skip{};
}

struct Rows {
    const void* p;
    int32_t n, d;
    int64_t ld;
};

// A bf16 or fp32 matrix with contiguous rows, of the size and type of `like`.
Rows rows(const Tensor& t, int device, const Tensor* like = nullptr) {
    on(t, device);
    if (t.dim() != 2 || (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kFloat)) throw Skip{};
    const int64_t n = t.size(0), d = t.size(1), ld = t.stride(0);
    if (n < 1 || d < 1 || n > INT32_MAX || d > INT32_MAX || t.stride(1) != 1 || ld < d) throw Skip{};
    if (like && (like->size(0) != n || like->size(1) != d || like->scalar_type() != t.scalar_type())) throw Skip{};
    return {t.const_data_ptr(), (int32_t)n, (int32_t)d, ld};
}

// Codes with whole 16-byte chunks inside their storage.
Rows codes(const Tensor& t, int device) {
    on(t, device);
    if (t.dim() != 2 || t.scalar_type() != at::kChar) throw Skip{};
    const int64_t n = t.size(0), d = t.size(1), ld = t.stride(0), padded = (d + 15) / 16 * 16;
    if (n < 1 || d < 1 || n > INT32_MAX || d > INT32_MAX || t.stride(1) != 1 || ld < padded || ld % 16) throw Skip{};
    if (d != padded && t.storage_offset() + (n - 1) * ld + padded > (int64_t)t.storage().nbytes()) throw Skip{};
    const void* p = t.const_data_ptr();
    if ((uintptr_t)p % 16) throw Skip{};
    return {p, (int32_t)n, (int32_t)d, ld};
}

const float* vec(const Tensor& t, int device, int64_t n) {
    on(t, device);
    if (t.scalar_type() != at::kFloat || t.numel() < n || !t.is_contiguous()) throw Skip{};
    return t.const_data_ptr<float>();
}

// The tensor's device, which is the current one.
int current_of(const Tensor& t) {
    if (!t.is_cuda() || t.get_device() != c10::hip::current_device()) throw Skip{};
    return t.get_device();
}

void* stream(int device) { return c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream(); }

qamw_dtype dtype(const Tensor& t) { return t.scalar_type() == at::kBFloat16 ? QAMW_BF16 : QAMW_F32; }

Tensor make(const Tensor& like, at::IntArrayRef size, at::ScalarType type) {
    return at::empty(size, like.options().dtype(type).requires_grad(false));
}

// Codes for n rows of d columns: rows of whole 16-byte chunks.
Tensor make_codes(const Tensor& like, int64_t n, int64_t d) {
    const int64_t pitch = (d + 15) / 16 * 16;
    Tensor q = make(like, {n, pitch}, at::kChar);
    return pitch == d ? q : q.slice(1, 0, d);
}

int64_t pitch_of(int64_t d) { return (d + 15) / 16 * 16; }

// A tuple of new references; null if one of them is.
PyObject* tuple(std::initializer_list<PyObject*> items) {
    PyObject* t = PyTuple_New((Py_ssize_t)items.size());
    bool whole = t;
    Py_ssize_t i = 0;
    for (PyObject* o : items) {
        whole = whole && o;
        if (t) PyTuple_SET_ITEM(t, i++, o);
        else Py_XDECREF(o);
    }
    if (!whole) Py_CLEAR(t);
    return t;
}

// The interpreter's lock is free as long as one of these lives.
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    Unlocked() = default;
    Unlocked(const Unlocked&) = delete;
    ~Unlocked() { PyEval_RestoreThread(state); }
};

template <typename F>
PyObject* ordinary(Py_ssize_t given, Py_ssize_t wanted, F&& f) {
    HANDLE_TH_ERRORS
    try {
        if (given != wanted || !lib.gemm8) throw Skip{};
        return f();
    } catch (const Skip&) {
        Py_RETURN_NONE;
    } catch (const Raised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject* quant8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary(n, 3, [&]() -> PyObject* {
        const Tensor& x = tensor(a[0]);
        const int dev = current_of(x);
        const Rows r = rows(x, dev);
        const float* scale = a[1] == Py_None ? nullptr : vec(tensor(a[1]), dev, r.d);
        Rows g{nullptr, 0, 0, 0};
        if (a[2] != Py_None) g = rows(tensor(a[2]), dev, &x);
        Tensor q, s;
        int rc;
        {
            const Unlocked unlocked;
            q = make_codes(x, r.n, r.d);
            s = make(x, {r.n}, at::kFloat);
            rc = lib.quant8(r.p, dtype(x), r.n, r.d, r.ld, g.p, g.ld, scale, q.data_ptr<int8_t>(), pitch_of(r.d),
                            s.data_ptr<float>(), nullptr, stream(dev));
        }
        check(rc, "qamw_quant8");
        return tuple({THPVariable_Wrap(std::move(q)), THPVariable_Wrap(std::move(s))});
    });
}

PyObject* dequant8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary(n, 4, [&]() -> PyObject* {
        const Tensor& c = tensor(a[0]);
        const int dev = current_of(c);
        const Rows r = codes(c, dev);
        const float* s = vec(tensor(a[1]), dev, r.n);
        const float* scale = a[2] == Py_None ? nullptr : vec(tensor(a[2]), dev, r.d);
        Tensor y;
        int rc;
        {
            const Unlocked unlocked;
            y = make(c, {r.n, r.d}, a[3] == Py_True ? at::kBFloat16 : at::kFloat);
            rc = lib.dequant8((const int8_t*)r.p, r.n, r.d, r.ld, s, scale, y.data_ptr(), dtype(y), r.d, stream(dev));
        }
        check(rc, "qamw_dequant8");
        return THPVariable_Wrap(std::move(y));
    });
}

PyObject* rmsnorm8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary(n, 4, [&]() -> PyObject* {
        const Tensor& x = tensor(a[0]);
        const int dev = current_of(x);
        const Rows r = rows(x, dev);
        const float* w = a[1] == Py_None ? nullptr : vec(tensor(a[1]), dev, r.d);
        const double eps = PyFloat_AsDouble(a[2]);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            throw Skip{};
        }
        Rows o{nullptr, 0, 0, 0};
        if (a[3] != Py_None) {
            const Tensor& res = tensor(a[3]);
            o = rows(res, dev, &x);
            if (c10::GradMode::is_enabled() && (x.requires_grad() || res.requires_grad())) throw Skip{};
        }
        Tensor h, q, s;
        int rc;
        {
            const Unlocked unlocked;
            if (o.p) h = make(x, {r.n, r.d}, x.scalar_type());
            q = make_codes(x, r.n, r.d);
            s = make(x, {r.n}, at::kFloat);
            rc = lib.rmsnorm8(r.p, dtype(x), r.n, r.d, r.ld, o.p, o.ld, w, (float)eps, o.p ? h.data_ptr() : nullptr,
                              r.d, q.data_ptr<int8_t>(), pitch_of(r.d), s.data_ptr<float>(), nullptr, stream(dev));
        }
        check(rc, "qamw_rmsnorm8");
        PyObject* sum = h.defined() ? THPVariable_Wrap(std::move(h)) : Py_NewRef(a[0]);   // without a residual: x
        return tuple({THPVariable_Wrap(std::move(q)), THPVariable_Wrap(std::move(s)), sum});
    });
}

PyObject* gemm8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary(n, 5, [&]() -> PyObject* {
        const Tensor& xq = tensor(a[0]);
        const Tensor& wq = tensor(a[2]);
        const int dev = current_of(xq);
        const Rows x = codes(xq, dev), w = codes(wq, dev);
        if (x.d != w.d) throw Skip{};
        const float *xs = vec(tensor(a[1]), dev, x.n), *ws = vec(tensor(a[3]), dev, w.n);
        Tensor y, work;
        int rc;
        {
            const Unlocked unlocked;
            y = make(xq, {x.n, w.n}, a[4] == Py_True ? at::kBFloat16 : at::kFloat);
            const size_t need = lib.gemm8_workspace(x.n, w.n, x.d);
            if (need) work = make(xq, {(int64_t)need}, at::kByte);
            rc = lib.gemm8((const int8_t*)x.p, x.ld, xs, x.n, (const int8_t*)w.p, w.ld, ws, w.n, x.d, y.data_ptr(),
                           dtype(y), w.n, need ? work.data_ptr() : nullptr, need, stream(dev));
        }
        check(rc, "qamw_gemm8");
        return THPVariable_Wrap(std::move(y));
    });
}

// bind(quant8, dequant8, rmsnorm8, gemm8_workspace, gemm8, failed): the library's functions, as addresses, and
// what raises the error of a return code.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "bind takes 5 addresses and a callable");
        return nullptr;
    }
    void* p[5];
    for (Py_ssize_t i = 0; i < 5; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    Py_INCREF(a[5]);
    Py_XSETREF(failed, a[5]);
    lib = {(decltype(lib.quant8))p[0], (decltype(lib.dequant8))p[1], (decltype(lib.rmsnorm8))p[2],
           (decltype(lib.gemm8_workspace))p[3], (decltype(lib.gemm8))p[4]};
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, nullptr},
    {"quant8", (PyCFunction)(void (*)(void))quant8, METH_FASTCALL, nullptr},
    {"dequant8", (PyCFunction)(void (*)(void))dequant8, METH_FASTCALL, nullptr},
    {"rmsnorm8", (PyCFunction)(void (*)(void))rmsnorm8, METH_FASTCALL, nullptr},
    {"gemm8", (PyCFunction)(void (*)(void))gemm8, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_w8_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__w8_host(void) { return PyModule_Create(&module); }
