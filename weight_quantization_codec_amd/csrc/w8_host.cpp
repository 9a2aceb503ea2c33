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
// its outputs and passed it on (one row, calls one behind the other): quant8 7.5 us there and 4.4 here, dequant8 6.8
// and 4.1, rmsnorm8 with a residual 10 and 5.0, gemm8 8.4 and 4.2.
#include "host_calls.hpp"
#include "qamw_w8.h"

extern PyMethodDef mx4_methods[];

namespace {

using namespace host;

struct Entry {
    decltype(&qamw_quant8) quant8;
    decltype(&qamw_dequant8) dequant8;
    decltype(&qamw_rmsnorm8) rmsnorm8;
    decltype(&qamw_gemm8_workspace) gemm8_workspace;
    decltype(&qamw_gemm8) gemm8;
} lib;

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

// Codes for n rows of d columns: rows of whole 16-byte chunks.
Tensor make_codes(int64_t n, int64_t d) {
    const int64_t pitch = (d + 15) / 16 * 16;
    Tensor q = make({n, pitch}, at::kChar);
    return pitch == d ? q : q.slice(1, 0, d);
}

int64_t pitch_of(int64_t d) { return (d + 15) / 16 * 16; }

PyObject* quant8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary(n == 3 && lib.gemm8, [&]() -> PyObject* {
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
            q = make_codes(r.n, r.d);
            s = make({r.n}, at::kFloat);
            rc = lib.quant8(r.p, dtype(x), r.n, r.d, r.ld, g.p, g.ld, scale, q.data_ptr<int8_t>(), pitch_of(r.d),
                            s.data_ptr<float>(), nullptr, stream(dev));
        }
        check(rc, "qamw_quant8");
        return tuple({THPVariable_Wrap(std::move(q)), THPVariable_Wrap(std::move(s))});
    });
}

PyObject* dequant8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary(n == 4 && lib.gemm8, [&]() -> PyObject* {
        const Tensor& c = tensor(a[0]);
        const int dev = current_of(c);
        const Rows r = codes(c, dev);
        const float* s = vec(tensor(a[1]), dev, r.n);
        const float* scale = a[2] == Py_None ? nullptr : vec(tensor(a[2]), dev, r.d);
        Tensor y;
        int rc;
        {
            const Unlocked unlocked;
            y = make({r.n, r.d}, a[3] == Py_True ? at::kBFloat16 : at::kFloat);
            rc = lib.dequant8((const int8_t*)r.p, r.n, r.d, r.ld, s, scale, y.data_ptr(), dtype(y), r.d, stream(dev));
        }
        check(rc, "qamw_dequant8");
        return THPVariable_Wrap(std::move(y));
    });
}

PyObject* rmsnorm8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary(n == 4 && lib.gemm8, [&]() -> PyObject* {
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
            if (o.p) h = make({r.n, r.d}, x.scalar_type());
            q = make_codes(r.n, r.d);
            s = make({r.n}, at::kFloat);
            rc = lib.rmsnorm8(r.p, dtype(x), r.n, r.d, r.ld, o.p, o.ld, w, (float)eps, o.p ? h.data_ptr() : nullptr,
                              r.d, q.data_ptr<int8_t>(), pitch_of(r.d), s.data_ptr<float>(), nullptr, stream(dev));
        }
        check(rc, "qamw_rmsnorm8");
        PyObject* sum = h.defined() ? THPVariable_Wrap(std::move(h)) : Py_NewRef(a[0]);   // without a residual: x
        return tuple({THPVariable_Wrap(std::move(q)), THPVariable_Wrap(std::move(s)), sum});
    });
}

PyObject* gemm8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary(n == 5 && lib.gemm8, [&]() -> PyObject* {
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
            y = make({x.n, w.n}, a[4] == Py_True ? at::kBFloat16 : at::kFloat);
            const size_t need = lib.gemm8_workspace(x.n, w.n, x.d);
            if (need) work = make({(int64_t)need}, at::kByte);
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

// The module: these functions, and those of the 4-bit operators (mx4_host.cpp).
PyMODINIT_FUNC PyInit__w8_host(void) {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddFunctions(m, mx4_methods) < 0) Py_CLEAR(m);
    return m;
}
