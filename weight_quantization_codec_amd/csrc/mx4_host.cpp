// The ordinary calls of the 4-bit operators, without the interpreter between their checks, as w8_host.cpp has those of
// the 8-bit ones: a function here returns None for every other call, before anything is queued, and mx4.py does it.
//
// Calls one behind the other, one row (us, in the interpreter and here): quant4 8.4 and 4.3, dequant4 7.4 and 3.7,
// rmsnorm4 with a residual 11 and 5.0, gemm4 10 and 4.4.
#include "host_calls.hpp"
#include "qamw_mx4.h"

extern PyMethodDef mx4_methods[];

namespace {

using namespace host;

struct Entry {
    decltype(&qamw_quant4) quant4;
    decltype(&qamw_dequant4) dequant4;
    decltype(&qamw_rmsnorm4) rmsnorm4;
    decltype(&qamw_gemm4_workspace) gemm4_workspace;
    decltype(&qamw_gemm4) gemm4;
    decltype(&qamw_gemm4_grouped) gemm4_grouped;
} lib;

int64_t groups_of(int64_t d) { return (d + 255) / 256; }

struct Form {
    const uint8_t *q, *e;
    int32_t n, groups;
    int64_t ld_q, ld_e;
};

// Codes (rows x whole groups) and their scales (groups x rows x 8).
Form form(const Tensor& q, const Tensor& e, int device) {
    on(q, device);
    on(e, device);
    if (q.dim() != 2 || q.scalar_type() != at::kByte || e.dim() != 3 || e.scalar_type() != at::kByte) throw Skip{};
    const int64_t n = q.size(0), b = q.size(1), g = b / 128;
    if (n < 1 || b < 1 || b % 128 || n > INT32_MAX || b > INT32_MAX || q.stride(1) != 1 || q.stride(0) < b) throw Skip{};
    if (e.size(0) != g || e.size(1) != n || e.size(2) != 8 || e.stride(2) != 1 || e.stride(1) != 8) throw Skip{};
    // (a dimension of size 1 may have any stride: the library takes what a packed matrix has)
    const int64_t ld_q = n > 1 ? q.stride(0) : b, ld_e = g > 1 ? e.stride(0) : 8 * n;
    const auto* pq = static_cast<const uint8_t*>(q.const_data_ptr());
    const auto* pe = static_cast<const uint8_t*>(e.const_data_ptr());
    if (ld_q % 16 || ld_e % 8 || ld_e < 8 * n || (uintptr_t)pq % 16 || (uintptr_t)pe % 8) throw Skip{};
    return {pq, pe, (int32_t)n, (int32_t)g, ld_q, ld_e};
}

const int32_t* ints(const Tensor& t, int device, int64_t n) {
    on(t, device);
    if (t.scalar_type() != at::kInt || t.numel() < n || !t.is_contiguous()) throw Skip{};
    return t.const_data_ptr<int32_t>();
}

void make_form(int64_t n, int64_t d, Tensor& q, Tensor& e) {
    q = make({n, 128 * groups_of(d)}, at::kByte);
    e = make({groups_of(d), n, 8}, at::kByte);
}

PyObject* quant4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary(n == 3 && lib.gemm4, [&]() -> PyObject* {
        const Tensor& x = tensor(a[0]);
        const int dev = current_of(x);
        const Rows r = rows(x, dev);
        const float* scale = a[1] == Py_None ? nullptr : vec(tensor(a[1]), dev, r.d);
        Rows g{nullptr, 0, 0, 0};
        if (a[2] != Py_None) g = rows(tensor(a[2]), dev, &x);
        Tensor q, e;
        int rc;
        {
            const Unlocked unlocked;
            make_form(r.n, r.d, q, e);
            rc = lib.quant4(r.p, dtype(x), r.n, r.d, r.ld, g.p, g.ld, scale, q.data_ptr<uint8_t>(), q.size(1),
                            e.data_ptr<uint8_t>(), 8ll * r.n, nullptr, stream(dev));
        }
        check(rc, "qamw_quant4");
        return tuple({THPVariable_Wrap(std::move(q)), THPVariable_Wrap(std::move(e))});
    });
}

PyObject* dequant4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary(n == 5 && lib.gemm4, [&]() -> PyObject* {
        const Tensor& q = tensor(a[0]);
        const int dev = current_of(q);
        const Form f = form(q, tensor(a[1]), dev);
        if (!PyLong_CheckExact(a[2])) throw Skip{};
        int over = 0;
        const int64_t d = PyLong_AsLongLongAndOverflow(a[2], &over);
        if (over || d < 1 || groups_of(d) != f.groups) throw Skip{};
        const float* scale = a[3] == Py_None ? nullptr : vec(tensor(a[3]), dev, d);
        Tensor y;
        int rc;
        {
            const Unlocked unlocked;
            y = make({f.n, d}, a[4] == Py_True ? at::kBFloat16 : at::kFloat);
            rc = lib.dequant4(f.q, f.n, (int32_t)d, f.ld_q, f.e, f.ld_e, scale, y.data_ptr(), dtype(y), d, stream(dev));
        }
        check(rc, "qamw_dequant4");
        return THPVariable_Wrap(std::move(y));
    });
}

PyObject* rmsnorm4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary(n == 4 && lib.gemm4, [&]() -> PyObject* {
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
        Tensor h, q, e;
        int rc;
        {
            const Unlocked unlocked;
            if (o.p) h = make({r.n, r.d}, x.scalar_type());
            make_form(r.n, r.d, q, e);
            rc = lib.rmsnorm4(r.p, dtype(x), r.n, r.d, r.ld, o.p, o.ld, w, (float)eps, o.p ? h.data_ptr() : nullptr,
                              r.d, q.data_ptr<uint8_t>(), q.size(1), e.data_ptr<uint8_t>(), 8ll * r.n, nullptr, stream(dev));
        }
        check(rc, "qamw_rmsnorm4");
        PyObject* sum = h.defined() ? THPVariable_Wrap(std::move(h)) : Py_NewRef(a[0]);   // without a residual: x
        return tuple({THPVariable_Wrap(std::move(q)), THPVariable_Wrap(std::move(e)), sum});
    });
}

PyObject* gemm4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary(n == 5 && lib.gemm4, [&]() -> PyObject* {
        const Tensor& xq = tensor(a[0]);
        const int dev = current_of(xq);
        const Form x = form(xq, tensor(a[1]), dev), w = form(tensor(a[2]), tensor(a[3]), dev);
        if (x.groups != w.groups) throw Skip{};
        Tensor y, work;
        int rc;
        {
            const Unlocked unlocked;
            y = make({x.n, w.n}, a[4] == Py_True ? at::kBFloat16 : at::kFloat);
            const size_t need = lib.gemm4_workspace(x.n, w.n, x.groups);
            if (need) work = make({(int64_t)need}, at::kByte);
            rc = lib.gemm4(x.q, x.ld_q, x.e, x.ld_e, x.n, w.q, w.ld_q, w.e, w.ld_e, w.n, x.groups, y.data_ptr(), dtype(y),
                           w.n, need ? work.data_ptr() : nullptr, need, stream(dev));
        }
        check(rc, "qamw_gemm4");
        return THPVariable_Wrap(std::move(y));
    });
}

PyObject* gemm4_grouped(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary(n == 7 && lib.gemm4, [&]() -> PyObject* {
        const Tensor& xq = tensor(a[0]);
        const int dev = current_of(xq);
        const Form x = form(xq, tensor(a[1]), dev);
        const Tensor &wq = tensor(a[2]), &we = tensor(a[3]);
        on(wq, dev);
        on(we, dev);
        if (wq.dim() != 3 || wq.scalar_type() != at::kByte || we.dim() != 4 || we.scalar_type() != at::kByte) throw Skip{};
        const int64_t E = wq.size(0), N = wq.size(1), ld_w = wq.stride(1), by = wq.stride(0);
        const int64_t ld_we = x.groups > 1 ? we.stride(0) : 8 * N, eby = we.stride(1);
        if (E < 1 || N < 1 || E > INT32_MAX || N > INT32_MAX || wq.size(2) != 128ll * x.groups || wq.stride(2) != 1)
            throw Skip{};
        if (we.size(0) != x.groups || we.size(1) != E || we.size(2) != N || we.size(3) != 8 || we.stride(3) != 1 ||
            we.stride(2) != 8)
            throw Skip{};
        const auto* pw = static_cast<const uint8_t*>(wq.const_data_ptr());
        const auto* pe = static_cast<const uint8_t*>(we.const_data_ptr());
        if (ld_w < wq.size(2) || ld_w % 16 || by % 16 || ld_we % 8 || ld_we < 8 * N || eby % 8 || (uintptr_t)pw % 16 ||
            (uintptr_t)pe % 8)
            throw Skip{};
        const int32_t* offsets = ints(tensor(a[4]), dev, E + 1);
        const int32_t* index = nullptr;
        int64_t many = x.n;
        if (a[5] != Py_None) {
            const Tensor& t = tensor(a[5]);
            index = ints(t, dev, 1);
            many = t.numel();
            if (many > INT32_MAX) throw Skip{};
        }
        Tensor y;
        int rc;
        {
            const Unlocked unlocked;
            y = make({many, N}, a[6] == Py_True ? at::kBFloat16 : at::kFloat);
            rc = lib.gemm4_grouped(x.q, x.ld_q, x.e, x.ld_e, x.n, index, (int32_t)many, pw, ld_w, by, pe, ld_we, eby,
                                   offsets, (int32_t)E, (int32_t)N, x.groups, y.data_ptr(), dtype(y), N, stream(dev));
        }
        check(rc, "qamw_gemm4_grouped");
        return THPVariable_Wrap(std::move(y));
    });
}

// bind4(quant4, dequant4, rmsnorm4, gemm4_workspace, gemm4, gemm4_grouped): the library's functions, as addresses.
PyObject* bind4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "bind4 takes 6 addresses");
        return nullptr;
    }
    void* p[6];
    for (Py_ssize_t i = 0; i < 6; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    lib = {(decltype(lib.quant4))p[0], (decltype(lib.dequant4))p[1], (decltype(lib.rmsnorm4))p[2],
           (decltype(lib.gemm4_workspace))p[3], (decltype(lib.gemm4))p[4], (decltype(lib.gemm4_grouped))p[5]};
    Py_RETURN_NONE;
}

}  // namespace

PyMethodDef mx4_methods[] = {
    {"bind4", (PyCFunction)(void (*)(void))bind4, METH_FASTCALL, nullptr},
    {"quant4", (PyCFunction)(void (*)(void))quant4, METH_FASTCALL, nullptr},
    {"dequant4", (PyCFunction)(void (*)(void))dequant4, METH_FASTCALL, nullptr},
    {"rmsnorm4", (PyCFunction)(void (*)(void))rmsnorm4, METH_FASTCALL, nullptr},
    {"gemm4", (PyCFunction)(void (*)(void))gemm4, METH_FASTCALL, nullptr},
    {"gemm4_grouped", (PyCFunction)(void (*)(void))gemm4_grouped, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
