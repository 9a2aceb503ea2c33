// What the binding's compiled ways share (w8_host.cpp, mx4_host.cpp): the checks of tensors, the outputs, the
// interpreter's lock, and the way back to Python.
#pragma once
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/EmptyTensor.h>
#include <ATen/hip/impl/HIPCachingAllocatorMasqueradingAsCUDA.h>
#include <ATen/record_function.h>
#include <c10/core/GradMode.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "qamw.h"

namespace host {

using at::Tensor;

struct Skip {};     // not an ordinary call
struct Raised {};   // a Python error is set

inline PyObject* failed = nullptr;   // failed(return code, function) raises

// The answer of the library: done, or a refusal, before anything was queued (w8.py gives its reason), or an
// error of the runtime.
inline void check(int rc, const char* name) {
    if (rc == QAMW_OK) return;
    if (rc == QAMW_ERR_ARG || rc == QAMW_ERR_UNSUPPORTED || rc == QAMW_ERR_WORKSPACE) throw Skip{};
    Py_XDECREF(PyObject_CallFunction(failed, "is", rc, name));
    throw Raised{};
}

inline const Tensor& tensor(PyObject* o) {
    if (!THPVariable_CheckExact(o)) throw Skip{};
    return THPVariable_Unpack(o);
}

inline void on(const Tensor& t, int device) {
    if (!t.is_cuda() || t.get_device() != device || t.layout() != at::kStrided) throw Skip{};
}

struct Rows {
    const void* p;
    int32_t n, d;
    int64_t ld;
};

// A bf16 or fp32 matrix with contiguous rows, of the size and type of `like`.
inline Rows rows(const Tensor& t, int device, const Tensor* like = nullptr) {
    on(t, device);
    if (t.dim() != 2 || (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kFloat)) throw Skip{};
    const int64_t n = t.size(0), d = t.size(1), ld = t.stride(0);
    if (n < 1 || d < 1 || n > INT32_MAX || d > INT32_MAX || t.stride(1) != 1 || ld < d) throw Skip{};
    if (like && (like->size(0) != n || like->size(1) != d || like->scalar_type() != t.scalar_type())) throw Skip{};
    return {t.const_data_ptr(), (int32_t)n, (int32_t)d, ld};
}

inline const float* vec(const Tensor& t, int device, int64_t n) {
    on(t, device);
    if (t.scalar_type() != at::kFloat || t.numel() < n || !t.is_contiguous()) throw Skip{};
    return t.const_data_ptr<float>();
}

// The tensor's device, which is the current one.
inline int current_of(const Tensor& t) {
    if (!t.is_cuda() || t.get_device() != c10::hip::current_device()) throw Skip{};
    return t.get_device();
}

inline void* stream(int device) { return c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream(); }

inline qamw_dtype dtype(const Tensor& t) { return t.scalar_type() == at::kBFloat16 ? QAMW_BF16 : QAMW_F32; }

// Whether somebody watches or fills new tensors: a dispatch mode, a profiler, or deterministic algorithms, under which
// memory that nothing has written yet holds NaN.
inline bool watched() {
    const auto& context = at::globalContext();
    return c10::impl::dispatch_mode_enabled() || at::hasCallbacks() ||
           (context.deterministicAlgorithms() && context.deterministicFillUninitializedMemory());
}

// An output on the current device, made by at::empty where that is watched, and otherwise as at::empty makes it at the end
// of its way through the dispatcher; that way takes as long again (quant4 of a row, calls one behind the other: 4.8 us
// with it, 4.3 without).
inline Tensor make(at::IntArrayRef size, at::ScalarType type) {
    if (watched()) return at::empty(size, at::TensorOptions().device(at::kCUDA).dtype(type));
    return at::detail::empty_generic(size, c10::hip::HIPCachingAllocatorMasqueradingAsCUDA::get(),
                                     c10::DispatchKeySet(c10::DispatchKey::CUDA), type, std::nullopt);
}

// A tuple of new references; null if one of them is.
inline PyObject* tuple(std::initializer_list<PyObject*> items) {
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

// What f gives, or None for a call that is not an ordinary one.
template <typename F>
PyObject* ordinary(bool as_expected, F&& f) {
    HANDLE_TH_ERRORS
    try {
        if (!as_expected) throw Skip{};
        return f();
    } catch (const Skip&) {
        Py_RETURN_NONE;
    } catch (const Raised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

}  // namespace host
