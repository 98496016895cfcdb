// call.h -- what the Python extensions that marshal calls share (attn_call.cpp, step_call.cpp): the checks of
// their arguments, where a call works, how its outputs go back, and the way out for exceptions.
#pragma once

#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/record_function.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <optional>
#include <stdexcept>
#include <string>

#include "ssm.h"

namespace ssm_call {

struct TypeProblem : std::runtime_error {
    using std::runtime_error::runtime_error;
};
[[noreturn]] inline void value_error(const std::string& s) { throw std::invalid_argument(s); }

inline const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw TypeProblem(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
inline const at::Tensor& cuda_tensor(PyObject* o, const char* name) {
    const at::Tensor& t = tensor(o, name);
    if (!t.is_cuda()) value_error(std::string(name) + " must be a CUDA tensor (libssm has no CPU path)");
    return t;
}
inline bool given(PyObject* o) { return o != nullptr && o != Py_None; }

struct Arg {
    int at;
    const char* name;
};
// Where a call works.  The one GPU that its tensors lie on is made current while it allocates and
// launches: the library works on the current device, whatever the pointers are.  A caller's stream is
// made current too: an output or workspace made here then comes from that stream's memory, and what is
// written into it follows whatever still uses that memory there.  (Memory of another stream may be free to
// be handed out on that stream and yet be in use: its last work there need not have run.)
class Place {
public:
    Place(PyObject* const* a, std::initializer_list<Arg> tensors, PyObject* stream) {
        for (const Arg& x : tensors) {
            PyObject* o = a[x.at];
            if (!given(o) || PyBool_Check(o) || !THPVariable_Check(o)) continue;
            const c10::Device d = THPVariable_Unpack(o).device();
            if (!d.is_cuda()) continue;                 // what has to be a CUDA tensor is seen to by name
            const int i = d.index();
            if (index_ >= 0 && i != index_)
                value_error(std::string(x.name) + " is on cuda:" + std::to_string(i) + ", other arguments on cuda:" +
                            std::to_string(index_));
            index_ = i;
        }
        if (index_ < 0) return;
        const auto index = static_cast<c10::DeviceIndex>(index_);
        if (c10::cuda::device_count() > 1 && c10::cuda::current_device() != index) device_.emplace(index);
        const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(index);
        launch_ = current.stream();
        if (!given(stream)) return;
        const unsigned long long raw = PyLong_AsUnsignedLongLong(stream);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            throw TypeProblem("stream must be a CUDA stream");
        }
        auto* handle = reinterpret_cast<cudaStream_t>(static_cast<uintptr_t>(raw));
        if (handle == launch_) return;
        launch_ = handle;
        before_ = current.unwrap();
        stream_.emplace(c10::cuda::getStreamFromExternal(handle, index));
    }
    void* stream() const { return launch_; }
    // Memory of the call's stream, asked for without the dispatcher (a norm's two outputs 1.9 us of 4.2 a call, else 2.5)
    // unless someone looks at what goes through it: a dispatch mode, a profiler, the fill of new memory that goes with
    // deterministic algorithms.
    at::Tensor scratch(at::IntArrayRef shape, at::ScalarType s, const at::Tensor& like) const {
        if (watched_) return at::empty(shape, like.options().dtype(s).memory_format(c10::nullopt).requires_grad(false));
        return at::Tensor(at::detail::empty_cuda(shape, s, like.device(), std::nullopt));
    }
    // An output: the caller goes on with it on the stream that was current, so that is noted as its user.
    at::Tensor fresh(at::IntArrayRef shape, at::ScalarType s, const at::Tensor& like) const {
        at::Tensor t = scratch(shape, s, like);
        if (stream_ && t.numel() > 0) t.record_stream(*before_);
        return t;
    }

private:
    static bool watched() {
        const at::Context& global = at::globalContext();
        return c10::impl::TorchDispatchModeTLS::any_modes_set() || at::hasCallbacks() ||
               (global.deterministicAlgorithms() && global.deterministicFillUninitializedMemory());
    }

    const bool watched_ = watched();
    int index_ = -1;
    cudaStream_t launch_ = nullptr;
    std::optional<c10::cuda::CUDAGuard> device_;
    std::optional<c10::Stream> before_;
    std::optional<c10::cuda::CUDAStreamGuard> stream_;
};

inline void need_type(const at::Tensor& t, at::ScalarType s, const char* name, const char* what) {
    if (t.scalar_type() != s) value_error(std::string(name) + " must be " + what);
}
inline int as_int(int64_t v, const char* name) {
    if (v < INT32_MIN || v > INT32_MAX) value_error(std::string(name) + " does not fit 32 bits");
    return static_cast<int>(v);
}
inline int64_t integer(PyObject* o, const char* name) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw TypeProblem(std::string(name) + " must be an integer");
    }
    return v;
}
inline double number(PyObject* o, const char* name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw TypeProblem(std::string(name) + " must be a number");
    }
    return v;
}
inline bool truth(PyObject* o, const char* name) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) {
        PyErr_Clear();
        throw TypeProblem(std::string(name) + " must be a truth value");
    }
    return v != 0;
}
inline ssm_dtype_t out_code(at::ScalarType s) {
    if (s == at::kFloat) return SSM_F32;
    if (s == at::kBFloat16) return SSM_BF16;
    throw TypeProblem("unsupported dtype (float32 or bfloat16)");
}
inline at::ScalarType scalar_type(PyObject* o) {
    if (!THPDtype_Check(o)) throw TypeProblem("out_dtype must be a torch dtype");
    return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

inline PyObject* wrap(const at::Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

// The outputs of a call as a tuple, None for what was not asked.
inline PyObject* several(std::initializer_list<at::Tensor> ts) {
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    Py_ssize_t i = 0;
    for (const at::Tensor& t : ts) {
        PyObject* x = r ? wrap(t) : nullptr;
        if (!x) {
            Py_XDECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, x);
    }
    return r;
}

// No C++ exception leaves the module.
template <PyObject* (*F)(PyObject* const*), int kArgs>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != kArgs) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", kArgs, n);
        return nullptr;
    }
    try {
        return F(a);
    } catch (const TypeProblem& e) {
        PyErr_SetString(PyExc_TypeError, e.what());
    } catch (const std::invalid_argument& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (...) {                                     // torch's own (out of memory among them)
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

// The addresses of a library's entry points, handed over once by the binding.
inline bool addresses(PyObject* const* a, Py_ssize_t n, void** p, Py_ssize_t want) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%zd addresses expected", want);
        return false;
    }
    for (Py_ssize_t i = 0; i < n; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
            return false;
        }
    }
    return true;
}

template <typename F>
PyCFunction fast(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

}  // namespace ssm_call
