// binding.hpp -- what the Python bindings of the operators beside the state update share:
// checks of tensors, the call into the library, the Python entry.
//
// Every function raises ValueError for inconsistent arguments, NotImplementedError for
// valid ones that the library does not implement. Nothing here reads device data.
#pragma once

#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <string>

#include "ssu.h"

namespace binding {

using at::Tensor;

struct Error {
    PyObject* kind;
    std::string text;
};

[[noreturn]] inline void value_error(const std::string& text) { throw Error{PyExc_ValueError, text}; }
[[noreturn]] inline void unsupported(const std::string& text) {
    throw Error{PyExc_NotImplementedError, text};
}

inline std::string list(at::IntArrayRef v) {
    std::string s = "[";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + "]";
}

inline std::string name_of(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return "torch.float32";
        case at::kHalf: return "torch.float16";
        case at::kBFloat16: return "torch.bfloat16";
        default: return std::string("torch.") + at::toString(t);
    }
}

// A required tensor, or an optional one (None: an undefined tensor).
inline const Tensor& tensor(const char* name, PyObject* o) {
    if (!THPVariable_Check(o)) value_error(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

inline const Tensor& optional(const char* name, PyObject* o) {
    static const Tensor none;
    return o == Py_None ? none : tensor(name, o);
}

inline void on_gpu(const char* name, const Tensor& t) {
    if (!t.is_cuda()) value_error(std::string(name) + " must be on a GPU, got " + t.device().str());
}

inline void same_device(const char* name, const Tensor& t, at::Device device) {
    if (t.defined() && t.device() != device)
        value_error(std::string(name) + " is on " + t.device().str() + ", expected " + device.str());
}

inline int32_t io_code(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return SSU_F32;
        case at::kHalf: return SSU_F16;
        case at::kBFloat16: return SSU_BF16;
        default: return -1;
    }
}

inline void* pointer(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// Whether the dimensions of t after the first are dense. A dimension of size 1 has any stride.
inline bool dense_inside(const Tensor& t, int64_t* size) {
    int64_t dense = 1;
    for (int64_t d = t.dim() - 1; d >= 1; --d) {
        if (t.size(d) != 1 && t.stride(d) != dense) return false;
        dense *= t.size(d);
    }
    *size = dense;
    return true;
}

// Element stride between the rows of an operand of this shape and type whose rows are dense.
inline int64_t rows_of(const char* name, const Tensor& t, at::IntArrayRef shape, at::ScalarType dtype) {
    if (t.sizes() != shape)
        value_error(std::string(name) + " must be " + list(shape) + ", got " + list(t.sizes()));
    if (t.scalar_type() != dtype)
        value_error(std::string(name) + " must be " + name_of(dtype) + ", got " +
                    name_of(t.scalar_type()));
    int64_t size;
    if (!dense_inside(t, &size) && t.numel() > 0)
        value_error(std::string(name) + "'s rows must be contiguous, got strides " +
                    list(t.strides()));
    return shape[0] > 1 ? t.stride(0) : size;
}

// Element stride between the slots of a cache whose slots are dense inside.
inline int64_t slots_of(const char* name, const Tensor& t) {
    int64_t size;
    if (!dense_inside(t, &size) && t.numel() > 0)
        value_error(std::string(name) + "'s slots must be contiguous inside, got strides " +
                    list(t.strides()));
    return t.size(0) > 1 ? t.stride(0) : size;
}

inline void vector(const char* name, const Tensor& t, int64_t n, at::ScalarType dtype) {
    if (!t.defined()) return;
    if (t.dim() != 1 || t.size(0) != n)
        value_error(std::string(name) + " must be [" + std::to_string(n) + "], got " +
                    list(t.sizes()));
    if (t.scalar_type() != dtype)
        value_error(std::string(name) + " must be " + name_of(dtype) + ", got " +
                    name_of(t.scalar_type()));
    if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
}

// The index dtype code of a contiguous 1-D tensor of ids.
inline int32_t ids_of(const char* name, const Tensor& t, at::Device device) {
    if (t.scalar_type() != at::kInt && t.scalar_type() != at::kLong)
        value_error(std::string(name) + " must be int32 or int64, got " + name_of(t.scalar_type()));
    if (t.dim() != 1) value_error(std::string(name) + " must be 1-D, got " + list(t.sizes()));
    same_device(name, t, device);
    if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
    return t.scalar_type() == at::kLong ? SSU_I64 : SSU_I32;
}

inline Tensor output(PyObject* o, const Tensor& x, int64_t rows, int64_t dim, int64_t* stride) {
    Tensor out = o == Py_None ? at::empty({rows, dim}, x.options()) : tensor("out", o);
    same_device("out", out, x.device());
    *stride = rows_of("out", out, {rows, dim}, x.scalar_type());
    return out;
}

// The sequences of a call: packed ones with cu_seqlens, else one per row.
template <typename Args>
inline void sequences(Args& a, const Tensor& cu, const Tensor& has, const Tensor& slots, int64_t rows,
               int64_t nslots, at::Device device) {
    a.nseq = rows;
    if (cu.defined()) {
        a.cu_dtype = ids_of("cu_seqlens", cu, device);
        if (cu.size(0) < 1) value_error("cu_seqlens must be a 1-D [sequences + 1] tensor");
        a.nseq = cu.size(0) - 1;
        a.cu_seqlens = cu.data_ptr();
        if (has.defined()) {
            if (has.scalar_type() != at::kBool && has.scalar_type() != at::kByte)
                value_error("has_initial_state must be bool, got " + name_of(has.scalar_type()));
            vector("has_initial_state", has, a.nseq, has.scalar_type());
            same_device("has_initial_state", has, device);
            a.has_initial = static_cast<const uint8_t*>(has.data_ptr());
        }
    }
    if (slots.defined()) {
        a.slot_dtype = ids_of("state_batch_indices", slots, device);
        if (slots.size(0) != a.nseq)
            value_error("state_batch_indices must be [" + std::to_string(a.nseq) + "], got " +
                        list(slots.sizes()));
        a.slots = slots.data_ptr();
    } else if (a.nseq > nslots) {
        value_error(std::to_string(a.nseq) + " sequences need as many slots without "
                    "state_batch_indices, got " + std::to_string(nslots));
    }
}

// The tensors' GPU is made the current one for the call: a default stream's handle names the
// default stream of whichever GPU is current.
template <typename Args>
inline void call(const char* entry, int (*f)(const Args*, void*), const Args& a, at::Device device) {
    c10::OptionalDeviceGuard guard;
    if (c10::hip::current_device() != device.index()) guard.reset_device(device);
    void* stream = c10::hip::getCurrentHIPStream(device.index()).stream();
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f(&a, stream);
    Py_END_ALLOW_THREADS
    if (rc == SSU_OK) return;
    const std::string text = std::string(entry) + ": " + ssu_last_error();
    if (rc == SSU_ERR_INVALID_ARGUMENT) value_error(text);
    if (rc == SSU_ERR_UNSUPPORTED) unsupported(text);
    throw Error{PyExc_RuntimeError, text + " (status " + std::to_string(rc) + ")"};
}

inline int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Error{nullptr, ""};
    return v;
}

// Python entry of `f` with `count` positional arguments: no C++ exception leaves it. torch's
// become what they are from any of its functions (torch.OutOfMemoryError among them).
template <PyObject* (*f)(PyObject* const*), Py_ssize_t count>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        if (n != count) throw Error{PyExc_TypeError, "wrong number of arguments"};
        return f(args);
    } catch (const Error& e) {
        if (e.kind) PyErr_SetString(e.kind, e.text.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*f)(PyObject* const*), Py_ssize_t count>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, count>)),
            METH_FASTCALL, nullptr};
}

}  // namespace binding
