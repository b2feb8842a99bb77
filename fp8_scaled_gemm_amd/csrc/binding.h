// Argument handling that the files of the Python binding _block share: checked
// tensors, outputs and workspaces from torch's allocator, torch's current
// stream, and C++ exceptions turned into Python errors.
#pragma once

#include <Python.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "fp8g.h"

namespace {

struct TypeErr : std::runtime_error {
    using std::runtime_error::runtime_error;
};

using at::Tensor;
using Sizes = at::IntArrayRef;

std::string text(Sizes s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); i++) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + ")";
}

const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw TypeErr(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
bool given(PyObject* o) { return o != Py_None; }

// t: on the current device, of that dtype and shape, contiguous unless told otherwise
void need(const Tensor& t, const char* name, at::ScalarType dtype, Sizes shape, int device, bool dense = true) {
    if (!t.is_cuda()) throw std::invalid_argument(std::string(name) + " must be a device tensor");
    if (t.get_device() != device)     // the kernels run on the current device and take raw pointers
        throw std::invalid_argument(std::string(name) + " is on cuda:" + std::to_string(t.get_device()) +
                                    " but the current device is cuda:" + std::to_string(device) +
                                    " (call under torch.cuda.device)");
    if (t.scalar_type() != dtype)
        throw TypeErr(std::string(name) + " must be " + c10::toString(dtype) + ", got " + c10::toString(t.scalar_type()));
    if (t.sizes() != shape)
        throw std::invalid_argument(std::string(name) + " must have shape " + text(shape) + ", got " + text(t.sizes()));
    if (dense && !t.is_contiguous()) throw std::invalid_argument(std::string(name) + " must be contiguous");
}
void dims(const Tensor& t, const char* name, int64_t n) {
    if (t.dim() != n) throw std::invalid_argument(std::string(name) + " must have " + std::to_string(n) + " dimensions");
}
// 0: bfloat16, 1: float32 (fp8g_out_t)
int out_code(at::ScalarType t, const char* name) {
    if (t == at::kBFloat16) return FP8G_OUT_BF16;
    if (t == at::kFloat) return FP8G_OUT_F32;
    throw TypeErr(std::string(name) + " must be bfloat16 or float32, got " + c10::toString(t));
}
// elements between the tokens of t [T, H, D], whose rows of one token must be dense
int64_t rows(const Tensor& t, const char* name) {
    const int64_t T = t.size(0), H = t.size(1), D = t.size(2);
    if (H && D && ((D > 1 && t.stride(2) != 1) || (H > 1 && t.stride(1) != D)))
        throw std::invalid_argument(std::string(name) + " must be dense within a token (the stride of the token axis is free), got strides " +
                                    text(t.strides()));
    return T > 1 ? t.stride(0) : H * D;
}

int64_t integer(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw TypeErr("an integer argument is required");
    return v;
}
float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw TypeErr("a number is required");
    return (float)v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw TypeErr("a truth value is required");     // the object's own error stays set
    return v == 1;
}

struct Call {
    int device;
    hipStream_t stream;
    Call() : device(c10::hip::current_device()), stream(c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream()) {}
    Tensor make(Sizes shape, at::ScalarType t) const {
        return at::empty(shape, at::TensorOptions().dtype(t).device(at::kCUDA, (c10::DeviceIndex)device));
    }
};

// A dense tensor of `shape` at byte `at` of a block of bytes that several outputs
// share: one allocation for all of them.
Tensor part(const Tensor& block, int64_t at, Sizes shape, at::ScalarType t) {
    auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(block.storage()), block.key_set(), c10::scalarTypeToTypeMeta(t));
    impl->set_storage_offset(block.storage_offset() + at / (int64_t)c10::elementSize(t));
    impl->set_sizes_contiguous(shape);
    return Tensor(std::move(impl));
}

// The caller's workspace, or one from torch's allocator for this call: freed
// behind the call, its memory is handed out again in stream order.
struct Workspace {
    Tensor own;
    void* ptr = nullptr;
    int64_t bytes = 0;
    Workspace(PyObject* o, int64_t need_bytes, const Call& c) {
        if (given(o)) {
            own = tensor(o, "workspace");
            if (!own.is_cuda() || own.get_device() != c.device || !own.is_contiguous())
                throw std::invalid_argument("workspace must be a contiguous tensor on the current device");
        } else if (need_bytes > 0) {
            own = c.make({need_bytes}, at::kByte);
        } else {
            return;
        }
        ptr = own.data_ptr();
        bytes = own.numel() * own.element_size();
    }
};

// an output: given and checked, or a fresh one
Tensor output(PyObject* o, const char* name, at::ScalarType t, Sizes shape, const Call& c, bool dense = true) {
    if (!given(o)) return c.make(shape, t);
    const Tensor& r = tensor(o, name);
    need(r, name, t, shape, c.device, dense);
    return r;
}

uint8_t* bytes_of(const Tensor& t) { return static_cast<uint8_t*>(t.data_ptr()); }

PyObject* pair(const Tensor& a, const Tensor& b) {
    PyObject *x = THPVariable_Wrap(a), *y = THPVariable_Wrap(b);
    PyObject* r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
}

void arguments(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) throw TypeErr("wrong number of arguments");
}

// Nothing but Python errors leaves a function of the module.
template <class F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (const TypeErr& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, e.what());
    } catch (const std::invalid_argument& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

}  // namespace
