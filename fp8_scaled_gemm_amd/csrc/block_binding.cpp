// Python binding of the attention block's operators (fp8g_block.h) on torch
// tensors: the module fp8_scaled_gemm_amd._block.
//
// A decode step calls these operators once a layer with little work each, and
// a call through ctypes costs 13-20 us of host time (measured: twenty attribute
// reads and compares a tensor argument each, 25 conversions, two allocations),
// more than the kernels take.  Here a call costs about 5 us.  Functions take
// every argument by position, check the tensors, allocate outputs and
// workspaces with torch, and queue the library's kernels on torch's current
// stream; block.py gives them their public signatures.  A status other than
// FP8G_OK comes back as an int.

#include <Python.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "fp8g_block.h"

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

struct Cache {
    const Tensor &k, &ks, &v, &vs;
    int64_t pages, heads, page_size, dk, dv;
    Cache(PyObject* const* a, const Call& c)
        : k(tensor(a[0], "cache.k")), ks(tensor(a[1], "cache.k_scale")), v(tensor(a[2], "cache.v")),
          vs(tensor(a[3], "cache.v_scale")) {
        dims(k, "cache.k", 4);
        dims(v, "cache.v", 4);
        pages = k.size(0), heads = k.size(1), page_size = k.size(2), dk = 2 * k.size(3), dv = 2 * v.size(3);
        need(k, "cache.k", at::kByte, {pages, heads, page_size, dk / 2}, c.device);
        need(ks, "cache.k_scale", at::kByte, {pages, heads, dk / 32, page_size}, c.device);
        need(v, "cache.v", at::kByte, {pages, heads, page_size, dv / 2}, c.device);
        need(vs, "cache.v_scale", at::kByte, {pages, heads, dv / 32, page_size}, c.device);
    }
};
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

// base, x, A, B, scale, seg_start, seg_adapter, out, workspace
PyObject* lora_add_(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        arguments(n, 9);
        const Tensor &base = tensor(a[0], "base"), &x = tensor(a[1], "x"), &A = tensor(a[2], "A"), &B = tensor(a[3], "B");
        const Tensor &scale = tensor(a[4], "scale"), &start = tensor(a[5], "seg_start"), &adapter = tensor(a[6], "seg_adapter");
        dims(base, "base", 2);
        dims(x, "x", 2);
        dims(A, "A", 3);
        const Call c;
        const int64_t T = x.size(0), k = x.size(1), cols = base.size(1), N = A.size(0), rank = A.size(1), S = adapter.numel();
        const at::ScalarType dt = base.scalar_type();
        const int code = out_code(dt, "base");
        need(base, "base", dt, {T, cols}, c.device);
        need(x, "x", at::kBFloat16, {T, k}, c.device);
        need(A, "A", at::kBFloat16, {N, rank, k}, c.device);
        need(B, "B", at::kBFloat16, {N, cols, rank}, c.device);
        need(scale, "scale", at::kFloat, {N}, c.device);
        need(start, "seg_start", at::kInt, {S + 1}, c.device);
        need(adapter, "seg_adapter", at::kInt, {S}, c.device);
        const Tensor out = output(a[7], "out", dt, {T, cols}, c);
        const Workspace ws(a[8], lora_add_workspace(T, cols, k, rank, N, S), c);
        const int st = lora_add(base.data_ptr(), x.data_ptr(), A.data_ptr(), B.data_ptr(), scale.data_ptr<float>(),
                                start.data_ptr<int32_t>(), adapter.data_ptr<int32_t>(), T, cols, k, rank, N, S, code,
                                out.data_ptr(), ws.ptr, ws.bytes, c.stream);
        return st ? PyLong_FromLong(st) : THPVariable_Wrap(out);
    });
}

// q, k, q_weight, k_weight, positions, cos_sin, axis, eps, interleaved, q_out, k_out
PyObject* qk_norm_rope_(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        arguments(n, 11);
        const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &pos = tensor(a[4], "positions"), &table = tensor(a[5], "cos_sin");
        dims(q, "q", 3);
        dims(k, "k", 3);
        dims(table, "cos_sin", 2);
        const Call c;
        const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2), Hk = k.size(1), P = table.size(0), rotary = table.size(1);
        const at::ScalarType dt = q.scalar_type();
        const int code = out_code(dt, "q");
        need(q, "q", dt, {T, Hq, D}, c.device, false);
        need(k, "k", dt, {T, Hk, D}, c.device, false);
        const float *wq = nullptr, *wk = nullptr;
        if (given(a[2])) {
            need(tensor(a[2], "q_weight"), "q_weight", at::kFloat, {D}, c.device);
            wq = tensor(a[2], "q_weight").data_ptr<float>();
        }
        if (given(a[3])) {
            need(tensor(a[3], "k_weight"), "k_weight", at::kFloat, {D}, c.device);
            wk = tensor(a[3], "k_weight").data_ptr<float>();
        }
        const int64_t axes = pos.dim() == 1 ? 1 : pos.size(0);
        if (pos.dim() == 1) need(pos, "positions", at::kInt, {T}, c.device);
        else need(pos, "positions", at::kInt, {axes, T}, c.device);
        need(table, "cos_sin", at::kFloat, {P, rotary}, c.device);
        const int32_t* axis = nullptr;
        if (given(a[6])) {
            need(tensor(a[6], "axis"), "axis", at::kInt, {rotary / 2}, c.device);
            axis = tensor(a[6], "axis").data_ptr<int32_t>();
        } else if (axes > 1) {
            throw std::invalid_argument("positions of several axes need axis, the axis of each pair");
        }
        const float eps = real(a[7]);
        const Tensor qo = output(a[9], "q_out", dt, {T, Hq, D}, c, false), ko = output(a[10], "k_out", dt, {T, Hk, D}, c, false);
        const int st = qk_norm_rope(q.data_ptr(), rows(q, "q"), k.data_ptr(), rows(k, "k"), code, T, Hq, Hk, D, wq, wk, eps,
                                    pos.data_ptr<int32_t>(), axes, axis, table.data_ptr<float>(), P, rotary, truth(a[8]),
                                    qo.data_ptr(), rows(qo, "q_out"), ko.data_ptr(), rows(ko, "k_out"), c.stream);
        return st ? PyLong_FromLong(st) : pair(qo, ko);
    });
}

// cache (4), k, v, slots
PyObject* kv4_append_(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        arguments(n, 7);
        const Call c;
        const Cache cache(a, c);
        const Tensor &k = tensor(a[4], "k"), &v = tensor(a[5], "v"), &slots = tensor(a[6], "slots");
        dims(k, "k", 3);
        const int64_t T = k.size(0);
        const at::ScalarType dt = k.scalar_type();
        const int code = out_code(dt, "k") == FP8G_OUT_F32 ? FP8G_IN_F32 : FP8G_IN_BF16;
        need(k, "k", dt, {T, cache.heads, cache.dk}, c.device, false);
        need(v, "v", dt, {T, cache.heads, cache.dv}, c.device, false);
        need(slots, "slots", at::kLong, {T}, c.device);
        const int st = kv4_append(k.data_ptr(), rows(k, "k"), v.data_ptr(), rows(v, "v"), code, T, cache.heads, cache.dk,
                                  cache.dv, slots.data_ptr<int64_t>(), cache.pages, cache.page_size, bytes_of(cache.k),
                                  bytes_of(cache.ks), bytes_of(cache.v), bytes_of(cache.vs), c.stream);
        if (st) return PyLong_FromLong(st);
        Py_RETURN_NONE;
    });
}

// cache (4), slots, k_out, v_out, float32
PyObject* kv4_gather_(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        arguments(n, 8);
        const Call c;
        const Cache cache(a, c);
        const Tensor& slots = tensor(a[4], "slots");
        const int64_t T = slots.numel();
        const bool f32 = truth(a[7]);
        const at::ScalarType dt = f32 ? at::kFloat : at::kBFloat16;
        need(slots, "slots", at::kLong, {T}, c.device);
        const Tensor k = output(a[5], "k_out", dt, {T, cache.heads, cache.dk}, c), v = output(a[6], "v_out", dt, {T, cache.heads, cache.dv}, c);
        const int st = kv4_gather(bytes_of(cache.k), bytes_of(cache.ks), bytes_of(cache.v), bytes_of(cache.vs), cache.pages,
                                  cache.page_size, cache.heads, cache.dk, cache.dv, slots.data_ptr<int64_t>(), T,
                                  f32 ? FP8G_OUT_F32 : FP8G_OUT_BF16, k.data_ptr(), v.data_ptr(), c.stream);
        return st ? PyLong_FromLong(st) : pair(k, v);
    });
}

// q, cache (4), page_table, q_start, kv_len, scale, causal, window, out, lse, return_lse, workspace
PyObject* kv4_attention_(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        arguments(n, 15);
        const Call c;
        const Tensor& q = tensor(a[0], "q");
        const Cache cache(a + 1, c);
        const Tensor &table = tensor(a[5], "page_table"), &start = tensor(a[6], "q_start"), &length = tensor(a[7], "kv_len");
        dims(q, "q", 3);
        dims(table, "page_table", 2);
        const int64_t Tq = q.size(0), Hq = q.size(1), B = length.numel(), most = table.size(1);
        need(q, "q", at::kBFloat16, {Tq, Hq, cache.dk}, c.device, false);
        need(table, "page_table", at::kInt, {B, most}, c.device);
        need(start, "q_start", at::kInt, {B + 1}, c.device);
        need(length, "kv_len", at::kInt, {B}, c.device);
        const float scale = given(a[8]) ? real(a[8]) : (float)(1.0 / std::sqrt((double)cache.dk));
        const int64_t window = integer(a[10]);
        const Tensor out = output(a[11], "out", at::kBFloat16, {Tq, Hq, cache.dv}, c);
        const bool with_lse = given(a[12]) || truth(a[13]);
        Tensor lse;
        if (with_lse) lse = output(a[12], "lse", at::kFloat, {Tq, Hq}, c);
        const Workspace ws(a[14], kv4_attention_workspace(Tq, Hq, cache.heads, cache.dk, cache.dv, B, most, cache.page_size, window), c);
        const int st = kv4_attention(q.data_ptr(), rows(q, "q"), Tq, Hq, bytes_of(cache.k), bytes_of(cache.ks), bytes_of(cache.v),
                                     bytes_of(cache.vs), cache.pages, cache.page_size, cache.heads, cache.dk, cache.dv,
                                     table.data_ptr<int32_t>(), B, most, start.data_ptr<int32_t>(), length.data_ptr<int32_t>(),
                                     scale, truth(a[9]), window, out.data_ptr(), with_lse ? lse.data_ptr<float>() : nullptr,
                                     ws.ptr, ws.bytes, c.stream);
        if (st) return PyLong_FromLong(st);
        return with_lse ? pair(out, lse) : THPVariable_Wrap(out);
    });
}

PyMethodDef methods[] = {
    {"lora_add", (PyCFunction)(void (*)())lora_add_, METH_FASTCALL, nullptr},
    {"qk_norm_rope", (PyCFunction)(void (*)())qk_norm_rope_, METH_FASTCALL, nullptr},
    {"kv4_append", (PyCFunction)(void (*)())kv4_append_, METH_FASTCALL, nullptr},
    {"kv4_gather", (PyCFunction)(void (*)())kv4_gather_, METH_FASTCALL, nullptr},
    {"kv4_attention", (PyCFunction)(void (*)())kv4_attention_, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block() { return PyModule_Create(&module); }
