// Python binding of the attention block's operators (fp8g_block.h) on torch
// tensors, and the module fp8_scaled_gemm_amd._block, which also holds the
// feed-forward half's (ffn_binding.cpp).
//
// A decode step calls these operators once a layer with little work each, and
// a call through ctypes costs 13-20 us of host time (measured: twenty attribute
// reads and compares a tensor argument each, 25 conversions, two allocations),
// more than the kernels take.  Here a call costs about 5 us.  Functions take
// every argument by position, check the tensors, allocate outputs and
// workspaces with torch, and queue the library's kernels on torch's current
// stream; block.py and ffn.py give them their public signatures.  A status other than
// FP8G_OK comes back as an int.

#include "binding.h"
#include "fp8g_block.h"

PyObject* norm_quantize_(PyObject*, PyObject* const*, Py_ssize_t);     // ffn_binding.cpp
PyObject* gemm_fused_(PyObject*, PyObject* const*, Py_ssize_t);
PyObject* moe_route_(PyObject*, PyObject* const*, Py_ssize_t);
PyObject* moe_gemm_(PyObject*, PyObject* const*, Py_ssize_t);
PyObject* moe_combine_(PyObject*, PyObject* const*, Py_ssize_t);

namespace {

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
    {"norm_quantize", (PyCFunction)(void (*)())norm_quantize_, METH_FASTCALL, nullptr},
    {"gemm_fused", (PyCFunction)(void (*)())gemm_fused_, METH_FASTCALL, nullptr},
    {"moe_route", (PyCFunction)(void (*)())moe_route_, METH_FASTCALL, nullptr},
    {"moe_gemm", (PyCFunction)(void (*)())moe_gemm_, METH_FASTCALL, nullptr},
    {"moe_combine", (PyCFunction)(void (*)())moe_combine_, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block() { return PyModule_Create(&module); }
