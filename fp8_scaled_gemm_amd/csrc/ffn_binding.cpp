// Python binding of the feed-forward half's operators (fp8g_ffn.h) on torch
// tensors: functions of the module fp8_scaled_gemm_amd._block, in the manner of
// block_binding.cpp.

#include "binding.h"
#include "fp8g_ffn.h"

namespace {

// E4M3 (or E5M2) codes, or their bytes
const Tensor& codes(PyObject* o, const char* name, int fmt = FP8G_FMT_E4M3) {
    const Tensor& t = tensor(o, name);
    const at::ScalarType want = fmt == FP8G_FMT_E5M2 ? at::kFloat8_e5m2 : at::kFloat8_e4m3fn;
    if (t.scalar_type() != want && t.scalar_type() != at::kByte)
        throw TypeErr(std::string(name) + " must be " + c10::toString(want) + " or uint8 codes, got " + c10::toString(t.scalar_type()));
    return t;
}
const uint8_t* bytes_at(const Tensor& t) { return static_cast<const uint8_t*>(t.data_ptr()); }

// elements between the rows of t [R, C], whose rows must be dense
int64_t row_stride(const Tensor& t, const char* name) {
    const int64_t R = t.size(0), C = t.size(1);
    if (C > 1 && t.stride(1) != 1)
        throw std::invalid_argument(std::string(name) + " must be dense within a row (the stride of the row axis is free), got strides " +
                                    text(t.strides()));
    return R > 1 ? t.stride(0) : C;
}

const float* floats(PyObject* o, const char* name, Sizes shape, const Call& c) {
    if (!given(o)) return nullptr;
    const Tensor& t = tensor(o, name);
    need(t, name, at::kFloat, shape, c.device);
    return t.data_ptr<float>();
}

}  // namespace

// x, weight, residual, eps, mx, fmt, sum, norm, q, scale, with_norm
PyObject* norm_quantize_(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        arguments(n, 11);
        const Tensor& x = tensor(a[0], "x");
        dims(x, "x", 2);
        const Call c;
        const int64_t R = x.size(0), C = x.size(1);
        const at::ScalarType dt = x.scalar_type();
        const int code = out_code(dt, "x") == FP8G_OUT_F32 ? FP8G_IN_F32 : FP8G_IN_BF16;
        need(x, "x", dt, {R, C}, c.device, false);
        const float* w = floats(a[1], "weight", {C}, c);
        const void* res = nullptr;
        int64_t res_stride = C;
        if (given(a[2])) {
            const Tensor& r = tensor(a[2], "residual");
            need(r, "residual", dt, {R, C}, c.device, false);
            res = r.data_ptr(), res_stride = row_stride(r, "residual");
        }
        const float eps = real(a[3]);
        const bool mx = truth(a[4]);
        const int fmt = (int)integer(a[5]);
        if (fmt != FP8G_FMT_E4M3 && fmt != FP8G_FMT_E5M2) throw std::invalid_argument("fmt must be FMT_E4M3 or FMT_E5M2");
        if (mx && C % 32) throw std::invalid_argument("the row length must be a multiple of 32 for MXFP8");
        Tensor sum, norm, q, scale;
        if (res || given(a[6])) sum = output(a[6], "sum", dt, {R, C}, c);
        if (given(a[7]) || truth(a[10])) norm = output(a[7], "norm", dt, {R, C}, c);
        if (given(a[8])) {
            q = codes(a[8], "q", fmt);
            need(q, "q", q.scalar_type(), {R, C}, c.device);
        } else {
            q = c.make({R, C}, fmt == FP8G_FMT_E5M2 ? at::kFloat8_e5m2 : at::kFloat8_e4m3fn);
        }
        scale = mx ? output(a[9], "scale", at::kByte, {R, C / 32}, c) : output(a[9], "scale", at::kFloat, {R}, c);
        const int st = add_rms_norm_quantize(x.data_ptr(), row_stride(x, "x"), res, res_stride, code, R, C, w, eps,
                                             mx ? (int)FP8G_SCALE_MX : (int)FP8G_SCALE_PER_ROW, fmt,
                                             sum.defined() ? sum.data_ptr() : nullptr, norm.defined() ? norm.data_ptr() : nullptr,
                                             static_cast<uint8_t*>(q.data_ptr()), scale.data_ptr(), c.stream);
        if (st) return PyLong_FromLong(st);
        PyObject* r = PyTuple_New(4);
        if (!r) return nullptr;
        const Tensor* all[] = {&q, &scale, &sum, &norm};
        for (int i = 0; i < 4; i++) {
            PyObject* o = all[i]->defined() ? THPVariable_Wrap(*all[i]) : Py_NewRef(Py_None);
            if (!o) {
                Py_DECREF(r);
                return nullptr;
            }
            PyTuple_SET_ITEM(r, i, o);
        }
        return r;
    });
}

// m, n, k, A, B, scale_a, scale_b, mx, bias, act, gated, residual, D, float32, workspace
PyObject* gemm_fused_(PyObject*, PyObject* const* a, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        arguments(count, 15);
        const int64_t m = integer(a[0]), n = integer(a[1]), k = integer(a[2]);
        const Tensor &A = codes(a[3], "A"), &B = codes(a[4], "B"), &sa = tensor(a[5], "scale_a"), &sb = tensor(a[6], "scale_b");
        const bool mx = truth(a[7]), gated = truth(a[10]), f32 = truth(a[13]);
        const Call c;
        const int64_t rows = gated ? 2 * n : n;
        if (mx && k % 32) throw std::invalid_argument("k must be a multiple of 32 for MXFP8");
        need(A, "A", A.scalar_type(), {m, k}, c.device);
        need(B, "B", B.scalar_type(), {rows, k}, c.device);
        if (mx) {
            need(sa, "scale_a", at::kByte, {m, k / 32}, c.device);
            need(sb, "scale_b", at::kByte, {rows, k / 32}, c.device);
        } else {
            need(sa, "scale_a", at::kFloat, {m}, c.device);
            need(sb, "scale_b", at::kFloat, {rows}, c.device);
        }
        const float* bias = floats(a[8], "bias", {rows}, c);
        const int act = (int)integer(a[9]);
        const at::ScalarType dt = f32 ? at::kFloat : at::kBFloat16;
        const void* res = nullptr;
        if (given(a[11])) {
            const Tensor& r = tensor(a[11], "residual");
            need(r, "residual", dt, {m, n}, c.device);
            res = r.data_ptr();
        }
        const Tensor D = output(a[12], "D", dt, {m, n}, c);
        const int out = f32 ? FP8G_OUT_F32 : FP8G_OUT_BF16;
        const Workspace ws(a[14], gemm_fused_workspace(m, n, k, gated, mx), c);
        const int st = mx ? mxfp8_gemm_fused(m, n, k, bytes_at(A), bytes_at(B), bytes_at(sa), bytes_at(sb), bias, act, gated, res,
                                             D.data_ptr(), out, ws.ptr, ws.bytes, c.stream)
                          : fp8_gemm_fused(m, n, k, bytes_at(A), bytes_at(B), sa.data_ptr<float>(), sb.data_ptr<float>(), bias,
                                           act, gated, res, D.data_ptr(), out, ws.ptr, ws.bytes, c.stream);
        return st ? PyLong_FromLong(st) : THPVariable_Wrap(D);
    });
}

// logits, top_k, bias, score, groups, top_groups, group_top, renormalize, scale, workspace
PyObject* moe_route_(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        arguments(n, 10);
        const Tensor& x = tensor(a[0], "logits");
        dims(x, "logits", 2);
        const Call c;
        const int64_t T = x.size(0), E = x.size(1), k = integer(a[1]);
        const at::ScalarType dt = x.scalar_type();
        const int code = out_code(dt, "logits") == FP8G_OUT_F32 ? FP8G_IN_F32 : FP8G_IN_BF16;
        need(x, "logits", dt, {T, E}, c.device);
        const float* bias = floats(a[2], "bias", {E}, c);
        if (k < 1 || k > E) throw std::invalid_argument("top_k must be between 1 and the number of experts");
        // one allocation for the five: a decode step calls this once a layer
        const int64_t each = (4 * T * k + 15) / 16 * 16;
        const Tensor all = c.make({4 * each + 4 * (E + 1)}, at::kByte);
        const Tensor ids = part(all, 0, {T, k}, at::kInt), w = part(all, each, {T, k}, at::kFloat);
        const Tensor rows = part(all, 2 * each, {T * k}, at::kInt), slots = part(all, 3 * each, {T, k}, at::kInt);
        const Tensor start = part(all, 4 * each, {E + 1}, at::kInt);
        const Workspace ws(a[9], moe_route_workspace(T, E, k), c);
        const int st = moe_route(x.data_ptr(), code, T, E, k, bias, (int)integer(a[3]), integer(a[4]), integer(a[5]),
                                 integer(a[6]), truth(a[7]), real(a[8]), ids.data_ptr<int32_t>(), w.data_ptr<float>(),
                                 start.data_ptr<int32_t>(), rows.data_ptr<int32_t>(), slots.data_ptr<int32_t>(), ws.ptr,
                                 ws.bytes, c.stream);
        if (st) return PyLong_FromLong(st);
        PyObject* r = PyTuple_New(5);
        if (!r) return nullptr;
        const Tensor* out[] = {&ids, &w, &start, &rows, &slots};
        for (int i = 0; i < 5; i++) {
            PyObject* o = THPVariable_Wrap(*out[i]);
            if (!o) {
                Py_DECREF(r);
                return nullptr;
            }
            PyTuple_SET_ITEM(r, i, o);
        }
        return r;
    });
}

// A, B, scale_a, scale_b, mx, expert_start, rows, bias, act, gated, D, float32, workspace
PyObject* moe_gemm_(PyObject*, PyObject* const* a, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        arguments(count, 13);
        const Tensor &A = codes(a[0], "A"), &B = codes(a[1], "B"), &sa = tensor(a[2], "scale_a"), &sb = tensor(a[3], "scale_b");
        const Tensor& start = tensor(a[5], "expert_start");
        const bool mx = truth(a[4]), gated = truth(a[9]), f32 = truth(a[11]);
        dims(A, "A", 2);
        dims(B, "B", 3);
        const Call c;
        const int64_t Ra = A.size(0), k = A.size(1), E = B.size(0), b_rows = B.size(1), n = gated ? b_rows / 2 : b_rows;
        if (gated && b_rows % 2) throw std::invalid_argument("B must hold as many gate as up rows");
        if (mx && k % 32) throw std::invalid_argument("k must be a multiple of 32 for MXFP8");
        need(A, "A", A.scalar_type(), {Ra, k}, c.device);
        need(B, "B", B.scalar_type(), {E, b_rows, k}, c.device);
        if (mx) {
            need(sa, "scale_a", at::kByte, {Ra, k / 32}, c.device);
            need(sb, "scale_b", at::kByte, {E, b_rows, k / 32}, c.device);
        } else {
            need(sa, "scale_a", at::kFloat, {Ra}, c.device);
            need(sb, "scale_b", at::kFloat, {E, b_rows}, c.device);
        }
        need(start, "expert_start", at::kInt, {E + 1}, c.device);
        const int32_t* rows = nullptr;
        int64_t S = Ra;
        if (given(a[6])) {
            const Tensor& r = tensor(a[6], "rows");
            S = r.numel();
            need(r, "rows", at::kInt, {S}, c.device);
            rows = r.data_ptr<int32_t>();
        }
        const float* bias = floats(a[7], "bias", {E, b_rows}, c);
        const int act = (int)integer(a[8]);
        const Tensor D = output(a[10], "D", f32 ? at::kFloat : at::kBFloat16, {S, n}, c);
        const Workspace ws(a[12], moe_gemm_workspace(S, n, k, E, rows != nullptr, gated, mx), c);
        const int out = f32 ? FP8G_OUT_F32 : FP8G_OUT_BF16;
        const int st = mx ? mxfp8_moe_gemm(S, n, k, E, bytes_at(A), Ra, rows, start.data_ptr<int32_t>(), bytes_at(B), bytes_at(sa),
                                           bytes_at(sb), bias, act, gated, D.data_ptr(), out, ws.ptr, ws.bytes, c.stream)
                          : fp8_moe_gemm(S, n, k, E, bytes_at(A), Ra, rows, start.data_ptr<int32_t>(), bytes_at(B),
                                         sa.data_ptr<float>(), sb.data_ptr<float>(), bias, act, gated, D.data_ptr(), out, ws.ptr,
                                         ws.bytes, c.stream);
        return st ? PyLong_FromLong(st) : THPVariable_Wrap(D);
    });
}

// y, slots, weights, residual, out
PyObject* moe_combine_(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        arguments(n, 5);
        const Tensor &y = tensor(a[0], "y"), &slots = tensor(a[1], "slots"), &w = tensor(a[2], "weights");
        dims(y, "y", 2);
        dims(slots, "slots", 2);
        const Call c;
        const int64_t S = y.size(0), H = y.size(1), T = slots.size(0), k = slots.size(1);
        const at::ScalarType dt = y.scalar_type();
        const int code = out_code(dt, "y");
        need(y, "y", dt, {S, H}, c.device);
        need(slots, "slots", at::kInt, {T, k}, c.device);
        need(w, "weights", at::kFloat, {T, k}, c.device);
        const void* res = nullptr;
        if (given(a[3])) {
            const Tensor& r = tensor(a[3], "residual");
            need(r, "residual", dt, {T, H}, c.device);
            res = r.data_ptr();
        }
        const Tensor out = output(a[4], "out", dt, {T, H}, c);
        const int st = moe_combine(y.data_ptr(), S, slots.data_ptr<int32_t>(), w.data_ptr<float>(), res, code, T, k, H,
                                   out.data_ptr(), c.stream);
        return st ? PyLong_FromLong(st) : THPVariable_Wrap(out);
    });
}
