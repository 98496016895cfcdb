// step_call.cpp -- the marshalling of the calls around the mixers of a decode step (norm_rms, w4_quantize,
// w4_linear, spec_probs, spec_verify), as a Python extension.
//
// One row's norm or projection takes two or three microseconds on the GPU, less than a check of its tensors in
// Python.  As in attn_call.cpp nothing is computed here: tensors are checked, outputs that were not passed are
// allocated, and libssm's entry point (include/ssm.h) is called with pointers, strides and the current stream.
// Each function returns its outputs, or the library's negative status as an int.
#include "call.h"

namespace {

using namespace ssm_call;

decltype(&norm_rms) f_norm = nullptr;
decltype(&w4_quantize) f_quantize = nullptr;
decltype(&w4_linear_workspace_bytes) f_linear_bytes = nullptr;
decltype(&w4_linear) f_linear = nullptr;
decltype(&spec_probs) f_probs = nullptr;
decltype(&spec_verify) f_verify = nullptr;

// A [rows, columns] view with contiguous columns.  The stride of a single row moves nothing, so it is given as
// one that the library accepts for any element size.
struct Rows {
    int64_t n = 0, w = 0, st = 0;
    void* p = nullptr;
};
Rows rows(const at::Tensor& t, const char* name) {
    if (t.dim() != 2) value_error(std::string(name) + " must have two dimensions");
    Rows r;
    r.n = t.size(0), r.w = t.size(1), r.st = t.stride(0);
    if (t.stride(1) != 1 && r.w > 1) value_error(std::string(name) + " must have contiguous rows");
    if (r.n <= 1) r.st = (r.w + 15) / 16 * 16;
    r.p = t.data_ptr();
    return r;
}
Rows rows(PyObject* o, const char* name, const at::Tensor& like, const char* as) {
    const at::Tensor& t = cuda_tensor(o, name);
    if (t.sizes() != like.sizes()) value_error(std::string(name) + " must be shaped like " + as);
    return rows(t, name);
}
// A contiguous tensor of one type and shape.
void* exactly(const at::Tensor& t, at::ScalarType s, at::IntArrayRef shape, const char* name, const char* what) {
    if (t.scalar_type() != s || t.sizes() != shape || !t.is_contiguous())
        value_error(std::string(name) + " must be contiguous " + what);
    return t.data_ptr();
}

// (x, weight, residual, eps, n_groups, out, out_dtype, residual_out, out_scale, stream)
PyObject* do_norm(PyObject* const* a) {
    const Place on(a, {{0, "x"}, {1, "weight"}, {2, "residual"}, {5, "out"}, {7, "residual_out"}, {8, "out_scale"}}, a[9]);
    const at::Tensor& x = cuda_tensor(a[0], "x");
    const Rows xv = rows(x, "x");
    const int64_t groups = integer(a[4], "n_groups");
    const float* weight = nullptr;
    if (given(a[1])) weight = static_cast<const float*>(exactly(cuda_tensor(a[1], "weight"), at::kFloat, {xv.w}, "weight", "float32 [width]"));
    ssm_dtype_t res_code = SSM_BF16;
    Rows rv, ro;
    at::Tensor r_out;
    if (given(a[2])) {
        const at::Tensor& r = cuda_tensor(a[2], "residual");
        rv = rows(a[2], "residual", x, "x");
        res_code = out_code(r.scalar_type());
        if (a[7] != Py_False) {
            if (given(a[7])) {
                r_out = cuda_tensor(a[7], "residual_out");
                need_type(r_out, r.scalar_type(), "residual_out", "of residual's dtype");
                ro = rows(a[7], "residual_out", x, "x");
            } else {
                r_out = on.fresh(x.sizes(), r.scalar_type(), x);
                ro = rows(r_out, "residual_out");
            }
        }
    } else if (given(a[7]) && a[7] != Py_False) {
        value_error("residual_out needs residual");
    }
    const at::Tensor out = given(a[5]) ? cuda_tensor(a[5], "out") : on.fresh(x.sizes(), scalar_type(a[6]), x);
    if (out.sizes() != x.sizes()) value_error("out must be shaped like x");
    const bool i8 = out.scalar_type() == at::kChar;
    const ssm_dtype_t code = i8 ? SSM_I8 : out_code(out.scalar_type());
    const Rows ov = rows(out, "out");
    at::Tensor scale;
    if (i8) {
        const int64_t shape[2] = {xv.n, groups};
        if (groups < 1) value_error("n_groups must be positive");
        scale = given(a[8]) ? cuda_tensor(a[8], "out_scale") : on.fresh(shape, at::kFloat, x);
        exactly(scale, at::kFloat, at::IntArrayRef(shape, 2), "out_scale", "float32 [rows, n_groups]");
    } else if (given(a[8])) {
        value_error("out_scale goes with an int8 out");
    }
    const int rc = f_norm(xv.n, as_int(xv.w, "width"), as_int(groups, "n_groups"), out_code(x.scalar_type()), xv.p, xv.st, res_code,
                          rv.p, rv.st, ro.p, ro.st, weight, (float)number(a[3], "eps"), code, ov.p, ov.st,
                          i8 ? static_cast<float*>(scale.data_ptr()) : nullptr, on.stream());
    return rc ? PyLong_FromLong(rc) : several({out, r_out, scale});
}

int64_t rounded(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// (W, group, zeros, scale_dtype, stream)
PyObject* do_quantize(PyObject* const* a) {
    const Place on(a, {{0, "W"}}, a[4]);
    const at::Tensor& W = cuda_tensor(a[0], "W");
    const Rows wv = rows(W, "W");
    const int64_t group = integer(a[1], "group");
    const bool zeros = truth(a[2], "zeros");
    if (group < 1 || wv.w % group != 0 || wv.w % 2 != 0) value_error("K must be a multiple of the group");
    const at::ScalarType st = scalar_type(a[3]);
    const ssm_dtype_t sc = out_code(st);
    const int64_t groups = wv.w / group;
    // rows start on 16 bytes
    const at::Tensor codes = on.fresh({wv.n, rounded(wv.w / 2, 16)}, at::kByte, W).narrow(1, 0, wv.w / 2);
    const at::Tensor scales = on.fresh({wv.n, rounded(groups, sc == SSM_BF16 ? 8 : 4)}, st, W).narrow(1, 0, groups);
    at::Tensor z;
    if (zeros) z = on.fresh({wv.n, rounded(groups, 16)}, at::kByte, W).narrow(1, 0, groups);
    const int rc = f_quantize(wv.n, wv.w, as_int(group, "group"), out_code(W.scalar_type()), wv.p, std::max(wv.st, wv.w),
                              static_cast<uint8_t*>(codes.data_ptr()), codes.stride(0), sc, scales.data_ptr(), scales.stride(0),
                              zeros ? static_cast<uint8_t*>(z.data_ptr()) : nullptr, zeros ? z.stride(0) : 0, on.stream());
    return rc ? PyLong_FromLong(rc) : several({codes, scales, z});
}

// Rows of scales or zeros: read up to the next 16 bytes, which have to be the tensor's own memory.
Rows grouped(const at::Tensor& t, int64_t n, int64_t groups, const char* name) {
    if (t.dim() != 2 || t.size(0) != n || t.size(1) != groups)
        value_error(std::string(name) + " must be [N, K / group] like scales");
    const Rows r = rows(t, name);
    const int64_t e = (int64_t)t.element_size();
    const int64_t most = (int64_t)t.storage().nbytes() - t.storage_offset() * e;
    if ((n > 1 ? (n - 1) * r.st * e : 0) + rounded(groups * e, 16) > most)
        value_error(std::string(name) + " must be readable up to a multiple of 16 bytes in its last row: pad its rows");
    return r;
}

// (x, codes, scales, zeros, x_scale, out, out_dtype, workspace, stream)
PyObject* do_linear(PyObject* const* a) {
    const Place on(a, {{0, "x"}, {1, "codes"}, {2, "scales"}, {3, "zeros"}, {4, "x_scale"}, {5, "out"}, {7, "workspace"}}, a[8]);
    const at::Tensor &x = cuda_tensor(a[0], "x"), &codes = cuda_tensor(a[1], "codes"), &scales = cuda_tensor(a[2], "scales");
    const Rows xv = rows(x, "x"), cv = rows(codes, "codes");
    need_type(codes, at::kByte, "codes", "uint8");
    if (xv.w != 2 * cv.w) value_error("x must be [M, K] and codes [N, K / 2]");
    if (scales.dim() != 2 || scales.size(1) < 1 || xv.w % scales.size(1) != 0) value_error("scales must be [N, K / group]");
    const int64_t groups = scales.size(1);
    const ssm_dtype_t sc = out_code(scales.scalar_type());
    const Rows sv = grouped(scales, cv.n, groups, "scales");
    Rows zv;
    if (given(a[3])) {
        const at::Tensor& z = cuda_tensor(a[3], "zeros");
        need_type(z, at::kByte, "zeros", "uint8");
        zv = grouped(z, cv.n, groups, "zeros");
    }
    const bool i8 = x.scalar_type() == at::kChar;
    const ssm_dtype_t xc = i8 ? SSM_I8 : out_code(x.scalar_type());
    int64_t blocks = 1;
    const float* xs = nullptr;
    if (given(a[4])) {
        const at::Tensor& s = cuda_tensor(a[4], "x_scale");
        if (s.scalar_type() != at::kFloat || s.dim() < 1 || s.dim() > 2 || s.size(0) != xv.n || !s.is_contiguous())
            value_error("x_scale must be contiguous float32 [M] or [M, blocks]");
        blocks = s.dim() == 2 ? s.size(1) : 1;
        xs = static_cast<const float*>(s.data_ptr());
    }
    if (i8 != given(a[4])) value_error(i8 ? "x_scale is needed for int8 x" : "x_scale goes with int8 x");
    const int64_t shape[2] = {xv.n, cv.n};
    const at::Tensor out = given(a[5]) ? cuda_tensor(a[5], "out") : on.fresh(at::IntArrayRef(shape, 2), scalar_type(a[6]), x);
    if (out.sizes() != at::IntArrayRef(shape, 2)) value_error("out must be [M, N]");
    const Rows ov = rows(out, "out");
    const int group = as_int(xv.w / groups, "group");
    at::Tensor ws;
    if (given(a[7])) {
        ws = cuda_tensor(a[7], "workspace");
        if (!ws.is_contiguous()) value_error("workspace must be contiguous");
    } else {
        const size_t need = f_linear_bytes(xv.n, cv.n, xv.w, group);
        if (need) ws = on.scratch({(int64_t)need}, at::kByte, x);
    }
    const int rc = f_linear(xv.n, cv.n, xv.w, group, xc, xv.p, xv.st, xs, as_int(blocks, "x_blocks"),
                            static_cast<const uint8_t*>(cv.p), cv.st, sc, sv.p, sv.st, static_cast<const uint8_t*>(zv.p), zv.st,
                            out_code(out.scalar_type()), ov.p, ov.st, ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? (size_t)ws.nbytes() : 0,
                            on.stream());
    return rc ? PyLong_FromLong(rc) : several({out});
}

// (logits, temperature, out, stream)
PyObject* do_probs(PyObject* const* a) {
    const Place on(a, {{0, "logits"}, {1, "temperature"}, {2, "out"}}, a[3]);
    const at::Tensor& x = cuda_tensor(a[0], "logits");
    const Rows xv = rows(x, "logits");
    const ssm_dtype_t xc = out_code(x.scalar_type());
    const float* t = nullptr;
    if (given(a[1])) t = static_cast<const float*>(exactly(cuda_tensor(a[1], "temperature"), at::kFloat, {xv.n}, "temperature", "float32 [rows]"));
    const at::Tensor out = given(a[2]) ? cuda_tensor(a[2], "out") : on.fresh(x.sizes(), at::kFloat, x);
    if (out.sizes() != x.sizes() || out.scalar_type() != at::kFloat) value_error("out must be float32, shaped like logits");
    const Rows ov = rows(out, "out");
    const int rc = f_probs(xv.n, xv.w, xc, xv.p, xv.st, t, static_cast<float*>(ov.p), ov.st, on.stream());
    return rc ? PyLong_FromLong(rc) : several({out});
}

// Probabilities [batch, places, vocab] with contiguous rows.
struct Table {
    const float* p = nullptr;
    int64_t sb = 0, st = 0;
};
Table table(const at::Tensor& t, int64_t batch, int64_t places, int64_t vocab, const char* name) {
    if (t.scalar_type() != at::kFloat || t.dim() != 3 || t.size(0) != batch || t.size(1) != places || t.size(2) != vocab ||
        (t.stride(2) != 1 && vocab > 1))
        value_error(std::string(name) + " must be float32 [batch, " + std::to_string(places) + ", vocab] with contiguous rows");
    Table v;
    v.p = static_cast<const float*>(t.data_ptr());
    v.st = places > 1 ? t.stride(1) : vocab;
    v.sb = batch > 1 ? t.stride(0) : vocab;
    return v;
}

// (draft, target_probs, u, draft_probs, n_draft, tokens, n_kept, stream)
PyObject* do_verify(PyObject* const* a) {
    const Place on(a, {{1, "target_probs"}, {0, "draft"}, {2, "u"}, {3, "draft_probs"}, {4, "n_draft"}, {5, "tokens"}, {6, "n_kept"}}, a[7]);
    const at::Tensor &p = cuda_tensor(a[1], "target_probs"), &d = cuda_tensor(a[0], "draft"), &u = cuda_tensor(a[2], "u");
    if (p.dim() != 3 || p.size(1) < 1) value_error("target_probs must be [batch, drafts + 1, vocab]");
    const int64_t batch = p.size(0), n = p.size(1) - 1, vocab = p.size(2);
    const Table pv = table(p, batch, n + 1, vocab, "target_probs");
    const auto* draft = static_cast<const int32_t*>(exactly(d, at::kInt, {batch, n}, "draft", "int32 [batch, drafts]"));
    const auto* up = static_cast<const float*>(exactly(u, at::kFloat, {batch, n + 1}, "u", "float32 [batch, drafts + 1]"));
    Table qv;
    if (given(a[3])) qv = table(cuda_tensor(a[3], "draft_probs"), batch, n, vocab, "draft_probs");
    const int32_t* count = nullptr;
    if (given(a[4])) count = static_cast<const int32_t*>(exactly(cuda_tensor(a[4], "n_draft"), at::kInt, {batch}, "n_draft", "int32 [batch]"));
    const at::Tensor tokens = given(a[5]) ? cuda_tensor(a[5], "tokens") : on.fresh({batch, n + 1}, at::kInt, p);
    auto* tp = static_cast<int32_t*>(exactly(tokens, at::kInt, {batch, n + 1}, "tokens", "int32 [batch, drafts + 1]"));
    const at::Tensor kept = given(a[6]) ? cuda_tensor(a[6], "n_kept") : on.fresh({batch}, at::kInt, p);
    auto* kp = static_cast<int32_t*>(exactly(kept, at::kInt, {batch}, "n_kept", "int32 [batch]"));
    const int rc = f_verify(as_int(batch, "batch"), as_int(n, "drafts"), vocab, draft, count, pv.p, pv.sb, pv.st, qv.p, qv.sb,
                            qv.st, up, tp, kp, on.stream());
    return rc ? PyLong_FromLong(rc) : several({tokens, kept});
}

// bind(addresses of norm_rms, w4_quantize, w4_linear_workspace_bytes, w4_linear, spec_probs, spec_verify)
PyObject* do_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void* p[6];
    if (!addresses(a, n, p, 6)) return nullptr;
    f_norm = reinterpret_cast<decltype(f_norm)>(p[0]);
    f_quantize = reinterpret_cast<decltype(f_quantize)>(p[1]);
    f_linear_bytes = reinterpret_cast<decltype(f_linear_bytes)>(p[2]);
    f_linear = reinterpret_cast<decltype(f_linear)>(p[3]);
    f_probs = reinterpret_cast<decltype(f_probs)>(p[4]);
    f_verify = reinterpret_cast<decltype(f_verify)>(p[5]);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", fast(do_bind), METH_FASTCALL, "Take libssm's entry points."},
    {"norm", fast(guarded<do_norm, 10>), METH_FASTCALL, "norm_rms"},
    {"quantize", fast(guarded<do_quantize, 5>), METH_FASTCALL, "w4_quantize"},
    {"linear", fast(guarded<do_linear, 9>), METH_FASTCALL, "w4_linear"},
    {"probs", fast(guarded<do_probs, 4>), METH_FASTCALL, "spec_probs"},
    {"verify", fast(guarded<do_verify, 8>), METH_FASTCALL, "spec_verify"},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_step_call", "Marshalling of the calls around a decode step's mixers.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__step_call() { return PyModule_Create(&module); }
