// attn_call.cpp -- the marshalling of the attention calls, as a Python extension.
//
// A decode step or a short prompt takes a few microseconds on the GPU; checking a dozen tensors and
// converting thirty arguments in Python takes longer.  This module does exactly what a Python
// binding would: check the tensors, allocate the outputs that were not passed, and call libssm's
// entry point (include/ssm.h) with device pointers, element strides and the current stream.  It
// computes nothing.  Each function returns its outputs, or the library's negative status as an int.
#include "call.h"

namespace {

using namespace ssm_call;

decltype(&attn_append) f_append = nullptr;
decltype(&attn_cache_read) f_read = nullptr;
decltype(&attn_prefill) f_prefill = nullptr;
decltype(&attn_decode_workspace_bytes) f_decode_bytes = nullptr;
decltype(&attn_decode_step) f_decode = nullptr;

// A [tokens, heads, dim] view.  A stride along an extent of one moves nothing, so it is given as a
// value the library accepts.
struct View {
    int64_t n = 0, h = 0, d = 0, st = 0, sh = 0;
    void* p = nullptr;
};
View view(const at::Tensor& t, const char* name) {
    if (t.dim() != 3) value_error(std::string(name) + " must be [tokens, heads, head_dim]");
    View v;
    v.n = t.size(0), v.h = t.size(1), v.d = t.size(2);
    v.st = t.stride(0), v.sh = t.stride(1);
    if (t.stride(2) != 1 && v.d > 1) value_error(std::string(name) + " must have channel stride 1");
    if (v.h == 1) v.sh = v.d;
    if (v.n <= 1) v.st = v.h * v.sh;
    v.p = t.data_ptr();
    return v;
}
int32_t* int32s(PyObject* o, int64_t n, const char* name) {
    const at::Tensor& t = cuda_tensor(o, name);
    if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
        value_error(std::string(name) + " must be contiguous int32 [" + std::to_string(n) + "]");
    return static_cast<int32_t*>(t.data_ptr());
}
struct Cache {
    ssm_dtype_t code;
    int n_pages, h, page, d;
    void *k, *v;
    float *ks = nullptr, *vs = nullptr;
};
Cache cache(PyObject* ko, PyObject* vo, PyObject* kso, PyObject* vso) {
    const at::Tensor &k = tensor(ko, "k_cache"), &v = tensor(vo, "v_cache");
    Cache c;
    if (k.scalar_type() == at::kChar) c.code = SSM_I8;
    else if (k.scalar_type() == at::kBFloat16) c.code = SSM_BF16;
    else throw TypeProblem("unsupported cache dtype (int8 or bfloat16)");
    if (k.dim() != 4 || v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type() || !k.is_contiguous() ||
        !v.is_contiguous() || !k.is_cuda() || !v.is_cuda())
        value_error("k_cache and v_cache must be contiguous CUDA tensors of one shape "
                    "[n_pages, kv_heads, page_size, head_dim] and one dtype");
    c.n_pages = as_int(k.size(0), "n_pages"), c.h = as_int(k.size(1), "kv_heads");
    c.page = as_int(k.size(2), "page_size"), c.d = as_int(k.size(3), "head_dim");
    c.k = k.data_ptr(), c.v = v.data_ptr();
    if (c.code == SSM_I8) {
        float** to[2] = {&c.ks, &c.vs};
        PyObject* from[2] = {kso, vso};
        for (int i = 0; i < 2; ++i) {
            const char* name = i ? "v_scale" : "k_scale";
            if (!given(from[i])) value_error(std::string(name) + " is needed for an int8 cache");
            const at::Tensor& s = cuda_tensor(from[i], name);
            if (s.scalar_type() != at::kFloat || s.dim() != 3 || s.sizes() != k.sizes().slice(0, 3) || !s.is_contiguous())
                value_error(std::string(name) + " must be contiguous float32 [n_pages, kv_heads, page_size]");
            *to[i] = static_cast<float*>(s.data_ptr());
        }
    } else if (given(kso) || given(vso)) {
        value_error("a bfloat16 cache has no scales");
    }
    return c;
}

struct Table {
    int32_t* p;
    int64_t stride;
    int n;
};
Table table(PyObject* o, int64_t batch) {
    const at::Tensor& t = tensor(o, "page_table");
    if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != batch || (t.stride(1) != 1 && t.size(1) > 1) || !t.is_cuda())
        value_error("page_table must be an int32 CUDA tensor [batch, pages] with contiguous rows");
    const int n = as_int(t.size(1), "page_table");
    return Table{static_cast<int32_t*>(t.data_ptr()), batch > 1 ? t.stride(0) : std::max<int64_t>(n, 1), n};
}

// The attention output: given, shaped like q, or made.
at::Tensor attn_out(PyObject* o, PyObject* dtype, const at::Tensor& q, const Place& on) {
    if (!given(o)) return on.fresh(q.sizes(), scalar_type(dtype), q);
    const at::Tensor& t = cuda_tensor(o, "out");
    if (t.sizes() != q.sizes()) value_error("out must be shaped like q");
    return t;
}
// The lse tensor to write: given, made for True, or none.
at::Tensor attn_lse(PyObject* o, const at::Tensor& q, const Place& on) {
    if (!given(o) || o == Py_False) return at::Tensor();
    if (o == Py_True) return on.fresh(q.sizes().slice(0, 2), at::kFloat, q);
    const at::Tensor& t = cuda_tensor(o, "lse");
    if (t.scalar_type() != at::kFloat || t.sizes() != q.sizes().slice(0, 2) || !t.is_contiguous())
        value_error("lse must be contiguous float32 [tokens, heads]");
    return t;
}

// (q, k, v, positions, cos, sin, k_cache, v_cache, slots, k_scale, v_scale, interleaved, q_out, k_out, stream)
PyObject* do_append(PyObject* const* a) {
    const Place on(a, {{1, "k"}, {0, "q"}, {2, "v"}, {3, "positions"}, {4, "cos"}, {5, "sin"}, {6, "k_cache"}, {7, "v_cache"},
                          {8, "slots"}, {9, "k_scale"}, {10, "v_scale"}, {12, "q_out"}, {13, "k_out"}}, a[14]);
    const bool inter = truth(a[11], "interleaved");
    const Cache c = cache(a[6], a[7], a[9], a[10]);
    const at::Tensor &k = cuda_tensor(a[1], "k"), &v = cuda_tensor(a[2], "v");
    need_type(k, at::kBFloat16, "k", "bfloat16");
    need_type(v, at::kBFloat16, "v", "bfloat16");
    const View kv = view(k, "k"), vv = view(v, "v");
    if (kv.h != c.h || kv.d != c.d || vv.h != c.h || vv.d != c.d || vv.n != kv.n)
        value_error("k and v must be [tokens, kv_heads, head_dim] of the cache");
    const int32_t* slots = int32s(a[8], kv.n, "slots");
    int64_t n_pos = 0, half = 0;
    const float *cp = nullptr, *sp = nullptr;
    const int32_t* positions = nullptr;
    if (given(a[4])) {
        const at::Tensor &cs = cuda_tensor(a[4], "cos"), &sn = cuda_tensor(a[5], "sin");
        if (cs.scalar_type() != at::kFloat || sn.scalar_type() != at::kFloat || cs.dim() != 2 || sn.sizes() != cs.sizes() ||
            !cs.is_contiguous() || !sn.is_contiguous())
            value_error("cos and sin must be contiguous float32 [n_pos, half]");
        n_pos = cs.size(0), half = cs.size(1);
        cp = static_cast<const float*>(cs.data_ptr()), sp = static_cast<const float*>(sn.data_ptr());
        positions = int32s(a[3], kv.n, "positions");
    }
    View qv, qo, ko;
    at::Tensor q_out, k_out;
    if (given(a[0])) {
        const at::Tensor& q = cuda_tensor(a[0], "q");
        need_type(q, at::kBFloat16, "q", "bfloat16");
        qv = view(q, "q");
        if (qv.n != kv.n || qv.d != c.d) value_error("q must be [tokens, heads, head_dim]");
        if (given(a[12])) {
            q_out = cuda_tensor(a[12], "q_out");
            if (q_out.scalar_type() != at::kBFloat16 || q_out.sizes() != q.sizes()) value_error("q_out must be shaped like q, bfloat16");
        } else {
            q_out = on.fresh(q.sizes(), at::kBFloat16, q);
        }
        qo = view(q_out, "q_out");
    } else if (given(a[12])) {
        value_error("q_out needs q");
    }
    if (given(a[13]) && a[13] != Py_False) {
        if (a[13] == Py_True) {
            k_out = on.fresh(k.sizes(), at::kBFloat16, k);
        } else {
            k_out = cuda_tensor(a[13], "k_out");
            if (k_out.scalar_type() != at::kBFloat16 || k_out.sizes() != k.sizes()) value_error("k_out must be shaped like k, bfloat16");
        }
        ko = view(k_out, "k_out");
    }
    const int rc = f_append(kv.n, as_int(qv.p || given(a[0]) ? qv.h : c.h, "heads"), c.h, c.d, as_int(2 * half, "rot_dim"), inter,
                            qv.p, qv.st, qv.sh, kv.p, kv.st, kv.sh, vv.p, vv.st, vv.sh, positions, cp, sp, n_pos, slots,
                            c.code, c.k, c.v, c.ks, c.vs, c.n_pages, c.page, qo.p, qo.st, qo.sh, ko.p, ko.st, ko.sh, on.stream());
    return rc ? PyLong_FromLong(rc) : several({q_out, k_out});
}

// (k_cache, v_cache, page_table, cu_len, n_tokens, k_scale, v_scale, first, k_out, v_out, out_dtype, stream)
PyObject* do_read(PyObject* const* a) {
    const Place on(a, {{0, "k_cache"}, {1, "v_cache"}, {2, "page_table"}, {3, "cu_len"}, {5, "k_scale"}, {6, "v_scale"},
                          {7, "first"}, {8, "k_out"}, {9, "v_out"}}, a[11]);
    const Cache c = cache(a[0], a[1], a[5], a[6]);
    const at::Tensor& kc = THPVariable_Unpack(a[0]);
    const int64_t batch = cuda_tensor(a[3], "cu_len").numel() - 1, n = integer(a[4], "n_tokens");
    if (n < 0) value_error("n_tokens must not be negative");
    const int32_t* cu = int32s(a[3], batch + 1, "cu_len");
    const int32_t* first = given(a[7]) ? int32s(a[7], batch, "first") : nullptr;
    const Table tb = table(a[2], batch);
    const int64_t shape[3] = {n, c.h, c.d};
    at::Tensor k = given(a[8]) ? cuda_tensor(a[8], "k_out") : on.fresh(shape, scalar_type(a[10]), kc);
    at::Tensor v = given(a[9]) ? cuda_tensor(a[9], "v_out") : on.fresh(shape, k.scalar_type(), kc);
    if (k.sizes() != at::IntArrayRef(shape, 3) || v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type() ||
        !k.is_contiguous() || !v.is_contiguous())
        value_error("k_out and v_out must be contiguous [n_tokens, kv_heads, head_dim] of one dtype");
    const int rc = f_read(as_int(batch, "batch"), n, c.h, c.d, c.code, c.k, c.v, c.ks, c.vs, c.n_pages, c.page, tb.p, tb.stride,
                          tb.n, cu, first, out_code(k.scalar_type()), k.data_ptr(), v.data_ptr(), on.stream());
    return rc ? PyLong_FromLong(rc) : several({k, v});
}

double scale_of(PyObject* o, int64_t d) { return given(o) ? number(o, "scale") : 1.0 / std::sqrt((double)d); }

// (q, k, v, cu_q, cu_k, max_q, scale, out, out_dtype, lse, stream)
PyObject* do_prefill(PyObject* const* a) {
    const Place on(a, {{0, "q"}, {1, "k"}, {2, "v"}, {3, "cu_q"}, {4, "cu_k"}, {7, "out"}, {9, "lse"}}, a[10]);
    const at::Tensor &q = cuda_tensor(a[0], "q"), &k = cuda_tensor(a[1], "k"), &v = cuda_tensor(a[2], "v");
    const View qv = view(q, "q"), kv = view(k, "k"), vv = view(v, "v");
    if (kv.d != qv.d || vv.d != qv.d || vv.h != kv.h || vv.n != kv.n)
        value_error("k and v must be [tokens, kv_heads, head_dim] of one shape, with q's head_dim");
    if (k.scalar_type() != q.scalar_type() || v.scalar_type() != q.scalar_type()) value_error("q, k and v must share one dtype");
    const int64_t batch = cuda_tensor(a[3], "cu_q").numel() - 1;
    const int32_t *cq = int32s(a[3], batch + 1, "cu_q"), *ck = int32s(a[4], batch + 1, "cu_k");
    const at::Tensor out = attn_out(a[7], a[8], q, on), lse = attn_lse(a[9], q, on);
    const View ov = view(out, "out");
    const int rc = f_prefill(as_int(batch, "batch"), qv.n, kv.n, as_int(integer(a[5], "max_q"), "max_q"), as_int(qv.h, "heads"),
                             as_int(kv.h, "kv_heads"), as_int(qv.d, "head_dim"), out_code(q.scalar_type()),
                             out_code(out.scalar_type()), qv.p, qv.st, qv.sh, kv.p, kv.st, kv.sh, vv.p, vv.st, vv.sh, cq, ck,
                             (float)scale_of(a[6], qv.d), ov.p, ov.st, ov.sh,
                             lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr, on.stream());
    return rc ? PyLong_FromLong(rc) : several({out, lse});
}

// (q, k_cache, v_cache, page_table, lens, max_len, k_scale, v_scale, scale, out, out_dtype, lse, workspace, stream)
PyObject* do_decode(PyObject* const* a) {
    const Place on(a, {{0, "q"}, {1, "k_cache"}, {2, "v_cache"}, {3, "page_table"}, {4, "lens"}, {6, "k_scale"},
                          {7, "v_scale"}, {9, "out"}, {11, "lse"}, {12, "workspace"}}, a[13]);
    const Cache c = cache(a[1], a[2], a[6], a[7]);
    const at::Tensor& q = cuda_tensor(a[0], "q");
    const View qv = view(q, "q");
    if (qv.d != c.d) value_error("q must be [batch, heads, head_dim] with the cache's head_dim");
    const int32_t* lens = int32s(a[4], qv.n, "lens");
    const int max_len = as_int(integer(a[5], "max_len"), "max_len"), batch = as_int(qv.n, "batch"), heads = as_int(qv.h, "heads");
    const Table tb = table(a[3], qv.n);
    const at::Tensor out = attn_out(a[9], a[10], q, on), lse = attn_lse(a[11], q, on);
    const View ov = view(out, "out");
    at::Tensor ws;
    if (given(a[12])) {
        ws = cuda_tensor(a[12], "workspace");
        if (!ws.is_contiguous()) value_error("workspace must be contiguous");
    } else {
        const size_t need = f_decode_bytes(batch, heads, c.h, c.d, max_len);
        if (need) ws = on.scratch({(int64_t)need}, at::kByte, q);
    }
    const int rc = f_decode(batch, heads, c.h, c.d, out_code(q.scalar_type()), out_code(out.scalar_type()), qv.p, qv.st, qv.sh,
                            c.code, c.k, c.v, c.ks, c.vs, c.n_pages, c.page, tb.p, tb.stride, tb.n, lens, max_len,
                            (float)scale_of(a[8], c.d), ov.p, ov.st, ov.sh,
                            lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr,
                            ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? (size_t)ws.nbytes() : 0, on.stream());
    return rc ? PyLong_FromLong(rc) : several({out, lse});
}

// bind(addresses of attn_append, attn_cache_read, attn_prefill, attn_decode_workspace_bytes, attn_decode_step)
PyObject* do_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void* p[5];
    if (!addresses(a, n, p, 5)) return nullptr;
    f_append = reinterpret_cast<decltype(f_append)>(p[0]);
    f_read = reinterpret_cast<decltype(f_read)>(p[1]);
    f_prefill = reinterpret_cast<decltype(f_prefill)>(p[2]);
    f_decode_bytes = reinterpret_cast<decltype(f_decode_bytes)>(p[3]);
    f_decode = reinterpret_cast<decltype(f_decode)>(p[4]);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", fast(do_bind), METH_FASTCALL, "Take libssm's entry points."},
    {"append", fast(guarded<do_append, 15>), METH_FASTCALL, "attn_append"},
    {"read", fast(guarded<do_read, 12>), METH_FASTCALL, "attn_cache_read"},
    {"prefill", fast(guarded<do_prefill, 11>), METH_FASTCALL, "attn_prefill"},
    {"decode", fast(guarded<do_decode, 14>), METH_FASTCALL, "attn_decode_step"},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn_call", "Marshalling of the attention calls.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__attn_call() { return PyModule_Create(&module); }
