// api.cu -- the extern "C" boundary of libssm (declared in include/ssm.h).
//
// Every entry point validates its arguments on the host, returns a negative
// status (with a message for ssm_last_error) before launching anything when they
// are wrong, and otherwise enqueues its kernels on the caller's stream (one
// kernel; three for a prefill cut into several sequence segments; two for the
// SSD prefill and decode; up to three for w4_linear: x put in order, products,
// the sums of slices).
// No entry point allocates memory or keeps per-call state.
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <cuda.h>

#include "ssm.h"
#include "kernels.h"

namespace ssm {

uint64_t current_context_id() {
    using GetCurrent = CUresult (*)(CUcontext*);
    using GetId = CUresult (*)(CUcontext, unsigned long long*);
    static const GetCurrent get_current = []() -> GetCurrent {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        return cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                       q == cudaDriverEntryPointSuccess
                   ? reinterpret_cast<GetCurrent>(f)
                   : nullptr;
    }();
    static const GetId get_id = []() -> GetId {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        return cudaGetDriverEntryPointByVersion("cuCtxGetId", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                       q == cudaDriverEntryPointSuccess
                   ? reinterpret_cast<GetId>(f)
                   : nullptr;
    }();
    CUcontext c = nullptr;
    unsigned long long id = 0;
    if (!get_current || !get_id || get_current(&c) != CUDA_SUCCESS || c == nullptr ||
        get_id(c, &id) != CUDA_SUCCESS)
        return 0;
    return id;
}

}  // namespace ssm

namespace {

thread_local char g_err[512] = "";

int fail(int code, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return code;
}

// Device status word: SSM_DEV_* bits OR-ed in by kernels.
__device__ unsigned int g_status_word;

ssm::ContextMemo g_status_memo;

// Device address of the status word in the current device's context: a __device__ symbol's
// name in host code is not a device address, so it is asked of the runtime
// (cudaGetSymbolAddress) once per device and context.
unsigned int* status_ptr(int* err) {
    void* p = nullptr;
    if (!g_status_memo.get(&p, [](void** out) {
            return cudaGetSymbolAddress(out, g_status_word) == cudaSuccess && *out != nullptr;
        })) {
        *err = 1;
        return nullptr;
    }
    return static_cast<unsigned int*>(p);
}

}  // namespace

// Scratch of ssm_prefill_segmented_noalloc: a fixed array in the library's own device
// memory, present on every GPU that loads the library until the process exits.
static __device__ __align__(256) unsigned char g_noalloc_scratch[SSM_NOALLOC_SCRATCH_BYTES];

namespace {

ssm::ContextMemo g_noalloc_memo;

// Device address of g_noalloc_scratch in the current device's context.  In host code the
// array's name stands for a host-side shadow, not a device address, so the address is asked of
// the runtime (cudaGetSymbolAddress) with that device current, once per device and context.
void* noalloc_scratch_ptr(int* err) {
    void* p = nullptr;
    if (!g_noalloc_memo.get(&p, [](void** out) {
            return cudaGetSymbolAddress(out, g_noalloc_scratch) == cudaSuccess && *out != nullptr;
        })) {
        *err = 1;
        return nullptr;
    }
    return p;
}

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool dtype_ok(int t) { return t == SSM_F32 || t == SSM_BF16; }
int esize(int t) { return t == SSM_BF16 ? 2 : 4; }

}  // namespace

namespace {

// Shared by ssm_prefill (one segment) and ssm_prefill_segmented.
int prefill_impl(const char* fn, int batch, int seqlen, int d_inner, int d_state, int d_conv,
                 ssm_dtype_t in_dtype, ssm_dtype_t out_dtype,
                 const void* x, const void* z, const void* dt,
                 int64_t in_stride_b, int64_t in_stride_t,
                 const void* Bmat, const void* Cmat,
                 const float* A, const float* Dskip, const float* dt_bias,
                 const float* conv_w, const float* conv_b,
                 const float* conv_state_in, const float* ssm_state_in,
                 int64_t conv_state_ld, int64_t ssm_state_stride_b,
                 void* out, int64_t out_stride_b, int64_t out_stride_t,
                 float* conv_state_out, float* ssm_state_out,
                 int seg_len, void* workspace, size_t workspace_bytes,
                 void* cuda_stream, bool fixed_scratch = false) {
    g_err[0] = 0;
    if (batch < 1 || batch > 65535) return fail(SSM_ERR_INVALID_ARG, "%s: batch %lld not in [1, 65535]", fn, (long long)(batch));
    if (seqlen < 1 || seqlen > (1 << 30)) return fail(SSM_ERR_INVALID_ARG, "%s: seqlen %lld not in [1, 2^30]", fn, (long long)(seqlen));
    if (d_inner < 1) return fail(SSM_ERR_INVALID_ARG, "%s: d_inner %lld < 1", fn, (long long)(d_inner));
    if (!dtype_ok(in_dtype) || !dtype_ok(out_dtype)) return fail(SSM_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (d_state != 16) return fail(SSM_ERR_UNSUPPORTED, "%s: d_state %lld unsupported (16 only)", fn, (long long)(d_state));
    if (d_conv != 4) return fail(SSM_ERR_UNSUPPORTED, "%s: d_conv %lld unsupported (4 only)", fn, (long long)(d_conv));
    if (d_inner % 8 != 0) return fail(SSM_ERR_UNSUPPORTED, "%s: d_inner %lld is not a multiple of 8", fn, (long long)(d_inner));
    if (!x || !z || !dt || !Bmat || !Cmat || !A || !Dskip || !dt_bias || !conv_w || !conv_b || !out ||
        !conv_state_out || !ssm_state_out)
        return fail(SSM_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (in_stride_t < d_inner) return fail(SSM_ERR_INVALID_ARG, "%s: in_stride_t %lld < d_inner", fn, (long long)(in_stride_t));
    if (batch > 1 && in_stride_b < 1) return fail(SSM_ERR_INVALID_ARG, "%s: in_stride_b %lld < 1", fn, (long long)(in_stride_b));
    if (out_stride_t < d_inner) return fail(SSM_ERR_INVALID_ARG, "%s: out_stride_t %lld < d_inner", fn, (long long)(out_stride_t));
    if (batch > 1 && out_stride_b < (int64_t)(seqlen - 1) * out_stride_t + d_inner)
        return fail(SSM_ERR_INVALID_ARG, "%s: out_stride_b %lld lets batch rows overlap", fn, (long long)(out_stride_b));
    if (conv_state_ld < d_inner) return fail(SSM_ERR_INVALID_ARG, "%s: conv_state_ld %lld < d_inner", fn, (long long)(conv_state_ld));
    if (ssm_state_stride_b < 16LL * d_inner)
        return fail(SSM_ERR_INVALID_ARG, "%s: ssm_state_stride_b %lld < 16*d_inner", fn, (long long)(ssm_state_stride_b));
    const int es = esize(in_dtype);
    if (!aligned(x, 16) || !aligned(z, 16) || !aligned(dt, 16) || !aligned(Bmat, 16) || !aligned(Cmat, 16))
        return fail(SSM_ERR_MISALIGNED, "%s: x, z, dt, B and C must be 16-byte aligned", fn);
    if ((in_stride_t * es) % 16 != 0 || (batch > 1 && (in_stride_b * es) % 16 != 0))
        return fail(SSM_ERR_MISALIGNED, "%s: input strides must be multiples of 16 bytes", fn);
    if (!aligned(A, 16) || !aligned(conv_w, 16)) return fail(SSM_ERR_MISALIGNED, "%s: A and conv_w must be 16-byte aligned", fn);
    if (!aligned(ssm_state_out, 8) || (ssm_state_in && !aligned(ssm_state_in, 8)) || ssm_state_stride_b % 2 != 0)
        return fail(SSM_ERR_MISALIGNED, "%s: ssm states must be 8-byte aligned with an even batch stride", fn);
    if (!aligned(out, esize(out_dtype))) return fail(SSM_ERR_MISALIGNED, "%s: out is not element aligned", fn);
    if (seg_len < ssm::kPrefillChunk || seg_len % ssm::kPrefillChunk != 0)
        return fail(SSM_ERR_INVALID_ARG, "%s: seg_len %lld is not a positive multiple of %d", fn, (long long)seg_len,
                    ssm::kPrefillChunk);
    const int64_t n_seg = ((int64_t)seqlen + seg_len - 1) / seg_len;
    if (n_seg > 65535) return fail(SSM_ERR_INVALID_ARG, "%s: %lld segments (at most 65535)", fn, (long long)n_seg);
    if (n_seg > 1 && fixed_scratch) {
        // the library's own array stands in for the workspace; every other argument is valid
        const size_t need = ssm_prefill_workspace_bytes(batch, seqlen, d_inner, seg_len);
        if (need > (size_t)SSM_NOALLOC_SCRATCH_BYTES)
            return fail(SSM_ERR_INVALID_ARG,
                        "%s: these sizes need %zu bytes of scratch and the fixed array holds %zu "
                        "(use a longer seg_len, or ssm_prefill_segmented with a workspace)",
                        fn, need, (size_t)SSM_NOALLOC_SCRATCH_BYTES);
        int err = 0;
        workspace = noalloc_scratch_ptr(&err);
        workspace_bytes = (size_t)SSM_NOALLOC_SCRATCH_BYTES;
        if (err) return fail(SSM_ERR_CUDA, "%s: the scratch array's device address is unavailable", fn);
    }
    if (n_seg > 1) {
        const size_t need = ssm_prefill_workspace_bytes(batch, seqlen, d_inner, seg_len);
        if (!workspace || workspace_bytes < need)
            return fail(SSM_ERR_INVALID_ARG, "%s: workspace of %zu bytes given, %zu needed", fn,
                        workspace ? workspace_bytes : (size_t)0, need);
        if (!aligned(workspace, 16)) return fail(SSM_ERR_MISALIGNED, "%s: workspace must be 16-byte aligned", fn);
    }

    int serr = 0;
    unsigned int* status = status_ptr(&serr);
    if (serr) return fail(SSM_ERR_CUDA, "%s: no usable CUDA device", fn);

    ssm::PrefillLaunch q{};
    q.batch = batch;
    q.in_bf16 = in_dtype == SSM_BF16;
    q.out_bf16 = out_dtype == SSM_BF16;
    q.z = z;
    q.dt = dt;
    q.Bm = Bmat;
    q.Cm = Cmat;
    ssm::PrefillArgs& a = q.args;
    a.seqlen = seqlen;
    a.d_inner = d_inner;
    a.x = x;
    a.in_stride_b = in_stride_b;
    a.in_stride_t = in_stride_t;
    a.A = A;
    a.Dskip = Dskip;
    a.dt_bias = dt_bias;
    a.conv_w = conv_w;
    a.conv_b = conv_b;
    a.conv_state_in = conv_state_in;
    a.ssm_state_in = ssm_state_in;
    a.conv_state_ld = conv_state_ld;
    a.ssm_state_stride_b = ssm_state_stride_b;
    a.out = out;
    a.out_stride_b = out_stride_b;
    a.out_stride_t = out_stride_t;
    a.conv_state_out = conv_state_out;
    a.ssm_state_out = ssm_state_out;
    a.status = status;
    a.seg_len = n_seg > 1 ? seg_len : seqlen;
    a.n_seg = (int)n_seg;
    a.ws = n_seg > 1 ? static_cast<float*>(workspace) : nullptr;
    const char* why = "";
    if (ssm::launch_prefill(q, static_cast<cudaStream_t>(cuda_stream), &why) != 0)
        return fail(SSM_ERR_CUDA, "%s: %s", fn, why);
    return SSM_OK;
}


}  // namespace

extern "C" {

int ssm_abi_version(void) { return 108; }

const char* ssm_last_error(void) { return g_err; }

int ssm_prefill(int batch, int seqlen, int d_inner, int d_state, int d_conv,
                ssm_dtype_t in_dtype, ssm_dtype_t out_dtype,
                const void* x, const void* z, const void* dt,
                int64_t in_stride_b, int64_t in_stride_t,
                const void* Bmat, const void* Cmat,
                const float* A, const float* Dskip, const float* dt_bias,
                const float* conv_w, const float* conv_b,
                const float* conv_state_in, const float* ssm_state_in,
                int64_t conv_state_ld, int64_t ssm_state_stride_b,
                void* out, int64_t out_stride_b, int64_t out_stride_t,
                float* conv_state_out, float* ssm_state_out,
                void* cuda_stream) {
    // one segment covering the whole row (seg_len rounded up to whole chunks)
    const int one = seqlen > 0 && seqlen <= (1 << 30)
                        ? (seqlen + ssm::kPrefillChunk - 1) / ssm::kPrefillChunk * ssm::kPrefillChunk
                        : ssm::kPrefillChunk;
    return prefill_impl("ssm_prefill", batch, seqlen, d_inner, d_state, d_conv, in_dtype, out_dtype, x, z, dt,
                        in_stride_b, in_stride_t, Bmat, Cmat, A, Dskip, dt_bias, conv_w, conv_b, conv_state_in,
                        ssm_state_in, conv_state_ld, ssm_state_stride_b, out, out_stride_b, out_stride_t,
                        conv_state_out, ssm_state_out, one, nullptr, 0, cuda_stream);
}

int ssm_prefill_segmented_noalloc(int batch, int seqlen, int d_inner, int d_state, int d_conv,
                                  ssm_dtype_t in_dtype, ssm_dtype_t out_dtype,
                                  const void* x, const void* z, const void* dt,
                                  int64_t in_stride_b, int64_t in_stride_t,
                                  const void* Bmat, const void* Cmat,
                                  const float* A, const float* Dskip, const float* dt_bias,
                                  const float* conv_w, const float* conv_b,
                                  const float* conv_state_in, const float* ssm_state_in,
                                  int64_t conv_state_ld, int64_t ssm_state_stride_b,
                                  void* out, int64_t out_stride_b, int64_t out_stride_t,
                                  float* conv_state_out, float* ssm_state_out,
                                  int seg_len, void* cuda_stream) {
    // Nothing in the array has to start at zero: pass A writes every entry that passes B and C read.
    return prefill_impl("ssm_prefill_segmented_noalloc", batch, seqlen, d_inner, d_state, d_conv, in_dtype,
                        out_dtype, x, z, dt, in_stride_b, in_stride_t, Bmat, Cmat, A, Dskip, dt_bias, conv_w,
                        conv_b, conv_state_in, ssm_state_in, conv_state_ld, ssm_state_stride_b, out, out_stride_b,
                        out_stride_t, conv_state_out, ssm_state_out, seg_len, nullptr, 0, cuda_stream,
                        /*fixed_scratch=*/true);
}

int ssm_out_proj_partial(int64_t M, int64_t N, int64_t K, const void* y, int64_t ldy, const void* W, int64_t ldw,
                         ssm_dtype_t out_dtype, void* out, int64_t ldo, float* block_amax, void* cuda_stream) {
    static const char* fn = "ssm_out_proj_partial";
    g_err[0] = 0;
    if (M < 1 || M > 65535LL * 128) return fail(SSM_ERR_INVALID_ARG, "%s: M %lld not in [1, 65535*128]", fn, (long long)M);
    if (N < 1 || N > 65535LL * 256) return fail(SSM_ERR_INVALID_ARG, "%s: N %lld not in [1, 65535*256]", fn, (long long)N);
    if (K < 1 || K > (1LL << 31)) return fail(SSM_ERR_INVALID_ARG, "%s: K %lld out of range", fn, (long long)K);
    if (!dtype_ok(out_dtype)) return fail(SSM_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (!y || !W || !out) return fail(SSM_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (N % 128 != 0) return fail(SSM_ERR_UNSUPPORTED, "%s: N %lld is not a multiple of 128", fn, (long long)N);
    if (K % 8 != 0) return fail(SSM_ERR_UNSUPPORTED, "%s: K %lld is not a multiple of 8", fn, (long long)K);
    if (ldy < K || ldw < K || ldo < N) return fail(SSM_ERR_INVALID_ARG, "%s: a row stride is below the row length", fn);
    if (ldy % 8 != 0 || ldw % 8 != 0 || ldo % 8 != 0)
        return fail(SSM_ERR_MISALIGNED, "%s: row strides must be multiples of 8 elements", fn);
    if (!aligned(y, 16) || !aligned(W, 16) || !aligned(out, 16) || (block_amax && !aligned(block_amax, 4)))
        return fail(SSM_ERR_MISALIGNED, "%s: y, W and out must be 16-byte aligned", fn);
    // the kernel counts 128-row tiles and 64-wide K steps in 32 bits
    const int64_t tiles = ((M + 127) / 128) * ((N + 127) / 128);
    if (tiles * ((K + 63) / 64) >= (1LL << 31))
        return fail(SSM_ERR_UNSUPPORTED, "%s: %lld tiles x %lld K steps exceed 2^31", fn, (long long)tiles,
                    (long long)((K + 63) / 64));

    int serr = 0;
    unsigned int* status = status_ptr(&serr);
    if (serr) return fail(SSM_ERR_CUDA, "%s: no usable CUDA device", fn);
    ssm::OutProjArgs a{};
    a.M = M;
    a.N = N;
    a.K = K;
    a.out = out;
    a.ldo = ldo;
    a.amax = block_amax;
    a.status = status;
    const char* why = "";
    if (ssm::launch_out_proj(a, y, W, ldy, ldw, out_dtype == SSM_BF16, static_cast<cudaStream_t>(cuda_stream), &why) != 0)
        return fail(SSM_ERR_CUDA, "%s: %s", fn, why);
    return SSM_OK;
}

size_t ssd_prefill_workspace_bytes(int batch, int seqlen, int n_heads, int n_groups) {
    if (batch < 1 || batch > 65535 || seqlen < 1 || seqlen > (1 << 30) || n_heads < 1 || n_heads > 65535 ||
        n_groups < 1 || n_heads % n_groups != 0)
        return 0;
    return ssm::ssd_workspace_layout(batch, seqlen, n_heads, n_groups).bytes;
}

int ssd_prefill(int batch, int seqlen, int n_heads, int head_dim, int n_groups, int d_state, int d_conv,
                ssm_dtype_t in_dtype, ssm_dtype_t out_dtype,
                const void* xBC, int64_t xbc_stride_b, int64_t xbc_stride_t,
                const void* z, int64_t z_stride_b, int64_t z_stride_t,
                const void* dt, int64_t dt_stride_b, int64_t dt_stride_t,
                const float* conv_w, const float* conv_b,
                const float* A, const float* Dskip, const float* dt_bias,
                const float* conv_state_in, const float* ssm_state_in,
                void* out, int64_t out_stride_b, int64_t out_stride_t,
                float* conv_state_out, float* ssm_state_out,
                void* workspace, size_t workspace_bytes, void* cuda_stream) {
    static const char* fn = "ssd_prefill";
    g_err[0] = 0;
    if (batch < 1 || batch > 65535) return fail(SSM_ERR_INVALID_ARG, "%s: batch %d not in [1, 65535]", fn, batch);
    if (seqlen < 1 || seqlen > (1 << 30)) return fail(SSM_ERR_INVALID_ARG, "%s: seqlen %d not in [1, 2^30]", fn, seqlen);
    if (n_heads < 1 || n_heads > 65535) return fail(SSM_ERR_INVALID_ARG, "%s: n_heads %d not in [1, 65535]", fn, n_heads);
    if (n_groups < 1 || n_heads % n_groups != 0)
        return fail(SSM_ERR_INVALID_ARG, "%s: n_groups %d does not divide n_heads %d", fn, n_groups, n_heads);
    if (!dtype_ok(in_dtype) || !dtype_ok(out_dtype)) return fail(SSM_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (head_dim != 64 || d_state != 64 || d_conv != 4)
        return fail(SSM_ERR_UNSUPPORTED, "%s: head_dim %d, d_state %d, d_conv %d unsupported (64, 64, 4 only)", fn,
                    head_dim, d_state, d_conv);
    if (in_dtype != SSM_BF16) return fail(SSM_ERR_UNSUPPORTED, "%s: token inputs must be bf16", fn);
    if (!xBC || !z || !dt || !conv_w || !conv_b || !A || !Dskip || !dt_bias || !out || !conv_state_out ||
        !ssm_state_out || !workspace)
        return fail(SSM_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    const int64_t HP = 64LL * n_heads, Cx = HP + 128LL * n_groups;
    if (xbc_stride_t < Cx || z_stride_t < HP || dt_stride_t < n_heads || out_stride_t < HP)
        return fail(SSM_ERR_INVALID_ARG, "%s: a token stride is below the row width", fn);
    if (batch > 1 && (xbc_stride_b < (int64_t)(seqlen - 1) * xbc_stride_t + Cx ||
                      z_stride_b < (int64_t)(seqlen - 1) * z_stride_t + HP ||
                      dt_stride_b < (int64_t)(seqlen - 1) * dt_stride_t + n_heads))
        return fail(SSM_ERR_INVALID_ARG, "%s: a batch stride lets rows overlap", fn);
    if (batch > 1 && out_stride_b < (int64_t)(seqlen - 1) * out_stride_t + HP)
        return fail(SSM_ERR_INVALID_ARG, "%s: out_stride_b %lld lets batch rows overlap", fn, (long long)out_stride_b);
    const size_t need = ssm::ssd_workspace_layout(batch, seqlen, n_heads, n_groups).bytes;
    if (workspace_bytes < need)
        return fail(SSM_ERR_INVALID_ARG, "%s: workspace of %zu bytes given, %zu needed", fn, workspace_bytes, need);
    const int oe = esize(out_dtype);
    if (!aligned(xBC, 16) || !aligned(z, 16) || xbc_stride_t % 8 || xbc_stride_b % 8 || z_stride_t % 8 || z_stride_b % 8)
        return fail(SSM_ERR_MISALIGNED, "%s: xBC and z must be 16-byte aligned with strides of 16 bytes", fn);
    if (!aligned(out, 16) || (out_stride_t * oe) % 16 || (out_stride_b * oe) % 16)
        return fail(SSM_ERR_MISALIGNED, "%s: out must be 16-byte aligned with strides of 16 bytes", fn);
    if (!aligned(conv_w, 16) || !aligned(ssm_state_out, 16) || (ssm_state_in && !aligned(ssm_state_in, 16)) ||
        !aligned(workspace, 16) || !aligned(dt, 2))
        return fail(SSM_ERR_MISALIGNED, "%s: conv_w, the ssm states and the workspace need 16-byte alignment", fn);

    int serr = 0;
    unsigned int* status = status_ptr(&serr);
    if (serr) return fail(SSM_ERR_CUDA, "%s: no usable CUDA device", fn);
    ssm::SsdArgs a{};
    a.batch = batch;
    a.seqlen = seqlen;
    a.n_heads = n_heads;
    a.n_groups = n_groups;
    a.xBC = xBC;
    a.xbc_stride_b = xbc_stride_b;
    a.xbc_stride_t = xbc_stride_t;
    a.z = z;
    a.z_stride_b = z_stride_b;
    a.z_stride_t = z_stride_t;
    a.dt = dt;
    a.dt_stride_b = dt_stride_b;
    a.dt_stride_t = dt_stride_t;
    a.conv_w = conv_w;
    a.conv_b = conv_b;
    a.A = A;
    a.Dskip = Dskip;
    a.dt_bias = dt_bias;
    a.conv_state_in = conv_state_in;
    a.ssm_state_in = ssm_state_in;
    a.out = out;
    a.out_stride_b = out_stride_b;
    a.out_stride_t = out_stride_t;
    a.conv_state_out = conv_state_out;
    a.ssm_state_out = ssm_state_out;
    a.workspace = workspace;
    a.status = status;
    const char* why = "";
    if (ssm::launch_ssd_prefill(a, out_dtype == SSM_BF16, static_cast<cudaStream_t>(cuda_stream), &why) != 0)
        return fail(SSM_ERR_CUDA, "%s: %s", fn, why);
    return SSM_OK;
}

int ssd_decode_step(int batch, int n_heads, int head_dim, int n_groups, int d_state, int d_conv,
                    ssm_dtype_t in_dtype, ssm_dtype_t out_dtype,
                    const void* xBC, const void* z, const void* dt,
                    const float* conv_w, const float* conv_b,
                    const float* A, const float* Dskip, const float* dt_bias,
                    float* conv_state, float* ssm_state, int n_slots, const int32_t* state_slot,
                    void* out, void* cuda_stream) {
    static const char* fn = "ssd_decode_step";
    g_err[0] = 0;
    if (batch < 1 || batch > 65535) return fail(SSM_ERR_INVALID_ARG, "%s: batch %d not in [1, 65535]", fn, batch);
    if (n_heads < 1 || n_heads > 65535) return fail(SSM_ERR_INVALID_ARG, "%s: n_heads %d not in [1, 65535]", fn, n_heads);
    if (n_groups < 1 || n_heads % n_groups != 0)
        return fail(SSM_ERR_INVALID_ARG, "%s: n_groups %d does not divide n_heads %d", fn, n_groups, n_heads);
    if (!dtype_ok(in_dtype) || !dtype_ok(out_dtype)) return fail(SSM_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (head_dim != 64 || d_state != 64 || d_conv != 4)
        return fail(SSM_ERR_UNSUPPORTED, "%s: head_dim %d, d_state %d, d_conv %d unsupported (64, 64, 4 only)", fn,
                    head_dim, d_state, d_conv);
    if (!xBC || !z || !dt || !conv_w || !conv_b || !A || !Dskip || !dt_bias || !conv_state || !ssm_state || !out)
        return fail(SSM_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (n_slots < 1 || (!state_slot && n_slots < batch))
        return fail(SSM_ERR_INVALID_ARG, "%s: n_slots %d too small", fn, n_slots);
    const int es = esize(in_dtype);
    if (!aligned(conv_w, 16) || !aligned(ssm_state, 16))
        return fail(SSM_ERR_MISALIGNED, "%s: conv_w and ssm_state need 16-byte alignment", fn);
    if (!aligned(xBC, es) || !aligned(z, es) || !aligned(dt, es) || !aligned(out, esize(out_dtype)) ||
        !aligned(conv_state, 4) || (state_slot && !aligned(state_slot, 4)))
        return fail(SSM_ERR_MISALIGNED, "%s: a pointer is not element aligned", fn);
    int serr = 0;
    unsigned int* status = status_ptr(&serr);
    if (serr) return fail(SSM_ERR_CUDA, "%s: no usable CUDA device", fn);
    ssm::SsdDecodeArgs a{};
    a.batch = batch;
    a.n_heads = n_heads;
    a.n_groups = n_groups;
    a.n_slots = n_slots;
    a.xBC = xBC;
    a.z = z;
    a.dt = dt;
    a.conv_w = conv_w;
    a.conv_b = conv_b;
    a.A = A;
    a.Dskip = Dskip;
    a.dt_bias = dt_bias;
    a.conv_state = conv_state;
    a.ssm_state = ssm_state;
    a.state_slot = state_slot;
    a.out = out;
    a.status = status;
    const char* why = "";
    if (ssm::launch_ssd_decode(a, in_dtype == SSM_BF16, out_dtype == SSM_BF16, static_cast<cudaStream_t>(cuda_stream),
                               &why) != 0)
        return fail(SSM_ERR_CUDA, "%s: %s", fn, why);
    return SSM_OK;
}

static int expire_wait(const char* fn, int which, int limit_us, void* cuda_stream) {
    g_err[0] = 0;
    if (which < 0 || which > 2) return fail(SSM_ERR_INVALID_ARG, "%s: which %d not in [0, 2]", fn, which);
    if (limit_us < 1 || limit_us > 2000000) return fail(SSM_ERR_INVALID_ARG, "%s: limit_us %d not in [1, 2e6]", fn, limit_us);
    int serr = 0;
    unsigned int* status = status_ptr(&serr);
    if (serr) return fail(SSM_ERR_CUDA, "%s: no usable CUDA device", fn);
    const char* why = "";
    if (ssm::launch_expire_wait(which, status, (uint64_t)limit_us * 1000u, static_cast<cudaStream_t>(cuda_stream), &why) != 0)
        return fail(SSM_ERR_CUDA, "%s: %s", fn, why);
    return SSM_OK;
}

int ssm_selftest_expire_wait(int limit_us, void* cuda_stream) { return expire_wait("ssm_selftest_expire_wait", 0, limit_us, cuda_stream); }

int ssm_selftest_expire_wait_of(int which, int limit_us, void* cuda_stream) {
    return expire_wait("ssm_selftest_expire_wait_of", which, limit_us, cuda_stream);
}

size_t ssm_prefill_workspace_bytes(int batch, int seqlen, int d_inner, int seg_len) {
    if (batch < 1 || seqlen < 1 || d_inner < 1 || seg_len < 1) return 0;
    const int64_t n_seg = ((int64_t)seqlen + seg_len - 1) / seg_len;
    return (size_t)(n_seg - 1) * (size_t)batch * (size_t)d_inner * 32 * sizeof(float);
}

int ssm_prefill_segmented(int batch, int seqlen, int d_inner, int d_state, int d_conv,
                          ssm_dtype_t in_dtype, ssm_dtype_t out_dtype,
                          const void* x, const void* z, const void* dt,
                          int64_t in_stride_b, int64_t in_stride_t,
                          const void* Bmat, const void* Cmat,
                          const float* A, const float* Dskip, const float* dt_bias,
                          const float* conv_w, const float* conv_b,
                          const float* conv_state_in, const float* ssm_state_in,
                          int64_t conv_state_ld, int64_t ssm_state_stride_b,
                          void* out, int64_t out_stride_b, int64_t out_stride_t,
                          float* conv_state_out, float* ssm_state_out,
                          int seg_len, void* workspace, size_t workspace_bytes,
                          void* cuda_stream) {
    return prefill_impl("ssm_prefill_segmented", batch, seqlen, d_inner, d_state, d_conv, in_dtype, out_dtype,
                        x, z, dt, in_stride_b, in_stride_t, Bmat, Cmat, A, Dskip, dt_bias, conv_w, conv_b,
                        conv_state_in, ssm_state_in, conv_state_ld, ssm_state_stride_b, out, out_stride_b,
                        out_stride_t, conv_state_out, ssm_state_out, seg_len, workspace, workspace_bytes,
                        cuda_stream);
}

}  // extern "C"

namespace {

// Shared by ssm_decode_step (one token) and ssm_decode_tokens (T tokens).
int decode_impl(const char* fn, int batch, int n_tokens, int d_inner, int d_state, int d_conv,
                ssm_dtype_t in_dtype, ssm_dtype_t out_dtype,
                const void* x, const void* z, const void* dt, int64_t in_stride_b, int64_t in_stride_t,
                const void* Bmat, const void* Cmat,
                const float* A, const float* Dskip, const float* dt_bias,
                const float* conv_w, const float* conv_b,
                float* conv_state, float* ssm_state,
                int64_t conv_state_ld, int64_t ssm_state_stride_b,
                int n_slots, const int32_t* state_slot,
                void* out, int64_t out_stride_b, int64_t out_stride_t,
                void* cuda_stream) {
    g_err[0] = 0;
    if (batch < 1 || batch > 65535) return fail(SSM_ERR_INVALID_ARG, "%s: batch %lld not in [1, 65535]", fn, (long long)batch);
    if (n_tokens < 1 || n_tokens > 4096) return fail(SSM_ERR_INVALID_ARG, "%s: n_tokens %lld not in [1, 4096]", fn, (long long)n_tokens);
    if (d_inner < 1) return fail(SSM_ERR_INVALID_ARG, "%s: d_inner %lld < 1", fn, (long long)d_inner);
    if (!dtype_ok(in_dtype) || !dtype_ok(out_dtype)) return fail(SSM_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (d_state != 16) return fail(SSM_ERR_UNSUPPORTED, "%s: d_state %lld unsupported (16 only)", fn, (long long)d_state);
    if (d_conv != 4) return fail(SSM_ERR_UNSUPPORTED, "%s: d_conv %lld unsupported (4 only)", fn, (long long)d_conv);
    if (d_inner % 8 != 0) return fail(SSM_ERR_UNSUPPORTED, "%s: d_inner %lld is not a multiple of 8", fn, (long long)d_inner);
    if (!x || !z || !dt || !Bmat || !Cmat || !A || !Dskip || !dt_bias || !conv_w || !conv_b || !conv_state ||
        !ssm_state || !out)
        return fail(SSM_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (n_tokens > 1 && in_stride_t < d_inner) return fail(SSM_ERR_INVALID_ARG, "%s: in_stride_t %lld < d_inner", fn, (long long)in_stride_t);
    if (n_tokens > 1 && out_stride_t < d_inner) return fail(SSM_ERR_INVALID_ARG, "%s: out_stride_t %lld < d_inner", fn, (long long)out_stride_t);
    const int64_t in_row = n_tokens > 1 ? (int64_t)(n_tokens - 1) * in_stride_t + d_inner : d_inner;
    const int64_t out_row = n_tokens > 1 ? (int64_t)(n_tokens - 1) * out_stride_t + d_inner : d_inner;
    if (batch > 1 && in_stride_b < in_row) return fail(SSM_ERR_INVALID_ARG, "%s: in_stride_b %lld too small", fn, (long long)in_stride_b);
    if (batch > 1 && out_stride_b < out_row) return fail(SSM_ERR_INVALID_ARG, "%s: out_stride_b %lld lets requests overlap", fn, (long long)out_stride_b);
    if (conv_state_ld < d_inner) return fail(SSM_ERR_INVALID_ARG, "%s: conv_state_ld %lld < d_inner", fn, (long long)conv_state_ld);
    if (ssm_state_stride_b < 16LL * d_inner)
        return fail(SSM_ERR_INVALID_ARG, "%s: ssm_state_stride_b %lld < 16*d_inner", fn, (long long)ssm_state_stride_b);
    if (n_slots < 1 || (!state_slot && n_slots < batch))
        return fail(SSM_ERR_INVALID_ARG, "%s: n_slots %lld too small", fn, (long long)n_slots);
    const int es = esize(in_dtype);
    if (!aligned(Bmat, 4 * es) || !aligned(Cmat, 4 * es))
        return fail(SSM_ERR_MISALIGNED, "%s: B and C must be aligned to 4 elements", fn);
    if (!aligned(A, 16) || !aligned(conv_w, 16) || !aligned(ssm_state, 16) || ssm_state_stride_b % 4 != 0)
        return fail(SSM_ERR_MISALIGNED, "%s: A, conv_w and ssm_state need 16-byte alignment", fn);
    if (!aligned(x, es) || !aligned(z, es) || !aligned(dt, es) || !aligned(out, esize(out_dtype)) ||
        !aligned(conv_state, 4) || (state_slot && !aligned(state_slot, 4)))
        return fail(SSM_ERR_MISALIGNED, "%s: a pointer is not element aligned", fn);

    int serr = 0;
    unsigned int* status = status_ptr(&serr);
    if (serr) return fail(SSM_ERR_CUDA, "%s: no usable CUDA device", fn);

    ssm::DecodeArgs a{};
    a.batch = batch;
    a.n_tokens = n_tokens;
    a.d_inner = d_inner;
    a.n_slots = n_slots;
    a.x = x;
    a.z = z;
    a.dt = dt;
    a.in_stride_b = in_stride_b;
    a.in_stride_t = in_stride_t;
    a.Bm = Bmat;
    a.Cm = Cmat;
    a.A = A;
    a.Dskip = Dskip;
    a.dt_bias = dt_bias;
    a.conv_w = conv_w;
    a.conv_b = conv_b;
    a.conv_state = conv_state;
    a.ssm_state = ssm_state;
    a.conv_state_ld = conv_state_ld;
    a.ssm_state_stride_b = ssm_state_stride_b;
    a.state_slot = state_slot;
    a.out = out;
    a.out_stride_b = out_stride_b;
    a.out_stride_t = out_stride_t;
    a.status = status;
    const char* why = "";
    if (ssm::launch_decode(a, in_dtype == SSM_BF16, out_dtype == SSM_BF16, static_cast<cudaStream_t>(cuda_stream),
                           &why) != 0)
        return fail(SSM_ERR_CUDA, "%s: %s", fn, why);
    return SSM_OK;
}

}  // namespace

extern "C" {

int ssm_decode_step(int batch, int d_inner, int d_state, int d_conv,
                    ssm_dtype_t in_dtype, ssm_dtype_t out_dtype,
                    const void* x, const void* z, const void* dt, int64_t in_stride_b,
                    const void* Bmat, const void* Cmat,
                    const float* A, const float* Dskip, const float* dt_bias,
                    const float* conv_w, const float* conv_b,
                    float* conv_state, float* ssm_state,
                    int64_t conv_state_ld, int64_t ssm_state_stride_b,
                    int n_slots, const int32_t* state_slot,
                    void* out, int64_t out_stride_b,
                    void* cuda_stream) {
    return decode_impl("ssm_decode_step", batch, 1, d_inner, d_state, d_conv, in_dtype, out_dtype, x, z, dt,
                       in_stride_b, d_inner, Bmat, Cmat, A, Dskip, dt_bias, conv_w, conv_b, conv_state, ssm_state,
                       conv_state_ld, ssm_state_stride_b, n_slots, state_slot, out, out_stride_b, d_inner,
                       cuda_stream);
}

int ssm_decode_tokens(int batch, int n_tokens, int d_inner, int d_state, int d_conv,
                      ssm_dtype_t in_dtype, ssm_dtype_t out_dtype,
                      const void* x, const void* z, const void* dt,
                      int64_t in_stride_b, int64_t in_stride_t,
                      const void* Bmat, const void* Cmat,
                      const float* A, const float* Dskip, const float* dt_bias,
                      const float* conv_w, const float* conv_b,
                      float* conv_state, float* ssm_state,
                      int64_t conv_state_ld, int64_t ssm_state_stride_b,
                      int n_slots, const int32_t* state_slot,
                      void* out, int64_t out_stride_b, int64_t out_stride_t,
                      void* cuda_stream) {
    return decode_impl("ssm_decode_tokens", batch, n_tokens, d_inner, d_state, d_conv, in_dtype, out_dtype, x, z,
                       dt, in_stride_b, in_stride_t, Bmat, Cmat, A, Dskip, dt_bias, conv_w, conv_b, conv_state,
                       ssm_state, conv_state_ld, ssm_state_stride_b, n_slots, state_slot, out, out_stride_b,
                       out_stride_t, cuda_stream);
}

int q8_reduce_partials(int P, const void* const* partials, ssm_dtype_t in_dtype, int64_t n, int block,
                       void* out, ssm_dtype_t out_dtype, int32_t* sums_out, float* scales_out,
                       void* cuda_stream) {
    g_err[0] = 0;
    if (P < 1 || P > ssm::kMaxPartials) return fail(SSM_ERR_UNSUPPORTED, "q8_reduce_partials: P %lld not in [1, 8]", (long long)(P));
    if (!partials) return fail(SSM_ERR_INVALID_ARG, "q8_reduce_partials: partials is NULL");
    if (n < 1) return fail(SSM_ERR_INVALID_ARG, "q8_reduce_partials: n %lld < 1", (long long)(n));
    if (block != 128) return fail(SSM_ERR_UNSUPPORTED, "q8_reduce_partials: block %lld unsupported (128 only)", (long long)(block));
    if (!dtype_ok(in_dtype) || !dtype_ok(out_dtype)) return fail(SSM_ERR_INVALID_ARG, "q8_reduce_partials: unknown dtype");
    if (!out) return fail(SSM_ERR_INVALID_ARG, "q8_reduce_partials: out is NULL");
    ssm::Q8Args a{};
    for (int p = 0; p < P; ++p) {
        if (!partials[p]) return fail(SSM_ERR_INVALID_ARG, "q8_reduce_partials: partials[%lld] is NULL", (long long)(p));
        if (!aligned(partials[p], 16)) return fail(SSM_ERR_MISALIGNED, "q8_reduce_partials: partials[%lld] not 16-byte aligned", (long long)(p));
        a.partials[p] = partials[p];
    }
    if (!aligned(out, 16) || (sums_out && !aligned(sums_out, 16)) || (scales_out && !aligned(scales_out, 4)))
        return fail(SSM_ERR_MISALIGNED, "q8_reduce_partials: out and sums must be 16-byte aligned");
    a.P = P;
    a.n = n;
    a.out = out;
    a.sums = sums_out;
    a.scales = scales_out;
    const char* why = "";
    if (ssm::launch_q8(a, in_dtype == SSM_BF16, out_dtype == SSM_BF16, static_cast<cudaStream_t>(cuda_stream), &why) != 0)
        return fail(SSM_ERR_CUDA, "q8_reduce_partials: %s", why);
    return SSM_OK;
}

int q8_block_absmax(const void* x, ssm_dtype_t in_dtype, int64_t n, int block, float* block_amax,
                    void* cuda_stream) {
    static const char* fn = "q8_block_absmax";
    g_err[0] = 0;
    if (!x || !block_amax) return fail(SSM_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (n < 1) return fail(SSM_ERR_INVALID_ARG, "%s: n %lld < 1", fn, (long long)n);
    if (block != 128) return fail(SSM_ERR_UNSUPPORTED, "%s: block %d unsupported (128 only)", fn, block);
    if (!dtype_ok(in_dtype)) return fail(SSM_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (!aligned(x, 16) || !aligned(block_amax, 4)) return fail(SSM_ERR_MISALIGNED, "%s: x must be 16-byte aligned", fn);
    const char* why = "";
    if (ssm::launch_q8_absmax(x, in_dtype == SSM_BF16, n, block_amax, static_cast<cudaStream_t>(cuda_stream), &why) != 0)
        return fail(SSM_ERR_CUDA, "%s: %s", fn, why);
    return SSM_OK;
}

int q8_quantize_shared(const void* x, ssm_dtype_t in_dtype, int64_t n, int block, const float* block_amax,
                       int8_t* codes, float* scales_out, void* cuda_stream) {
    static const char* fn = "q8_quantize_shared";
    g_err[0] = 0;
    if (!x || !block_amax || !codes) return fail(SSM_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (n < 1) return fail(SSM_ERR_INVALID_ARG, "%s: n %lld < 1", fn, (long long)n);
    if (block != 128) return fail(SSM_ERR_UNSUPPORTED, "%s: block %d unsupported (128 only)", fn, block);
    if (!dtype_ok(in_dtype)) return fail(SSM_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(block_amax, 4) || (scales_out && !aligned(scales_out, 4)))
        return fail(SSM_ERR_MISALIGNED, "%s: x and codes must be 16-byte aligned", fn);
    const char* why = "";
    if (ssm::launch_q8_quantize(x, in_dtype == SSM_BF16, n, block_amax, codes, scales_out,
                                static_cast<cudaStream_t>(cuda_stream), &why) != 0)
        return fail(SSM_ERR_CUDA, "%s: %s", fn, why);
    return SSM_OK;
}

int q8_sum_dequant(int P, const int8_t* const* codes, const float* scales, int64_t n, int block,
                   void* out, ssm_dtype_t out_dtype, int32_t* sums_out, void* cuda_stream) {
    static const char* fn = "q8_sum_dequant";
    g_err[0] = 0;
    if (P < 1 || P > ssm::kMaxPartials) return fail(SSM_ERR_UNSUPPORTED, "%s: P %d not in [1, 8]", fn, P);
    if (!codes || !scales || !out) return fail(SSM_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (n < 1) return fail(SSM_ERR_INVALID_ARG, "%s: n %lld < 1", fn, (long long)n);
    if (block != 128) return fail(SSM_ERR_UNSUPPORTED, "%s: block %d unsupported (128 only)", fn, block);
    if (!dtype_ok(out_dtype)) return fail(SSM_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    for (int p = 0; p < P; ++p) {
        if (!codes[p]) return fail(SSM_ERR_INVALID_ARG, "%s: codes[%d] is NULL", fn, p);
        if (!aligned(codes[p], 16)) return fail(SSM_ERR_MISALIGNED, "%s: codes[%d] not 16-byte aligned", fn, p);
    }
    if (!aligned(out, 16) || !aligned(scales, 4) || (sums_out && !aligned(sums_out, 16)))
        return fail(SSM_ERR_MISALIGNED, "%s: out and sums must be 16-byte aligned", fn);
    const char* why = "";
    if (ssm::launch_q8_sum(P, codes, scales, n, out, out_dtype == SSM_BF16, sums_out,
                           static_cast<cudaStream_t>(cuda_stream), &why) != 0)
        return fail(SSM_ERR_CUDA, "%s: %s", fn, why);
    return SSM_OK;
}

int ssm_device_status(uint32_t* status, int clear) {
    g_err[0] = 0;
    if (!status) return fail(SSM_ERR_INVALID_ARG, "ssm_device_status: status is NULL");
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_status_word, sizeof v) != cudaSuccess)
        return fail(SSM_ERR_CUDA, "ssm_device_status: cudaMemcpyFromSymbol failed");
    if (clear) {
        const unsigned int zero = 0;
        if (cudaMemcpyToSymbol(g_status_word, &zero, sizeof zero) != cudaSuccess)
            return fail(SSM_ERR_CUDA, "ssm_device_status: cudaMemcpyToSymbol failed");
    }
    *status = v;
    return SSM_OK;
}

}  // extern "C"

// ------------------------------------------------------------------ attention
namespace {

// The parts of an attention call that several entry points share; each returns SSM_OK or fails.
int check_heads(const char* fn, int n_q, int n_kv, int dim) {
    if (n_kv < 1 || n_kv > 4096 || n_q < 1 || n_q > 65535 || n_q % n_kv != 0)
        return fail(SSM_ERR_INVALID_ARG, "%s: %d query heads over %d kv heads", fn, n_q, n_kv);
    if (dim < 16 || dim > 128 || dim % 16 != 0)
        return fail(SSM_ERR_UNSUPPORTED, "%s: head_dim %d unsupported (multiples of 16 up to 128)", fn, dim);
    return SSM_OK;
}

int check_view(const char* fn, const char* name, const void* p, int64_t st, int64_t sh, int dim) {
    if (!p) return fail(SSM_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
    if (st < dim || sh < dim) return fail(SSM_ERR_INVALID_ARG, "%s: a stride of %s is below head_dim", fn, name);
    if (!aligned(p, 16) || st % 8 != 0 || sh % 8 != 0)
        return fail(SSM_ERR_MISALIGNED, "%s: %s must be 16-byte aligned with strides that are multiples of 8", fn, name);
    return SSM_OK;
}

// An output's heads may not overlap inside a token, nor its tokens.
int check_out_view(const char* fn, const char* name, const void* p, int64_t n, int64_t st, int64_t sh, int heads, int dim) {
    const int rc = check_view(fn, name, p, st, sh, dim);
    if (rc != SSM_OK) return rc;
    const bool rows_apart = n <= 1 || st >= (int64_t)(heads - 1) * sh + dim;        // [token][head]
    const bool heads_apart = heads <= 1 || sh >= (n - 1) * st + dim;                // [head][token]
    if (!rows_apart && !heads_apart)
        return fail(SSM_ERR_INVALID_ARG, "%s: the strides of %s let rows overlap", fn, name);
    return SSM_OK;
}

int check_cache(const char* fn, int cache_dtype, const void* k, const void* v, const float* ks, const float* vs,
                int n_pages, int page_size) {
    if (cache_dtype != SSM_BF16 && cache_dtype != SSM_I8)
        return fail(cache_dtype == SSM_F32 ? SSM_ERR_UNSUPPORTED : SSM_ERR_INVALID_ARG,
                    "%s: the cache holds SSM_BF16 or SSM_I8 rows", fn);
    if (n_pages < 1 || page_size < 1) return fail(SSM_ERR_INVALID_ARG, "%s: n_pages %d, page_size %d", fn, n_pages, page_size);
    if (page_size % 16 != 0 || page_size > 4096)
        return fail(SSM_ERR_UNSUPPORTED, "%s: page_size %d unsupported (multiples of 16 up to 4096)", fn, page_size);
    if ((int64_t)n_pages * page_size >= (1LL << 31))
        return fail(SSM_ERR_UNSUPPORTED, "%s: %d pages of %d tokens pass 2^31 slots", fn, n_pages, page_size);
    if (!k || !v) return fail(SSM_ERR_INVALID_ARG, "%s: a cache pointer is NULL", fn);
    if (cache_dtype == SSM_I8 && (!ks || !vs)) return fail(SSM_ERR_INVALID_ARG, "%s: an int8 cache needs k_scale and v_scale", fn);
    if (cache_dtype == SSM_BF16 && (ks || vs)) return fail(SSM_ERR_INVALID_ARG, "%s: a bf16 cache has no scales", fn);
    if (!aligned(k, 16) || !aligned(v, 16) || (ks && !aligned(ks, 16)) || (vs && !aligned(vs, 16)))
        return fail(SSM_ERR_MISALIGNED, "%s: the caches and their scales must be 16-byte aligned", fn);
    return SSM_OK;
}

int check_table(const char* fn, const int32_t* table, int64_t stride, int n_table) {
    if (!table) return fail(SSM_ERR_INVALID_ARG, "%s: page_table is NULL", fn);
    if (n_table < 1 || stride < n_table)
        return fail(SSM_ERR_INVALID_ARG, "%s: page_table rows of %d entries with stride %lld", fn, n_table, (long long)stride);
    if (!aligned(table, 4)) return fail(SSM_ERR_MISALIGNED, "%s: page_table is not element aligned", fn);
    return SSM_OK;
}

ssm::AttnCache make_cache(const void* k, const void* v, const float* ks, const float* vs, int n_pages, int page_size,
                          int n_kv, int dim) {
    return ssm::AttnCache{k, v, ks, vs, n_pages, page_size, n_kv, dim};
}

}  // namespace

extern "C" {

int attn_rope_table(int64_t n_pos, int half, const double* inv_freq, double scale, float* cos_out, float* sin_out,
                    void* cuda_stream) {
    static const char* fn = "attn_rope_table";
    g_err[0] = 0;
    if (n_pos < 1 || n_pos > (1LL << 26)) return fail(SSM_ERR_INVALID_ARG, "%s: n_pos %lld not in [1, 2^26]", fn, (long long)n_pos);
    if (half < 1 || half > 64) return fail(SSM_ERR_INVALID_ARG, "%s: half %d not in [1, 64]", fn, half);
    if (!inv_freq || !cos_out || !sin_out) return fail(SSM_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (!(scale - scale == 0)) return fail(SSM_ERR_INVALID_ARG, "%s: scale is not finite", fn);
    if (!aligned(cos_out, 4) || !aligned(sin_out, 4)) return fail(SSM_ERR_MISALIGNED, "%s: a table is not element aligned", fn);
    ssm::AttnRopeArgs a{};
    for (int i = 0; i < half; ++i) {
        if (!(inv_freq[i] - inv_freq[i] == 0)) return fail(SSM_ERR_INVALID_ARG, "%s: inv_freq[%d] is not finite", fn, i);
        a.inv_freq[i] = inv_freq[i];
    }
    a.n_pos = n_pos;
    a.half = half;
    a.scale = scale;
    a.cos = cos_out;
    a.sin = sin_out;
    const char* why = "";
    if (ssm::launch_attn_rope_table(a, static_cast<cudaStream_t>(cuda_stream), &why) != 0)
        return fail(SSM_ERR_CUDA, "%s: %s", fn, why);
    return SSM_OK;
}

int attn_append(int64_t n_tokens, int n_q_heads, int n_kv_heads, int head_dim, int rot_dim, int interleaved,
                const void* q, int64_t q_stride_t, int64_t q_stride_h,
                const void* k, int64_t k_stride_t, int64_t k_stride_h,
                const void* v, int64_t v_stride_t, int64_t v_stride_h,
                const int32_t* positions, const float* cos, const float* sin, int64_t n_pos,
                const int32_t* slots, ssm_dtype_t cache_dtype, void* k_cache, void* v_cache,
                float* k_scale, float* v_scale, int n_pages, int page_size,
                void* q_out, int64_t qo_stride_t, int64_t qo_stride_h,
                void* k_out, int64_t ko_stride_t, int64_t ko_stride_h, void* cuda_stream) {
    static const char* fn = "attn_append";
    g_err[0] = 0;
    int rc;
    if (n_tokens < 0 || n_tokens >= (1LL << 31)) return fail(SSM_ERR_INVALID_ARG, "%s: n_tokens %lld not in [0, 2^31)", fn, (long long)n_tokens);
    if ((rc = check_heads(fn, n_q_heads, n_kv_heads, head_dim)) != SSM_OK) return rc;
    if (rot_dim < 0 || rot_dim > head_dim) return fail(SSM_ERR_INVALID_ARG, "%s: rot_dim %d not in [0, head_dim]", fn, rot_dim);
    if (rot_dim % 8 != 0) return fail(SSM_ERR_UNSUPPORTED, "%s: rot_dim %d is not a multiple of 8", fn, rot_dim);
    if ((rc = check_cache(fn, cache_dtype, k_cache, v_cache, k_scale, v_scale, n_pages, page_size)) != SSM_OK) return rc;
    if (n_tokens == 0) return SSM_OK;
    if ((rc = check_view(fn, "k", k, k_stride_t, k_stride_h, head_dim)) != SSM_OK) return rc;
    if ((rc = check_view(fn, "v", v, v_stride_t, v_stride_h, head_dim)) != SSM_OK) return rc;
    if ((q == nullptr) != (q_out == nullptr)) return fail(SSM_ERR_INVALID_ARG, "%s: q and q_out go together", fn);
    if (q && (rc = check_view(fn, "q", q, q_stride_t, q_stride_h, head_dim)) != SSM_OK) return rc;
    if (q && (rc = check_out_view(fn, "q_out", q_out, n_tokens, qo_stride_t, qo_stride_h, n_q_heads, head_dim)) != SSM_OK) return rc;
    if (k_out && (rc = check_out_view(fn, "k_out", k_out, n_tokens, ko_stride_t, ko_stride_h, n_kv_heads, head_dim)) != SSM_OK) return rc;
    if (q && q_out == q && (qo_stride_t != q_stride_t || qo_stride_h != q_stride_h))
        return fail(SSM_ERR_INVALID_ARG, "%s: q_out is q with other strides", fn);
    if (k_out && k_out == k && (ko_stride_t != k_stride_t || ko_stride_h != k_stride_h))
        return fail(SSM_ERR_INVALID_ARG, "%s: k_out is k with other strides", fn);
    if (!slots) return fail(SSM_ERR_INVALID_ARG, "%s: slots is NULL", fn);
    if (rot_dim > 0 && (!positions || !cos || !sin || n_pos < 1))
        return fail(SSM_ERR_INVALID_ARG, "%s: a rotation needs positions, cos, sin and n_pos", fn);
    if (!aligned(slots, 4) || (positions && !aligned(positions, 4)) || (rot_dim > 0 && (!aligned(cos, 16) || !aligned(sin, 16))))
        return fail(SSM_ERR_MISALIGNED, "%s: cos and sin must be 16-byte aligned, positions and slots element aligned", fn);
    int serr = 0;
    unsigned int* status = status_ptr(&serr);
    if (serr) return fail(SSM_ERR_CUDA, "%s: no usable CUDA device", fn);
    ssm::AttnAppendArgs a{};
    a.n_tokens = n_tokens;
    a.n_q = q ? n_q_heads : 0;
    a.rot = rot_dim;
    a.interleaved = interleaved != 0;
    a.q = q;
    a.q_st = q_stride_t;
    a.q_sh = q_stride_h;
    a.k = k;
    a.k_st = k_stride_t;
    a.k_sh = k_stride_h;
    a.v = v;
    a.v_st = v_stride_t;
    a.v_sh = v_stride_h;
    a.positions = positions;
    a.cos = cos;
    a.sin = sin;
    a.n_pos = n_pos;
    a.slots = slots;
    a.c = make_cache(k_cache, v_cache, k_scale, v_scale, n_pages, page_size, n_kv_heads, head_dim);
    a.q_out = q_out;
    a.qo_st = qo_stride_t;
    a.qo_sh = qo_stride_h;
    a.k_out = k_out;
    a.ko_st = ko_stride_t;
    a.ko_sh = ko_stride_h;
    a.status = status;
    const char* why = "";
    if (ssm::launch_attn_append(a, cache_dtype == SSM_I8, static_cast<cudaStream_t>(cuda_stream), &why) != 0)
        return fail(SSM_ERR_CUDA, "%s: %s", fn, why);
    return SSM_OK;
}

int attn_cache_read(int batch, int64_t n_tokens, int n_kv_heads, int head_dim, ssm_dtype_t cache_dtype,
                    const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                    int n_pages, int page_size, const int32_t* page_table, int64_t table_stride, int n_table,
                    const int32_t* cu_len, const int32_t* first, ssm_dtype_t out_dtype,
                    void* k_out, void* v_out, void* cuda_stream) {
    static const char* fn = "attn_cache_read";
    g_err[0] = 0;
    int rc;
    if (batch < 1 || batch > 65535) return fail(SSM_ERR_INVALID_ARG, "%s: batch %d not in [1, 65535]", fn, batch);
    if (n_tokens < 0 || n_tokens >= (1LL << 31)) return fail(SSM_ERR_INVALID_ARG, "%s: n_tokens %lld not in [0, 2^31)", fn, (long long)n_tokens);
    if ((rc = check_heads(fn, n_kv_heads, n_kv_heads, head_dim)) != SSM_OK) return rc;
    if (!dtype_ok(out_dtype)) return fail(SSM_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if ((rc = check_cache(fn, cache_dtype, k_cache, v_cache, k_scale, v_scale, n_pages, page_size)) != SSM_OK) return rc;
    if ((rc = check_table(fn, page_table, table_stride, n_table)) != SSM_OK) return rc;
    if (!cu_len) return fail(SSM_ERR_INVALID_ARG, "%s: cu_len is NULL", fn);
    if (n_tokens == 0) return SSM_OK;
    if (!k_out || !v_out) return fail(SSM_ERR_INVALID_ARG, "%s: an output is NULL", fn);
    if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(cu_len, 4) || (first && !aligned(first, 4)))
        return fail(SSM_ERR_MISALIGNED, "%s: the outputs must be 16-byte aligned, cu_len and first element aligned", fn);
    int serr = 0;
    unsigned int* status = status_ptr(&serr);
    if (serr) return fail(SSM_ERR_CUDA, "%s: no usable CUDA device", fn);
    ssm::AttnReadArgs a{};
    a.batch = batch;
    a.n_table = n_table;
    a.n_tokens = n_tokens;
    a.table_stride = table_stride;
    a.c = make_cache(k_cache, v_cache, k_scale, v_scale, n_pages, page_size, n_kv_heads, head_dim);
    a.page_table = page_table;
    a.cu_len = cu_len;
    a.first = first;
    a.k_out = k_out;
    a.v_out = v_out;
    a.status = status;
    const char* why = "";
    if (ssm::launch_attn_read(a, cache_dtype == SSM_I8, out_dtype == SSM_BF16, static_cast<cudaStream_t>(cuda_stream),
                              &why) != 0)
        return fail(SSM_ERR_CUDA, "%s: %s", fn, why);
    return SSM_OK;
}

int attn_prefill(int batch, int64_t total_q, int64_t total_k, int max_q, int n_q_heads, int n_kv_heads,
                 int head_dim, ssm_dtype_t in_dtype, ssm_dtype_t out_dtype,
                 const void* q, int64_t q_stride_t, int64_t q_stride_h,
                 const void* k, int64_t k_stride_t, int64_t k_stride_h,
                 const void* v, int64_t v_stride_t, int64_t v_stride_h,
                 const int32_t* cu_q, const int32_t* cu_k, float scale,
                 void* out, int64_t out_stride_t, int64_t out_stride_h, float* lse, void* cuda_stream) {
    static const char* fn = "attn_prefill";
    g_err[0] = 0;
    int rc;
    if (batch < 1 || batch > 65535) return fail(SSM_ERR_INVALID_ARG, "%s: batch %d not in [1, 65535]", fn, batch);
    if (total_q < 0 || total_q > (1LL << 30) || total_k < 0 || total_k > (1LL << 30))
        return fail(SSM_ERR_INVALID_ARG, "%s: total_q %lld, total_k %lld not in [0, 2^30]", fn, (long long)total_q, (long long)total_k);
    if (max_q < 0) return fail(SSM_ERR_INVALID_ARG, "%s: max_q %d < 0", fn, max_q);
    if ((rc = check_heads(fn, n_q_heads, n_kv_heads, head_dim)) != SSM_OK) return rc;
    if (!dtype_ok(in_dtype) || !dtype_ok(out_dtype)) return fail(SSM_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (in_dtype != SSM_BF16) return fail(SSM_ERR_UNSUPPORTED, "%s: q, k and v must be bf16", fn);
    if (!(scale > 0.0f) || !(scale - scale == 0.0f)) return fail(SSM_ERR_INVALID_ARG, "%s: scale must be finite and > 0", fn);
    if (!cu_q || !cu_k) return fail(SSM_ERR_INVALID_ARG, "%s: cu_q or cu_k is NULL", fn);
    if (total_q == 0 || max_q == 0) return SSM_OK;
    // the grid counts (256 query rows, sequence, head) items, up to eight CTAs each, in 31 bits
    const int64_t rows = max_q < total_q ? max_q : total_q;
    if ((rows + 255) / 256 * batch >= (1LL << 31) / 8 / n_q_heads)
        return fail(SSM_ERR_UNSUPPORTED, "%s: %d sequences of up to %lld rows and %d heads pass the grid", fn, batch,
                    (long long)rows, n_q_heads);
    if ((rc = check_view(fn, "q", q, q_stride_t, q_stride_h, head_dim)) != SSM_OK) return rc;
    if (total_k > 0) {
        if ((rc = check_view(fn, "k", k, k_stride_t, k_stride_h, head_dim)) != SSM_OK) return rc;
        if ((rc = check_view(fn, "v", v, v_stride_t, v_stride_h, head_dim)) != SSM_OK) return rc;
    }
    if ((rc = check_out_view(fn, "out", out, total_q, out_stride_t, out_stride_h, n_q_heads, head_dim)) != SSM_OK) return rc;
    if (!aligned(cu_q, 4) || !aligned(cu_k, 4) || (lse && !aligned(lse, 4)))
        return fail(SSM_ERR_MISALIGNED, "%s: cu_q, cu_k or lse is not element aligned", fn);
    int serr = 0;
    unsigned int* status = status_ptr(&serr);
    if (serr) return fail(SSM_ERR_CUDA, "%s: no usable CUDA device", fn);
    ssm::AttnPrefillArgs a{};
    a.batch = batch;
    a.max_q = max_q < total_q ? max_q : (int)total_q;
    a.n_q = n_q_heads;
    a.n_kv = n_kv_heads;
    a.dim = head_dim;
    a.total_q = total_q;
    a.total_k = total_k;
    a.q = q;
    a.q_st = q_stride_t;
    a.q_sh = q_stride_h;
    a.k = k;
    a.k_st = k_stride_t;
    a.k_sh = k_stride_h;
    a.v = v;
    a.v_st = v_stride_t;
    a.v_sh = v_stride_h;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.scale = scale;
    a.out = out;
    a.o_st = out_stride_t;
    a.o_sh = out_stride_h;
    a.lse = lse;
    a.status = status;
    const char* why = "";
    if (ssm::launch_attn_prefill(a, out_dtype == SSM_BF16, static_cast<cudaStream_t>(cuda_stream), &why) != 0)
        return fail(SSM_ERR_CUDA, "%s: %s", fn, why);
    return SSM_OK;
}

size_t attn_decode_workspace_bytes(int batch, int n_q_heads, int n_kv_heads, int head_dim, int max_len) {
    if (batch < 1 || batch > 65535 || n_kv_heads < 1 || n_kv_heads > 4096 || n_q_heads < 1 || n_q_heads > 65535 ||
        n_q_heads % n_kv_heads != 0 || head_dim < 16 || head_dim > 128 || head_dim % 16 != 0 || max_len < 1 || max_len > (1 << 30))
        return 0;
    return ssm::attn_decode_workspace(batch, n_q_heads, n_kv_heads, head_dim, max_len);
}

int attn_decode_step(int batch, int n_q_heads, int n_kv_heads, int head_dim, ssm_dtype_t in_dtype,
                     ssm_dtype_t out_dtype, const void* q, int64_t q_stride_t, int64_t q_stride_h,
                     ssm_dtype_t cache_dtype, const void* k_cache, const void* v_cache,
                     const float* k_scale, const float* v_scale, int n_pages, int page_size,
                     const int32_t* page_table, int64_t table_stride, int n_table, const int32_t* lens,
                     int max_len, float scale, void* out, int64_t out_stride_t, int64_t out_stride_h,
                     float* lse, void* workspace, size_t workspace_bytes, void* cuda_stream) {
    static const char* fn = "attn_decode_step";
    g_err[0] = 0;
    int rc;
    if (batch < 1 || batch > 65535) return fail(SSM_ERR_INVALID_ARG, "%s: batch %d not in [1, 65535]", fn, batch);
    if (max_len < 1 || max_len > (1 << 30)) return fail(SSM_ERR_INVALID_ARG, "%s: max_len %d not in [1, 2^30]", fn, max_len);
    if ((rc = check_heads(fn, n_q_heads, n_kv_heads, head_dim)) != SSM_OK) return rc;
    if (!dtype_ok(in_dtype) || !dtype_ok(out_dtype)) return fail(SSM_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (in_dtype != SSM_BF16) return fail(SSM_ERR_UNSUPPORTED, "%s: q must be bf16", fn);
    if (!(scale > 0.0f) || !(scale - scale == 0.0f)) return fail(SSM_ERR_INVALID_ARG, "%s: scale must be finite and > 0", fn);
    if ((rc = check_view(fn, "q", q, q_stride_t, q_stride_h, head_dim)) != SSM_OK) return rc;
    if ((rc = check_cache(fn, cache_dtype, k_cache, v_cache, k_scale, v_scale, n_pages, page_size)) != SSM_OK) return rc;
    if ((rc = check_table(fn, page_table, table_stride, n_table)) != SSM_OK) return rc;
    if (!lens) return fail(SSM_ERR_INVALID_ARG, "%s: lens is NULL", fn);
    if ((rc = check_out_view(fn, "out", out, batch, out_stride_t, out_stride_h, n_q_heads, head_dim)) != SSM_OK) return rc;
    if (!aligned(lens, 4) || (lse && !aligned(lse, 4)))
        return fail(SSM_ERR_MISALIGNED, "%s: lens or lse is not element aligned", fn);
    const size_t need = ssm::attn_decode_workspace(batch, n_q_heads, n_kv_heads, head_dim, max_len);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(SSM_ERR_INVALID_ARG, "%s: workspace of %zu bytes given, %zu needed", fn,
                    workspace ? workspace_bytes : (size_t)0, need);
    if (need > 0 && !aligned(workspace, 16)) return fail(SSM_ERR_MISALIGNED, "%s: workspace must be 16-byte aligned", fn);
    int serr = 0;
    unsigned int* status = status_ptr(&serr);
    if (serr) return fail(SSM_ERR_CUDA, "%s: no usable CUDA device", fn);
    ssm::AttnDecodeArgs a{};
    a.batch = batch;
    a.n_q = n_q_heads;
    a.n_table = n_table;
    a.max_len = max_len;
    a.q = q;
    a.q_st = q_stride_t;
    a.q_sh = q_stride_h;
    a.table_stride = table_stride;
    a.c = make_cache(k_cache, v_cache, k_scale, v_scale, n_pages, page_size, n_kv_heads, head_dim);
    a.page_table = page_table;
    a.lens = lens;
    a.scale = scale;
    a.out = out;
    a.o_st = out_stride_t;
    a.o_sh = out_stride_h;
    a.lse = lse;
    a.workspace = workspace;
    a.status = status;
    const char* why = "";
    if (ssm::launch_attn_decode(a, cache_dtype == SSM_I8, out_dtype == SSM_BF16, static_cast<cudaStream_t>(cuda_stream),
                                &why) != 0)
        return fail(SSM_ERR_CUDA, "%s: %s", fn, why);
    return SSM_OK;
}

}  // extern "C"

// ------------------------------------------------------------------ around the mixers of a decode step
namespace {

// Rows of a 2-D view that is read or written eight elements at a time.
int check_rows(const char* fn, const char* name, const void* p, int64_t stride, int64_t width, unsigned align) {
    if (!p) return fail(SSM_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
    if (stride < width) return fail(SSM_ERR_INVALID_ARG, "%s: the row stride of %s is below the row", fn, name);
    if (!aligned(p, align) || stride % 8 != 0)
        return fail(SSM_ERR_MISALIGNED, "%s: %s must be %u-byte aligned with a row stride that is a multiple of 8", fn, name, align);
    return SSM_OK;
}

int check_w4(const char* fn, int64_t N, int64_t K, int group, const void* codes, int64_t ldc, int scale_dtype,
             const void* scales, int64_t lds, const void* zeros, int64_t ldz) {
    if (N < 1 || N > (1LL << 27)) return fail(SSM_ERR_INVALID_ARG, "%s: N %lld not in [1, 2^27]", fn, (long long)N);
    if (group != 32 && group != 64 && group != 128)
        return fail(SSM_ERR_UNSUPPORTED, "%s: group %d unsupported (32, 64 or 128)", fn, group);
    if (K < 1 || K % group != 0) return fail(SSM_ERR_INVALID_ARG, "%s: K %lld is not a multiple of the group %d", fn, (long long)K, group);
    if (K > 32768) return fail(SSM_ERR_UNSUPPORTED, "%s: K %lld above 32768", fn, (long long)K);
    if (!dtype_ok(scale_dtype)) return fail(SSM_ERR_INVALID_ARG, "%s: unknown scale dtype", fn);
    if (!codes || !scales) return fail(SSM_ERR_INVALID_ARG, "%s: codes or scales is NULL", fn);
    if (ldc < K / 2 || lds < K / group || (zeros && ldz < K / group))
        return fail(SSM_ERR_INVALID_ARG, "%s: a row stride of the weight is below the row length", fn);
    if (!aligned(codes, 16) || ldc % 16 != 0 || !aligned(scales, 16) || lds * esize(scale_dtype) % 16 != 0 ||
        (zeros && (!aligned(zeros, 16) || ldz % 16 != 0)))
        return fail(SSM_ERR_MISALIGNED, "%s: rows of codes, scales and zeros must start on 16 bytes", fn);
    return SSM_OK;
}

ssm::W4Weight make_w4(int64_t N, int64_t K, int group, const uint8_t* codes, int64_t ldc, int scale_dtype, const void* scales,
                      int64_t lds, const uint8_t* zeros, int64_t ldz) {
    return ssm::W4Weight{(int)N, (int)K, group, codes, zeros, scales, scale_dtype == SSM_BF16, ldc, lds, ldz};
}

}  // namespace

extern "C" {

int norm_rms(int64_t n_rows, int width, int n_groups, ssm_dtype_t in_dtype, const void* x, int64_t x_stride,
             ssm_dtype_t res_dtype, const void* residual, int64_t res_stride, void* residual_out, int64_t ro_stride,
             const float* weight, float eps, ssm_dtype_t out_dtype, void* out, int64_t out_stride,
             float* out_scale, void* cuda_stream) {
    static const char* fn = "norm_rms";
    g_err[0] = 0;
    int rc;
    if (n_rows < 0) return fail(SSM_ERR_INVALID_ARG, "%s: n_rows %lld < 0", fn, (long long)n_rows);
    if (width < 1 || n_groups < 1 || width % n_groups != 0)
        return fail(SSM_ERR_INVALID_ARG, "%s: %d channels in %d groups", fn, width, n_groups);
    if (width / n_groups % 8 != 0 || width / n_groups > 32768)
        return fail(SSM_ERR_UNSUPPORTED, "%s: a group of %d channels (multiples of 8 up to 32768)", fn, width / n_groups);
    if (n_rows >= (1LL << 31) / n_groups)
        return fail(SSM_ERR_UNSUPPORTED, "%s: %lld rows of %d groups pass 2^31", fn, (long long)n_rows, n_groups);
    if (!dtype_ok(in_dtype) || ((residual || residual_out) && !dtype_ok(res_dtype)) || !(dtype_ok(out_dtype) || out_dtype == SSM_I8))
        return fail(SSM_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (!(eps >= 0.0f) || !(eps - eps == 0.0f)) return fail(SSM_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", fn);
    if (residual_out && !residual) return fail(SSM_ERR_INVALID_ARG, "%s: residual_out needs residual", fn);
    if (n_rows == 0) return SSM_OK;
    if ((rc = check_rows(fn, "x", x, x_stride, width, 16)) != SSM_OK) return rc;
    if (residual && (rc = check_rows(fn, "residual", residual, res_stride, width, 16)) != SSM_OK) return rc;
    if (residual_out && (rc = check_rows(fn, "residual_out", residual_out, ro_stride, width, 16)) != SSM_OK) return rc;
    if (residual_out == residual && residual && ro_stride != res_stride)
        return fail(SSM_ERR_INVALID_ARG, "%s: residual_out is residual with another stride", fn);
    if ((rc = check_rows(fn, "out", out, out_stride, width, out_dtype == SSM_I8 ? 8 : 16)) != SSM_OK) return rc;
    if ((out_dtype == SSM_I8) != (out_scale != nullptr))
        return fail(SSM_ERR_INVALID_ARG, "%s: out_scale goes with an SSM_I8 out", fn);
    if ((weight && !aligned(weight, 16)) || (out_scale && !aligned(out_scale, 4)))
        return fail(SSM_ERR_MISALIGNED, "%s: weight must be 16-byte aligned, out_scale element aligned", fn);
    int serr = 0;
    status_ptr(&serr);
    if (serr) return fail(SSM_ERR_CUDA, "%s: no usable CUDA device", fn);
    ssm::NormArgs a{};
    a.n_rows = n_rows;
    a.width = width;
    a.n_groups = n_groups;
    a.in_type = in_dtype;
    a.res_type = residual ? res_dtype : SSM_BF16;
    a.out_type = out_dtype;
    a.x = x;
    a.residual = residual;
    a.residual_out = residual_out;
    a.out = out;
    a.x_st = x_stride;
    a.res_st = res_stride;
    a.ro_st = ro_stride;
    a.out_st = out_stride;
    a.weight = weight;
    a.eps = eps;
    a.out_scale = out_scale;
    const char* why = "";
    if (ssm::launch_norm_rms(a, static_cast<cudaStream_t>(cuda_stream), &why) != 0) return fail(SSM_ERR_CUDA, "%s: %s", fn, why);
    return SSM_OK;
}

int w4_quantize(int64_t N, int64_t K, int group, ssm_dtype_t in_dtype, const void* W, int64_t ldw,
                uint8_t* codes, int64_t ldc, ssm_dtype_t scale_dtype, void* scales, int64_t lds,
                uint8_t* zeros, int64_t ldz, void* cuda_stream) {
    static const char* fn = "w4_quantize";
    g_err[0] = 0;
    const int rc = check_w4(fn, N, K, group, codes, ldc, scale_dtype, scales, lds, zeros, ldz);
    if (rc != SSM_OK) return rc;
    if (!dtype_ok(in_dtype)) return fail(SSM_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (!W) return fail(SSM_ERR_INVALID_ARG, "%s: W is NULL", fn);
    if (ldw < K) return fail(SSM_ERR_INVALID_ARG, "%s: ldw is below K", fn);
    if (!aligned(W, esize(in_dtype))) return fail(SSM_ERR_MISALIGNED, "%s: W is not element aligned", fn);
    int serr = 0;
    status_ptr(&serr);
    if (serr) return fail(SSM_ERR_CUDA, "%s: no usable CUDA device", fn);
    const char* why = "";
    if (ssm::launch_w4_quantize(make_w4(N, K, group, codes, ldc, scale_dtype, scales, lds, zeros, ldz), W, ldw,
                                in_dtype == SSM_BF16, static_cast<cudaStream_t>(cuda_stream), &why) != 0)
        return fail(SSM_ERR_CUDA, "%s: %s", fn, why);
    return SSM_OK;
}

size_t w4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int group) {
    if (M < 1 || M > 256 || N < 1 || N > (1LL << 27) || (group != 32 && group != 64 && group != 128) || K < 1 || K % group != 0 || K > 32768)
        return 0;
    return ssm::w4_linear_workspace((int)M, make_w4(N, K, group, nullptr, 0, SSM_F32, nullptr, 0, nullptr, 0));
}

int w4_linear(int64_t M, int64_t N, int64_t K, int group, ssm_dtype_t x_dtype, const void* x, int64_t ldx,
              const float* x_scale, int x_blocks, const uint8_t* codes, int64_t ldc,
              ssm_dtype_t scale_dtype, const void* scales, int64_t lds, const uint8_t* zeros, int64_t ldz,
              ssm_dtype_t out_dtype, void* out, int64_t ldo, void* workspace, size_t workspace_bytes, void* cuda_stream) {
    static const char* fn = "w4_linear";
    g_err[0] = 0;
    if (M < 0) return fail(SSM_ERR_INVALID_ARG, "%s: M %lld < 0", fn, (long long)M);
    if (M > 256) return fail(SSM_ERR_UNSUPPORTED, "%s: M %lld above 256", fn, (long long)M);
    const int rc = check_w4(fn, N, K, group, codes, ldc, scale_dtype, scales, lds, zeros, ldz);
    if (rc != SSM_OK) return rc;
    if (x_dtype != SSM_BF16 && x_dtype != SSM_I8)
        return fail(x_dtype == SSM_F32 ? SSM_ERR_UNSUPPORTED : SSM_ERR_INVALID_ARG, "%s: x must be SSM_BF16 or SSM_I8", fn);
    if (!dtype_ok(out_dtype)) return fail(SSM_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (M == 0) return SSM_OK;
    if (!x || !out) return fail(SSM_ERR_INVALID_ARG, "%s: x or out is NULL", fn);
    if (ldx < K || ldo < N) return fail(SSM_ERR_INVALID_ARG, "%s: a row stride of x or out is below the row length", fn);
    if (!aligned(x, 16) || ldx * (x_dtype == SSM_I8 ? 1 : 2) % 16 != 0)
        return fail(SSM_ERR_MISALIGNED, "%s: rows of x must start on 16 bytes", fn);
    if ((x_dtype == SSM_I8) != (x_scale != nullptr)) return fail(SSM_ERR_INVALID_ARG, "%s: x_scale goes with SSM_I8 x", fn);
    if (x_blocks < 1 || x_blocks > 64 || (!x_scale && x_blocks != 1) || K % ((int64_t)x_blocks * group) != 0)
        return fail(SSM_ERR_INVALID_ARG, "%s: %d blocks of x (1 to 64 for SSM_I8, each a multiple of the group)", fn, x_blocks);
    if (!aligned(out, esize(out_dtype)) || (x_scale && !aligned(x_scale, 4)))
        return fail(SSM_ERR_MISALIGNED, "%s: out or x_scale is not element aligned", fn);
    const ssm::W4Weight w = make_w4(N, K, group, codes, ldc, scale_dtype, scales, lds, zeros, ldz);
    const size_t need = ssm::w4_linear_workspace((int)M, w);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(SSM_ERR_INVALID_ARG, "%s: workspace of %zu bytes given, %zu needed", fn,
                    workspace ? workspace_bytes : (size_t)0, need);
    if (need > 0 && !aligned(workspace, 16)) return fail(SSM_ERR_MISALIGNED, "%s: workspace must be 16-byte aligned", fn);
    int serr = 0;
    unsigned int* status = status_ptr(&serr);
    if (serr) return fail(SSM_ERR_CUDA, "%s: no usable CUDA device", fn);
    ssm::W4LinearArgs a{};
    a.M = (int)M;
    a.w = w;
    a.x = x;
    a.x_i8 = x_dtype == SSM_I8;
    a.out_bf16 = out_dtype == SSM_BF16;
    a.ldx = ldx;
    a.x_scale = x_scale;
    a.x_blocks = x_blocks;
    a.out = out;
    a.ldo = ldo;
    a.parts = static_cast<float*>(workspace);
    const char* why = "";
    if (ssm::launch_w4_linear(a, status, static_cast<cudaStream_t>(cuda_stream), &why) != 0) return fail(SSM_ERR_CUDA, "%s: %s", fn, why);
    return SSM_OK;
}

int spec_probs(int64_t n_rows, int64_t vocab, ssm_dtype_t in_dtype, const void* logits, int64_t ld_in,
               const float* temperature, float* probs, int64_t ld_out, void* cuda_stream) {
    static const char* fn = "spec_probs";
    g_err[0] = 0;
    if (n_rows < 0 || n_rows >= (1LL << 28)) return fail(SSM_ERR_INVALID_ARG, "%s: n_rows %lld not in [0, 2^28)", fn, (long long)n_rows);
    if (vocab < 1 || vocab > (1LL << 24)) return fail(SSM_ERR_INVALID_ARG, "%s: vocab %lld not in [1, 2^24]", fn, (long long)vocab);
    if (!dtype_ok(in_dtype)) return fail(SSM_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (n_rows == 0) return SSM_OK;
    if (!logits || !probs) return fail(SSM_ERR_INVALID_ARG, "%s: logits or probs is NULL", fn);
    if (ld_in < vocab || ld_out < vocab) return fail(SSM_ERR_INVALID_ARG, "%s: a row stride is below vocab", fn);
    if (!aligned(logits, esize(in_dtype)) || !aligned(probs, 4) || (temperature && !aligned(temperature, 4)))
        return fail(SSM_ERR_MISALIGNED, "%s: a tensor is not element aligned", fn);
    int serr = 0;
    unsigned int* status = status_ptr(&serr);
    if (serr) return fail(SSM_ERR_CUDA, "%s: no usable CUDA device", fn);
    const ssm::ProbsArgs a{n_rows, vocab, logits, ld_in, ld_out, temperature, probs, status};
    const char* why = "";
    if (ssm::launch_spec_probs(a, in_dtype == SSM_BF16, static_cast<cudaStream_t>(cuda_stream), &why) != 0)
        return fail(SSM_ERR_CUDA, "%s: %s", fn, why);
    return SSM_OK;
}

int spec_verify(int batch, int n_max, int64_t vocab, const int32_t* draft, const int32_t* n_draft,
                const float* target_probs, int64_t tp_stride_b, int64_t tp_stride_t,
                const float* draft_probs, int64_t dp_stride_b, int64_t dp_stride_t, const float* u,
                int32_t* tokens, int32_t* n_kept, void* cuda_stream) {
    static const char* fn = "spec_verify";
    g_err[0] = 0;
    if (batch < 0 || batch > 65535) return fail(SSM_ERR_INVALID_ARG, "%s: batch %d not in [0, 65535]", fn, batch);
    if (n_max < 0 || n_max > 1024) return fail(SSM_ERR_INVALID_ARG, "%s: n_max %d not in [0, 1024]", fn, n_max);
    if (vocab < 1 || vocab > (1LL << 24)) return fail(SSM_ERR_INVALID_ARG, "%s: vocab %lld not in [1, 2^24]", fn, (long long)vocab);
    if (batch == 0) return SSM_OK;
    if ((n_max > 0 && !draft) || !target_probs || !u || !tokens || !n_kept)
        return fail(SSM_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (tp_stride_t < vocab || tp_stride_b < vocab || (draft_probs && n_max > 0 && (dp_stride_t < vocab || dp_stride_b < vocab)))
        return fail(SSM_ERR_INVALID_ARG, "%s: a stride of the probabilities is below vocab", fn);
    for (const void* p : {(const void*)draft, (const void*)n_draft, (const void*)target_probs, (const void*)draft_probs,
                          (const void*)u, (const void*)tokens, (const void*)n_kept})
        if (!aligned(p, 4)) return fail(SSM_ERR_MISALIGNED, "%s: a tensor is not element aligned", fn);
    int serr = 0;
    unsigned int* status = status_ptr(&serr);
    if (serr) return fail(SSM_ERR_CUDA, "%s: no usable CUDA device", fn);
    const ssm::VerifyArgs a{batch, n_max, vocab, draft, n_draft, target_probs, n_max > 0 ? draft_probs : nullptr, u,
                            tp_stride_b, tp_stride_t, dp_stride_b, dp_stride_t, tokens, n_kept, status};
    const char* why = "";
    if (ssm::launch_spec_verify(a, static_cast<cudaStream_t>(cuda_stream), &why) != 0) return fail(SSM_ERR_CUDA, "%s: %s", fn, why);
    return SSM_OK;
}

}  // extern "C"
