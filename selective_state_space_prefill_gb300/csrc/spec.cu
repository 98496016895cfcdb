// spec.cu -- spec_probs (probabilities of logits at a temperature) and spec_verify (drafted tokens against the
// target's probabilities).
//
// First forms: a CTA per row, and a CTA per request.
#include "common.cuh"
#include "kernels.h"
#include "ssm.h"

namespace ssm {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;

// ------------------------------------------------------------------ probabilities
template <typename T>
__global__ void __launch_bounds__(kThreads) k_spec_probs(const ProbsArgs a) {
    __shared__ float s_m[kWarps], s_l[kWarps];
    __shared__ int s_i[kWarps];
    const int64_t row = blockIdx.x;
    const T* x = reinterpret_cast<const T*>(a.logits) + row * a.ld_in;
    float* p = a.probs + row * a.ld_out;
    const float t = a.temperature ? a.temperature[row] : 1.f;
    const bool greedy = t <= 0x1p-100f;
    // the maximum and its first place; a NaN wins
    float m = -INFINITY;
    int at = 0x7fffffff;
    for (int i = threadIdx.x; i < a.vocab; i += kThreads) {
        const float v = to_f32(x[i]);
        if (!(v <= m)) {
            if (m == m) m = v, at = i;
        }
    }
    for (int o = 16; o > 0; o >>= 1) {
        const float v = __shfl_xor_sync(~0u, m, o);
        const int j = __shfl_xor_sync(~0u, at, o);
        if (v != v || v > m || (v == m && j < at)) m = m != m ? m : v, at = j;
    }
    if (threadIdx.x % 32 == 0) s_m[threadIdx.x / 32] = m, s_i[threadIdx.x / 32] = at;
    __syncthreads();
    m = s_m[0], at = s_i[0];
    for (int w = 1; w < kWarps; ++w) {
        const float v = s_m[w];
        const int j = s_i[w];
        if (v != v || v > m || (v == m && j < at)) m = m != m ? m : v, at = j;
    }
    if (!(m < INFINITY) || t != t) {                     // NaN or +inf
        for (int i = threadIdx.x; i < a.vocab; i += kThreads) p[i] = __uint_as_float(0x7fc00000u);
        return;
    }
    if (greedy || m == -INFINITY) {
        for (int i = threadIdx.x; i < a.vocab; i += kThreads) p[i] = i == at && m > -INFINITY ? 1.f : 0.f;
        return;
    }
    const float f = __fdiv_rn(1.f, fminf(t, 3.0e38f)) * kLog2e;
    float l = 0.f;
    for (int i = threadIdx.x; i < a.vocab; i += kThreads) l += ex2((to_f32(x[i]) - m) * f);
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
    if (threadIdx.x % 32 == 0) s_l[threadIdx.x / 32] = l;
    __syncthreads();
    l = 0.f;
    for (int w = 0; w < kWarps; ++w) l += s_l[w];
    const float inv = __fdiv_rn(1.f, l);
    for (int i = threadIdx.x; i < a.vocab; i += kThreads) p[i] = ex2((to_f32(x[i]) - m) * f) * inv;
}

// ------------------------------------------------------------------ verification
// A probability as an integer of 2^-62; negative ones and NaN are 0.
__device__ __forceinline__ uint64_t fixed(float p) { return p > 0.f ? __float2ull_rz(p * 0x1p62f) : 0ull; }

// The row that the next token is drawn from, element by element.
struct Mass {
    const float *p, *q;
    int64_t off;
    __device__ __forceinline__ uint64_t operator()(int64_t i) const {
        const uint64_t a = fixed(p[i]), b = q ? fixed(q[i]) : i == off ? 1ull << 62 : 0ull;
        return a > b ? a - b : 0ull;
    }
};

__global__ void __launch_bounds__(kThreads) k_spec_verify(const VerifyArgs a) {
    __shared__ int s_kept, s_n;
    __shared__ uint64_t s_sum[kWarps];
    __shared__ float s_mag[kWarps];
    const int b = blockIdx.x, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int32_t* draft = a.draft + (int64_t)b * a.n_max;
    const float* u = a.u + (int64_t)b * (a.n_max + 1);
    if (warp == 0) {
        int n = a.n_draft ? a.n_draft[b] : a.n_max;
        bool bad = n < 0 || n > a.n_max;
        n = n < 0 ? 0 : n > a.n_max ? a.n_max : n;
        int kept = n;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int i = i0 + lane;
            bool no = false, out = false;
            if (i < n) {
                const int d = draft[i];
                out = d < 0 || d >= a.vocab;
                const float v = u[i], uu = v > 0.f ? fminf(v, 0x1.fffffep-1f) : 0.f;
                float pd = out ? 0.f : a.p[b * a.p_sb + i * a.p_st + d], qd = 1.f;
                if (a.q) qd = out ? 0.f : a.q[b * a.q_sb + i * a.q_st + d];
                pd = pd > 0.f ? pd : 0.f, qd = qd > 0.f ? qd : 0.f;
                no = !((double)uu * qd < (double)pd);       // 24 x 24 bits: exact
            }
            const unsigned first = __ballot_sync(~0u, no), outs = __ballot_sync(~0u, out);
            if (first) kept = i0 + __ffs(first) - 1;
            bad |= (outs & (first ? first ^ (first - 1) : ~0u)) != 0;   // those up to the first not kept
            if (first) break;
        }
        if (lane == 0) {
            s_kept = kept, s_n = n;
            if (bad) atomicOr(a.status, (unsigned)SSM_DEV_BAD_INDEX);
        }
    }
    __syncthreads();
    const int kept = s_kept, n = s_n;
    Mass w{a.p + b * a.p_sb + kept * a.p_st, nullptr, -1};
    if (kept < n) {
        if (a.q) w.q = a.q + b * a.q_sb + kept * a.q_st;
        else w.off = draft[kept];
    }
    const int64_t per = (a.vocab + kWarps - 1) / kWarps, lo = warp * per, hi = lo + per < a.vocab ? lo + per : a.vocab;
    uint64_t total;
    float mag;
    for (int turn = 0;; ++turn) {
        uint64_t sum = 0;
        mag = 0.f;
        for (int64_t i = lo + lane; i < hi; i += 32) {
            const float v = w.p[i];
            sum += w(i), mag += v > 0.f ? v : 0.f;
        }
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o), mag += __shfl_xor_sync(~0u, mag, o);
        __syncthreads();
        if (lane == 0) s_sum[warp] = sum, s_mag[warp] = mag;
        __syncthreads();
        total = 0, mag = 0.f;
        for (int i = 0; i < kWarps; ++i) total += s_sum[i], mag += s_mag[i];
        if (total > 0 || turn == 1 || (!w.q && w.off < 0)) break;
        w.q = nullptr, w.off = -1;                      // nothing left of p - q: p itself
    }
    const float v = u[a.n_max], uu = v > 0.f ? fminf(v, 0x1.fffffep-1f) : 0.f;
    // the first index whose running sum exceeds floor(u * total)
    const uint64_t border = __umul64hi(__float2ull_rz(uu * 0x1p64f), total);
    int32_t* out = a.tokens + (int64_t)b * (a.n_max + 1);
    uint64_t before = 0;
    for (int i = 0; i < warp; ++i) before += s_sum[i];
    const bool some = total > 0 && mag < 3.99f;
    if (some && before <= border && border < before + s_sum[warp]) {
        for (int64_t i0 = lo; i0 < hi; i0 += 32) {
            uint64_t c = i0 + lane < hi ? w(i0 + lane) : 0ull;
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t t = __shfl_up_sync(~0u, c, o);
                if (lane >= o) c += t;
            }
            const unsigned over = __ballot_sync(~0u, before + c > border);
            if (over) {
                if (lane == 0) out[kept] = (int32_t)(i0 + __ffs(over) - 1);
                break;
            }
            before += __shfl_sync(~0u, c, 31);
        }
    }
    if (threadIdx.x == 0) {
        a.n_kept[b] = kept;
        if (!some) out[kept] = -1;
    }
    for (int i = threadIdx.x; i <= a.n_max; i += kThreads)
        if (i != kept) out[i] = i < kept ? draft[i] : -1;
}

int done(const char** why) {
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return 0;
    *why = cudaGetErrorString(e);
    return -1;
}

}  // namespace

int launch_spec_probs(const ProbsArgs& a, bool in_bf16, cudaStream_t stream, const char** why) {
    if (in_bf16) k_spec_probs<__nv_bfloat16><<<(unsigned)a.n_rows, kThreads, 0, stream>>>(a);
    else k_spec_probs<float><<<(unsigned)a.n_rows, kThreads, 0, stream>>>(a);
    return done(why);
}

int launch_spec_verify(const VerifyArgs& a, cudaStream_t stream, const char** why) {
    k_spec_verify<<<(unsigned)a.batch, kThreads, 0, stream>>>(a);
    return done(why);
}

}  // namespace ssm
