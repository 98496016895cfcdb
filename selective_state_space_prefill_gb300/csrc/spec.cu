// spec.cu -- spec_probs (probabilities of logits at a temperature) and spec_verify (drafted tokens against the
// target's probabilities).
//
// Both read rows of the vocabulary's length, a few or hundreds of them: a row is a thread-block cluster's, cut into
// a slice per CTA, and what the CTAs have to know of each other (a maximum, sums) goes through distributed shared
// memory.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"
#include "ssm.h"

namespace cg = cooperative_groups;

namespace ssm {
namespace {

constexpr int kSms = 152;

// ------------------------------------------------------------------ probabilities
// The larger one; a NaN wins.
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}
__device__ __forceinline__ float quiet_nan() { return __uint_as_float(0x7fc00000u); }

// One float, whatever stands beside it: plain stores of four neighbours, next to one of them as a float4 in the other
// branch, came out as one 16-byte store, which faults where the row is not aligned.
__device__ __forceinline__ void store1(float* p, float v) { asm volatile("st.global.f32 [%0], %1;" ::"l"(p), "f"(v) : "memory"); }

// What a row's CTAs find out together: every CTA's value in its shared memory, combined by every thread.
enum Kind { kMax, kSum, kLeast };
template <Kind K, typename T>
__device__ __forceinline__ T two(T a, T b) {
    if constexpr (K == kMax) return max_nan(a, b);
    else if constexpr (K == kSum) return a + b;
    else return a < b ? a : b;
}
template <Kind K, int kWarps, typename T>
__device__ T row_wide(T v, T* s_warp, T* s_cta, int ctas) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = two<K>(v, __shfl_xor_sync(~0u, v, o));
    if (threadIdx.x % 32 == 0) s_warp[threadIdx.x / 32] = v;
    __syncthreads();
    v = s_warp[threadIdx.x % kWarps];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) v = two<K>(v, __shfl_xor_sync(~0u, v, o));
    if (ctas == 1) return v;
    auto cluster = cg::this_cluster();
    if (threadIdx.x == 0) *s_cta = v;
    cluster.sync();
    v = *cluster.map_shared_rank(s_cta, threadIdx.x % ctas);
    for (int o = ctas / 2; o > 0; o >>= 1) v = two<K>(v, __shfl_xor_sync(~0u, v, o));
    return v;
}

// Eight logits as they came.
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> {
    uint4 q;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { q = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void none() { q = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }   // -inf
    __device__ __forceinline__ float most() const {     // of the eight; a NaN wins
        const uint32_t m = max2(max2(q.x, q.y), max2(q.z, q.w));
        return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t m;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
        return m;
    }
    __device__ __forceinline__ float at(int k) const {
        const uint32_t w = k / 2 == 0 ? q.x : k / 2 == 1 ? q.y : k / 2 == 2 ? q.z : q.w;
        return __uint_as_float(k % 2 ? w & 0xffff0000u : w << 16);
    }
};
template <> struct Raw<float> {
    float4 q[2];
    __device__ __forceinline__ void load(const float* p) {
        q[0] = __ldg(reinterpret_cast<const float4*>(p)), q[1] = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void none() { q[0] = q[1] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY); }
    __device__ __forceinline__ float most() const {
        float m = at(0);
#pragma unroll
        for (int k = 1; k < 8; ++k) m = max_nan(m, at(k));
        return m;
    }
    __device__ __forceinline__ float at(int k) const {
        const float4& v = q[k / 4];
        return k % 4 == 0 ? v.x : k % 4 == 1 ? v.y : k % 4 == 2 ? v.z : v.w;
    }
};

// A row stays in registers, as it came, between its maximum, its sum and its output: read once, written once.  (The
// powers are taken twice: their unit would do three times as many in the time that the row's bytes take.)  V
// vectors of eight logits a thread, from the row's first 16-byte border on; what lies before that and behind the
// last whole vector (up to 14 logits) is one logit each for the first CTA's first threads.
template <typename T, int V, int kThreads>
__global__ void __launch_bounds__(kThreads, V * sizeof(T) <= 16 ? 1024 / kThreads : 1) k_spec_probs(const ProbsArgs a, int ctas) {
    constexpr int kWarps = kThreads / 32;
    __shared__ float s_max[kWarps], s_sum[kWarps], s_max_cta, s_sum_cta;
    __shared__ int s_at[kWarps], s_at_cta;
    const int64_t row = blockIdx.x / (unsigned)ctas;
    const int rank = blockIdx.x % (unsigned)ctas, vocab = (int)a.vocab;
    const T* x = reinterpret_cast<const T*>(a.logits) + row * a.ld_in;
    float* p = a.probs + row * a.ld_out;
    const float t = a.temperature ? a.temperature[row] : 1.f;
    int head = (int)((16 - reinterpret_cast<uintptr_t>(x) % 16) % 16 / sizeof(T));
    if (head > vocab) head = vocab;
    const int vecs = (vocab - head) / 8, edge = vocab - 8 * vecs;
    const int per = (vecs + ctas - 1) / ctas, first = rank * per, mine = min(per, vecs - first);
    Raw<T> v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int at = threadIdx.x + i * kThreads;
        if (at < mine) v[i].load(x + head + 8 * (first + at));
        else v[i].none();
    }
    const bool on_edge = rank == 0 && threadIdx.x < edge;
    const int w_at = threadIdx.x < head ? threadIdx.x : threadIdx.x + 8 * vecs;
    const float w = on_edge ? to_f32(x[w_at]) : -INFINITY;
    float m = w;
#pragma unroll
    for (int i = 0; i < V; ++i) m = max_nan(m, v[i].most());
    m = row_wide<kMax, kWarps>(m, s_max, &s_max_cta, ctas);

    // p = 2^((x - m) f) inv, or 1 at one place, or the same everywhere
    float f = 0.f, inv = quiet_nan();
    int least = -1;
    if (!(m < INFINITY) || t != t) {                    // NaN or +inf among the logits: NaN
    } else if (t <= 0x1p-100f || m == -INFINITY) {      // greedy: 1 at the first largest; nothing to choose from: zeros
        inv = 0.f;
        least = 0x7fffffff;
        if (m > -INFINITY) {
            if (on_edge && w == m) least = w_at;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (v[i].at(k) == m) least = min(least, head + 8 * (first + (int)threadIdx.x + i * kThreads) + k);
        }
        least = row_wide<kLeast, kWarps>(least, s_at, &s_at_cta, ctas);
    } else {
        f = __fdiv_rn(1.f, fminf(t, 3.0e38f)) * kLog2e;
        float l = ex2((w - m) * f);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) l += ex2((v[i].at(k) - m) * f);
        inv = __fdiv_rn(1.f, row_wide<kSum, kWarps>(l, s_sum, &s_sum_cta, ctas));
    }
    const int start = head + 8 * first;
    const bool whole = reinterpret_cast<uintptr_t>(p + start) % 16 == 0;
    auto write = [&](auto prob) {
        if (on_edge) p[w_at] = prob(w, w_at);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int at = threadIdx.x + i * kThreads;
            if (at >= mine) break;
#pragma unroll
            for (int k = 0; k < 8; k += 4) {
                const int n = start + 8 * at + k;
                const float4 o = make_float4(prob(v[i].at(k), n), prob(v[i].at(k + 1), n + 1), prob(v[i].at(k + 2), n + 2),
                                             prob(v[i].at(k + 3), n + 3));
                if (whole) *reinterpret_cast<float4*>(p + n) = o;
                else store1(p + n, o.x), store1(p + n + 1, o.y), store1(p + n + 2, o.z), store1(p + n + 3, o.w);
            }
        }
    };
    if (f > 0.f) write([&](float x, int) { return ex2((x - m) * f) * inv; });
    else write([&](float, int at) { return at == least ? 1.f : inv; });
    if (ctas > 1) cg::this_cluster().sync();            // no CTA leaves while its values are read
}

// Rows longer than a cluster's registers hold: read three times, from L2 after the first.
template <typename T>
__global__ void __launch_bounds__(512) k_spec_probs_long(const ProbsArgs a, int ctas) {
    constexpr int kThreads = 512, kWarps = kThreads / 32;
    __shared__ float s_max[kWarps], s_sum[kWarps], s_max_cta, s_sum_cta;
    __shared__ int s_at[kWarps], s_at_cta;
    const int64_t row = blockIdx.x / (unsigned)ctas;
    const int rank = blockIdx.x % (unsigned)ctas, vocab = (int)a.vocab;
    const T* x = reinterpret_cast<const T*>(a.logits) + row * a.ld_in;
    float* p = a.probs + row * a.ld_out;
    const float t = a.temperature ? a.temperature[row] : 1.f;
    const int per = (vocab + ctas - 1) / ctas, lo = rank * per, hi = min(lo + per, vocab);
    float m = -INFINITY;
#pragma unroll 8
    for (int i = lo + threadIdx.x; i < hi; i += kThreads) m = max_nan(m, to_f32(x[i]));
    m = row_wide<kMax, kWarps>(m, s_max, &s_max_cta, ctas);
    if (!(m < INFINITY) || t != t) {
        for (int i = lo + threadIdx.x; i < hi; i += kThreads) p[i] = quiet_nan();
    } else if (t <= 0x1p-100f || m == -INFINITY) {
        int least = 0x7fffffff;
#pragma unroll 8
        for (int i = lo + threadIdx.x; i < hi; i += kThreads)
            if (to_f32(x[i]) == m && m > -INFINITY) least = min(least, i);
        least = row_wide<kLeast, kWarps>(least, s_at, &s_at_cta, ctas);
        for (int i = lo + threadIdx.x; i < hi; i += kThreads) p[i] = i == least ? 1.f : 0.f;
    } else {
        const float f = __fdiv_rn(1.f, fminf(t, 3.0e38f)) * kLog2e;
        float l = 0.f;
#pragma unroll 8
        for (int i = lo + threadIdx.x; i < hi; i += kThreads) l += ex2((to_f32(x[i]) - m) * f);
        l = row_wide<kSum, kWarps>(l, s_sum, &s_sum_cta, ctas);
        const float inv = __fdiv_rn(1.f, l);
#pragma unroll 8
        for (int i = lo + threadIdx.x; i < hi; i += kThreads) p[i] = ex2((to_f32(x[i]) - m) * f) * inv;
    }
    if (ctas > 1) cg::this_cluster().sync();
}

// ------------------------------------------------------------------ verification
// A probability as an integer of 2^-62, cut off: the mantissa with its leading one at the top of 64 bits, which is
// right for [2, 4), shifted down by what the exponent is below that.  Negative ones and NaN shift by more than 64
// and are 0, as is what is too small.  (A conversion to 64 bits is an instruction, but one that this GPU does at
// a few elements a clock.)
__device__ __forceinline__ uint64_t fixed(float p) {
    const uint32_t bits = __float_as_uint(p);
    uint64_t v;
    asm("shr.u64 %0, %1, %2;" : "=l"(v) : "l"((uint64_t)(bits << 8 | 0x80000000u) << 32), "r"(128u - (bits >> 23)));
    return v;
}
__device__ __forceinline__ float uniform(float v) { return v > 0.f ? fminf(v, 0x1.fffffep-1f) : 0.f; }

// The row that the next token is drawn from, element by element.
struct Mass {
    const float *p, *q;
    int off;
    __device__ __forceinline__ uint64_t less(float pv, float qv, int i) const {
        const uint64_t x = fixed(pv), y = q ? fixed(qv) : i == off ? 1ull << 62 : 0ull;
        return x > y ? x - y : 0ull;
    }
};

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// A cluster per request.  Sums are exact integers, so that the order of their parts and the cut do not matter: a
// warp sums a stretch of the row, and the warp in whose stretch the border falls reads that again (from L2).
constexpr int kVerifyThreads = 256;
__global__ void __launch_bounds__(kVerifyThreads, 4) k_spec_verify(const VerifyArgs a, int ctas) {
    constexpr int kThreads = kVerifyThreads, kWarps = kThreads / 32;
    constexpr int kBlock = 256;                         // elements that a warp takes at a time, eight loads a lane
    __shared__ int s_kept, s_n;
    __shared__ uint64_t s_sum[kWarps], s_total;
    __shared__ float s_mag[kWarps], s_mags;
    const int b = blockIdx.x / (unsigned)ctas, rank = blockIdx.x % (unsigned)ctas;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, vocab = (int)a.vocab;
    const int32_t* draft = a.draft + (int64_t)b * a.n_max;
    const float* u = a.u + (int64_t)b * (a.n_max + 1);
    const float draw = uniform(u[a.n_max]);             // asked for now, used at the end
    if (warp == 0) {
        const int d0 = lane < a.n_max ? draft[lane] : 0;                // as n_draft, not after it
        int n = a.n_draft ? a.n_draft[b] : a.n_max;
        bool bad = n < 0 || n > a.n_max;
        n = n < 0 ? 0 : n > a.n_max ? a.n_max : n;
        int kept = n;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int i = i0 + lane;
            bool no = false, out = false;
            if (i < n) {
                const int d = i0 == 0 ? d0 : draft[i];
                out = d < 0 || d >= vocab;
                float pd = out ? 0.f : a.p[b * a.p_sb + i * a.p_st + d], qd = 1.f;
                if (a.q) qd = out ? 0.f : a.q[b * a.q_sb + i * a.q_st + d];
                pd = pd > 0.f ? pd : 0.f, qd = qd > 0.f ? qd : 0.f;
                no = !((double)uniform(u[i]) * qd < (double)pd);        // 24 x 24 bits: exact
            }
            const unsigned first = __ballot_sync(~0u, no), outs = __ballot_sync(~0u, out);
            if (first) kept = i0 + __ffs(first) - 1;
            bad |= (outs & (first ? first ^ (first - 1) : ~0u)) != 0;   // those up to the first not kept
            if (first) break;
        }
        if (lane == 0) {
            s_kept = kept, s_n = n;
            if (bad && rank == 0) atomicOr(a.status, (unsigned)SSM_DEV_BAD_INDEX);
        }
    }
    __syncthreads();
    const int kept = s_kept, n = s_n;
    int32_t* out = a.tokens + (int64_t)b * (a.n_max + 1);
    if (rank == 0) {
        for (int i = threadIdx.x; i <= a.n_max; i += kThreads)
            if (i != kept) out[i] = i < kept ? draft[i] : -1;
        if (threadIdx.x == 0) a.n_kept[b] = kept;
    }
    Mass w{a.p + b * a.p_sb + kept * a.p_st, nullptr, -1};
    if (kept < n) {
        if (a.q) w.q = a.q + b * a.q_sb + kept * a.q_st;
        else w.off = draft[kept];
    }
    const int stretches = ctas * kWarps, per = (vocab + stretches - 1) / stretches;
    const int lo = min(vocab, (rank * kWarps + warp) * per), hi = min(vocab, lo + per);
    // a block's elements of this lane, all loads under way at once
    constexpr int kEach = kBlock / 32;
    auto load = [&](int i0, float (&pv)[kEach], float (&qv)[kEach]) {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = i0 + 32 * k + lane;
            pv[k] = i < hi ? w.p[i] : 0.f;
            qv[k] = w.q && i < hi ? w.q[i] : 0.f;
        }
    };
    float pv[kEach], qv[kEach];
    uint64_t total, before;
    float mags;
    for (int turn = 0;; ++turn) {
        uint64_t sum = 0;
        float mag = 0.f;
        load(lo, pv, qv);
        for (int i0 = lo; i0 < hi; i0 += kBlock) {      // the next block comes while this one is summed
            float pn[kEach], qn[kEach];
            load(i0 + kBlock, pn, qn);
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                sum += w.less(pv[k], qv[k], i0 + 32 * k + lane);
                mag += pv[k] > 0.f ? pv[k] : 0.f;
                pv[k] = pn[k], qv[k] = qn[k];
            }
        }
        sum = warp_sum(sum);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mag += __shfl_xor_sync(~0u, mag, o);
        if (lane == 0) s_sum[warp] = sum, s_mag[warp] = mag;
        __syncthreads();
        total = before = 0, mags = 0.f;
        for (int i = 0; i < kWarps; ++i) {
            before += i < warp ? s_sum[i] : 0;
            total += s_sum[i], mags += s_mag[i];
        }
        if (ctas > 1) {
            auto cluster = cg::this_cluster();
            if (threadIdx.x == 0) s_total = total, s_mags = mags;
            cluster.sync();
            total = 0, mags = 0.f;
            for (int r = 0; r < ctas; ++r) {
                const uint64_t v = *cluster.map_shared_rank(&s_total, r);
                before += r < rank ? v : 0;
                total += v, mags += *cluster.map_shared_rank(&s_mags, r);
            }
            cluster.sync();                             // read by all: free to be written again, or left
        } else {
            __syncthreads();
        }
        if (total > 0 || turn == 1 || (!w.q && w.off < 0)) break;
        w.q = nullptr, w.off = -1;                      // nothing left of p - q: p itself
    }
    if (total == 0 || !(mags < 3.99f)) {                // no distribution
        if (rank == 0 && threadIdx.x == 0) out[kept] = -1;
        return;
    }
    // the first index whose running sum exceeds floor(u * total)
    const uint64_t border = __umul64hi(__float2ull_rz(draw * 0x1p64f), total);
    if (before > border || border >= before + s_sum[warp]) return;
    for (int i0 = lo; i0 < hi; i0 += kBlock) {
        load(i0, pv, qv);
        uint64_t m[kEach], all = 0;
#pragma unroll
        for (int k = 0; k < kEach; ++k) m[k] = w.less(pv[k], qv[k], i0 + 32 * k + lane), all += m[k];
        all = warp_sum(all);
        if (before + all <= border) {
            before += all;
            continue;
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            uint64_t c = m[k];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t t = __shfl_up_sync(~0u, c, o);
                if (lane >= o) c += t;
            }
            const unsigned over = __ballot_sync(~0u, before + c > border);
            if (over) {
                if (lane == 0) out[kept] = i0 + 32 * k + __ffs(over) - 1;
                return;
            }
            before += __shfl_sync(~0u, c, 31);
        }
    }
}

template <typename... P, typename... A>
int launch(void (*kern)(P...), int threads, int64_t rows, int ctas, cudaStream_t stream, const char** why, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)(rows * ctas));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    if (ctas > 1) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)ctas;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args..., ctas);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e == cudaSuccess) return 0;
    *why = cudaGetErrorString(e);
    return -1;
}

// A row's CTAs: the fewest powers of two that hold it with kMost vectors a thread (up to eight CTAs), more while each
// still has a vector for every thread and all rows' CTAs are on the GPU at once.
template <typename T, int kThreads>
int probs(const ProbsArgs& a, cudaStream_t stream, const char** why) {
    constexpr int kVec = 8 * kThreads;                  // logits of a vector for each thread
    constexpr int kMost = sizeof(T) == 2 ? 8 : 4;       // vectors with which 1024 threads fit an SM
    int ctas = 1;
    while (ctas < 8 && (a.vocab > (int64_t)kMost * kVec * ctas || (a.n_rows * 2 * ctas <= 1024 / kThreads * kSms && a.vocab >= 2 * ctas * kVec)))
        ctas *= 2;
    const int64_t each = (a.vocab / 8 + ctas - 1) / ctas * 8;
    if (each <= kVec) return launch(k_spec_probs<T, 1, kThreads>, kThreads, a.n_rows, ctas, stream, why, a);
    if (each <= 2 * kVec) return launch(k_spec_probs<T, 2, kThreads>, kThreads, a.n_rows, ctas, stream, why, a);
    if (each <= 4 * kVec) return launch(k_spec_probs<T, 4, kThreads>, kThreads, a.n_rows, ctas, stream, why, a);
    if (each <= 8 * kVec) return launch(k_spec_probs<T, 8, kThreads>, kThreads, a.n_rows, ctas, stream, why, a);
    return launch(k_spec_probs_long<T>, 512, a.n_rows, ctas, stream, why, a);
}

// 256 threads where a cluster of eight such CTAs holds the row: four to an SM, in different phases.
template <typename T>
int probs_of(const ProbsArgs& a, cudaStream_t stream, const char** why) {
    return a.vocab <= 8 * 8 * 256 * (sizeof(T) == 2 ? 8 : 4) ? probs<T, 256>(a, stream, why) : probs<T, 512>(a, stream, why);
}

}  // namespace

int launch_spec_probs(const ProbsArgs& a, bool in_bf16, cudaStream_t stream, const char** why) {
    return in_bf16 ? probs_of<__nv_bfloat16>(a, stream, why) : probs_of<float>(a, stream, why);
}

int launch_spec_verify(const VerifyArgs& a, cudaStream_t stream, const char** why) {
    // up to eight CTAs a request, each with 2048 elements at least, as many as are on the GPU at once, four to an SM
    // (64 requests of 131072: eight CTAs of 256 threads 25 us, four 31; seven of 512 threads 30, four 26)
    int ctas = 1;
    while (ctas < 8 && (int64_t)a.batch * 2 * ctas <= 4 * kSms && a.vocab >= 2 * ctas * 2048) ctas *= 2;
    return launch(k_spec_verify, kVerifyThreads, a.batch, ctas, stream, why, a);
}

}  // namespace ssm
