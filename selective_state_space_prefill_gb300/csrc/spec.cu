// spec.cu -- spec_probs (probabilities of logits at a temperature) and spec_verify (drafted tokens against the
// target's probabilities).
//
// Both read rows of the vocabulary's length, a few or hundreds of them: a row is a thread-block cluster's, cut into
// a slice per CTA, and what the CTAs have to know of each other (a maximum, sums) goes through distributed shared
// memory.
#include <type_traits>

#include "common.cuh"
#include "exchange.cuh"
#include "kernels.h"
#include "ssm.h"

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

// e^((x - m) / t) of half the maximum m and twice the rate log2(e) / t: halves of logits differ by no more than the largest
// float, where logits may by twice that; all else is the same to the bit.
__device__ __forceinline__ float twice_rate(float t) { return __fdiv_rn(1.f, fminf(t, 0x1.fffffep127f)) * kLog2e * 2.f; }
__device__ __forceinline__ float power(float x, float half, float f) { return ex2(fmaf(x, 0.5f, -half) * f); }

// One float, whatever stands beside it: plain stores of four neighbours, next to one of them as a float4 in the other
// branch, came out as one 16-byte store, which faults where the row is not aligned.
__device__ __forceinline__ void store1(float* p, float v) { asm volatile("st.global.f32 [%0], %1;" ::"l"(p), "f"(v) : "memory"); }

// A value of all threads of a row (of no use to a warp that gave up).
enum Kind { kMax, kSum, kLeast };
template <Kind K, typename T>
__device__ __forceinline__ T two(T a, T b) {
    if constexpr (K == kMax) return max_nan(a, b);
    else if constexpr (K == kSum) return a + b;
    else return a < b ? a : b;
}
template <typename T> __device__ __forceinline__ uint32_t bits_of(T v) {
    if constexpr (std::is_same_v<T, float>) return __float_as_uint(v);
    else return (uint32_t)v;
}
template <typename T> __device__ __forceinline__ T from_bits(uint32_t v) {
    if constexpr (std::is_same_v<T, float>) return __uint_as_float(v);
    else return (T)v;
}
template <Kind K, int kWarps, typename T>
__device__ __forceinline__ T row_wide(Exchange<1, 1>& all, T* s_warp, T v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = two<K>(v, __shfl_xor_sync(~0u, v, o));
    if (threadIdx.x % 32 == 0) s_warp[threadIdx.x / 32] = v;
    __syncthreads();
    v = s_warp[threadIdx.x % kWarps];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) v = two<K>(v, __shfl_xor_sync(~0u, v, o));
    if (all.ctas == 1) return v;
    all.send({bits_of(v)});
    v = from_bits<T>(all.word(0, threadIdx.x % all.ctas));
    all.settle();
    for (int o = all.ctas / 2; o > 0; o >>= 1) v = two<K>(v, __shfl_xor_sync(~0u, v, o));
    return v;
}

// Of a warp that has no part in a row's second value, be it that the row is NaN or that the warp gave up: what the
// others of its CTA look for at their barrier there.
__device__ __forceinline__ void none_of_row(float* s_sum, int* s_at) {
    if (threadIdx.x % 32 == 0) s_sum[threadIdx.x / 32] = quiet_nan(), s_at[threadIdx.x / 32] = 0x7fffffff;
    __syncthreads();
}

// Eight logits as they came.
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> {
    uint4 q;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { q = *reinterpret_cast<const uint4*>(p); }
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
        q[0] = reinterpret_cast<const float4*>(p)[0], q[1] = reinterpret_cast<const float4*>(p)[1];
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
// last whole vector (up to 14 logits) is one logit each for the first CTA's first threads.  512 x 131072 bf16 (403 MB)
// 82 us, 4.9 TB/s, 0.72 of the copy rate: a CTA loads, waits for the row's maximum, takes powers, waits for the sum,
// writes, and four of them an SM do not keep memory busy all the time (2000 x 32000, shorter rows, 5.2 TB/s).  The
// next rows asked for from L2 ahead of time make 2 to 4 % and are left out.  5 x 50021 3.3 us in a graph.
template <typename T, int V, int kThreads>
__global__ void __launch_bounds__(kThreads, V * sizeof(T) <= 16 ? 1024 / kThreads : 1) k_spec_probs(const ProbsArgs a, int ctas) {
    constexpr int kWarps = kThreads / 32;
    __shared__ Exchange<1, 1>::Box box;
    __shared__ float s_max[kWarps], s_sum[kWarps];
    __shared__ int s_at[kWarps];
    const int64_t row = blockIdx.x / (unsigned)ctas;
    const int rank = blockIdx.x % (unsigned)ctas, vocab = (int)a.vocab;
    Exchange<1, 1> all(box, ctas, rank, a.status);
    const T* x = reinterpret_cast<const T*>(a.logits) + row * a.ld_in;
    float* p = a.probs + row * a.ld_out;
    after_previous();
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
    all.ready();
    m = row_wide<kMax, kWarps>(all, s_max, m);

    // p = 2^((x - m) f) inv, or 1 at one place, or the same everywhere
    float f = 0.f, half = 0.f, inv = quiet_nan();
    int least = -1;
    if (!(m < INFINITY) || t != t || all.dead) {        // NaN or +inf among the logits: NaN
        none_of_row(s_sum, s_at);
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
        least = row_wide<kLeast, kWarps>(all, s_at, least);
    } else {
        f = twice_rate(t), half = 0.5f * m;
        float l = power(w, half, f);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) l += power(v[i].at(k), half, f);
        inv = __fdiv_rn(1.f, row_wide<kSum, kWarps>(all, s_sum, l));
    }
    if (all.dead) f = 0.f, inv = quiet_nan(), least = -1;
    next_may_start();                                   // 64 x 32000 7.5 us, at the kernel's start 7.8
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
    if (f > 0.f) write([&](float x, int) { return power(x, half, f) * inv; });
    else write([&](float, int at) { return at == least ? 1.f : inv; });
    all.leave();
}

// Rows longer than a cluster's registers hold: read three times, from L2 after the first, a logit a load, by eight CTAs: 64 x
// 300001 bf16 (115 MB) 45 us, 0.38 of the copy rate, 8 x 300001 12.7; few very long rows leave most of the GPU idle (4 x
// 2^24 2.4 ms, 0.17 TB/s).
template <typename T>
__global__ void __launch_bounds__(512) k_spec_probs_long(const ProbsArgs a, int ctas) {
    constexpr int kThreads = 512, kWarps = kThreads / 32;
    __shared__ Exchange<1, 1>::Box box;
    __shared__ float s_max[kWarps], s_sum[kWarps];
    __shared__ int s_at[kWarps];
    const int64_t row = blockIdx.x / (unsigned)ctas;
    const int rank = blockIdx.x % (unsigned)ctas, vocab = (int)a.vocab;
    Exchange<1, 1> all(box, ctas, rank, a.status);
    const T* x = reinterpret_cast<const T*>(a.logits) + row * a.ld_in;
    float* p = a.probs + row * a.ld_out;
    after_previous();
    const float t = a.temperature ? a.temperature[row] : 1.f;
    const int per = (vocab + ctas - 1) / ctas, lo = rank * per, hi = min(lo + per, vocab);
    float m = -INFINITY;
#pragma unroll 8
    for (int i = lo + threadIdx.x; i < hi; i += kThreads) m = max_nan(m, to_f32(x[i]));
    all.ready();
    m = row_wide<kMax, kWarps>(all, s_max, m);
    if (!(m < INFINITY) || t != t || all.dead) {
        none_of_row(s_sum, s_at);
        for (int i = lo + threadIdx.x; i < hi; i += kThreads) p[i] = quiet_nan();
    } else if (t <= 0x1p-100f || m == -INFINITY) {
        int least = 0x7fffffff;
#pragma unroll 8
        for (int i = lo + threadIdx.x; i < hi; i += kThreads)
            if (to_f32(x[i]) == m && m > -INFINITY) least = min(least, i);
        least = row_wide<kLeast, kWarps>(all, s_at, least);
        const float rest = all.dead ? quiet_nan() : 0.f;
        for (int i = lo + threadIdx.x; i < hi; i += kThreads) p[i] = i == least ? 1.f : rest;
    } else {
        const float f = twice_rate(t), half = 0.5f * m;
        float l = 0.f;
#pragma unroll 8
        for (int i = lo + threadIdx.x; i < hi; i += kThreads) l += power(to_f32(x[i]), half, f);
        l = row_wide<kSum, kWarps>(all, s_sum, l);
        const float inv = all.dead ? quiet_nan() : __fdiv_rn(1.f, l);
#pragma unroll 8
        for (int i = lo + threadIdx.x; i < hi; i += kThreads) p[i] = power(to_f32(x[i]), half, f) * inv;
    }
    all.leave();
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

// What is left of p without q, both >= 0, in those integers.
__device__ __forceinline__ uint64_t less(float p, float q) { return p > q ? fixed(p) - fixed(q) : 0ull; }

// Sums of the same, without shifts of 64 bits (64 requests x 131072 21.5 us, with shifts 23.0).  A value below 4 is cut into three: added to 8 towards 0 its places down to 2^-20 are the sum's last bits,
// the rest, exact, added to 2^-20 gives those down to 2^-43, and what is left of that, added to 2^-39, those down to
// 2^-62.  The constants' bits go out in the differences of p's parts and q's.
struct Parts {
    uint32_t a = 0, b = 0, c = 0;
    __device__ __forceinline__ void add(float p, float q) {
        const float pa = __fadd_rz(p, 8.f), qa = __fadd_rz(q, 8.f);
        const float pr = p - (pa - 8.f), qr = q - (qa - 8.f);
        const float pb = __fadd_rz(pr, 0x1p-20f), qb = __fadd_rz(qr, 0x1p-20f);
        const float pc = __fadd_rz(pr - (pb - 0x1p-20f), 0x1p-39f), qc = __fadd_rz(qr - (qb - 0x1p-20f), 0x1p-39f);
        if (p > q) {
            a += __float_as_uint(pa) - __float_as_uint(qa);
            b += __float_as_uint(pb) - __float_as_uint(qb);
            c += __float_as_uint(pc) - __float_as_uint(qc);
        }
    }
    // of up to 256 values: the parts, below 2^22, 2^23 and 2^19, stay in 32 bits, the lower two with their signs
    __device__ __forceinline__ uint64_t sum() const {
        return ((uint64_t)a << 42) + ((uint64_t)(int64_t)(int32_t)b << 19) + (uint64_t)(int64_t)(int32_t)c;
    }
};

// The row that the next token is drawn from.
struct Mass {
    const float *p, *q;
    int off;
};

template <typename T> __device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// A cluster per request.  Sums are exact integers, so that the order of their parts and the cut do not matter: a
// warp sums a stretch of the row, its lanes note their sums up to eight times on the way, and the warp in whose
// stretch the border falls reads again (from L2) what lies between two notes.  Without notes it read its stretch
// from the start, block by block.  Of the 19 us of 64 requests x 131072 (67 MB, 9.9 us at the copy rate) the checks of the
// drafted tokens take 2 (three reads, each waiting for the one before), the sums 9, the slowest of a cluster's CTAs 2
// to 3, the search 2, starting and ending the rest.  One request: 6.0 us, the same chain of waits.  Without q half of the bytes
// go and little of the time, as q's arithmetic is done with zeros: 64 x 131072 18.8 us, without drafts 15.8, 128 x 151937
// 33 (11.5 of bytes).
constexpr int kVerifyThreads = 256;
__global__ void __launch_bounds__(kVerifyThreads, 4) k_spec_verify(const VerifyArgs a, int ctas) {
    constexpr int kThreads = kVerifyThreads, kWarps = kThreads / 32;
    constexpr int kEach = 8, kBlock = 32 * kEach;       // elements that a warp takes at a time
    constexpr int kNotes = 8;                           // of a lane's sum on the way
    __shared__ int s_kept, s_n;
    __shared__ uint64_t s_note[kWarps][kNotes][32];
    __shared__ Exchange<3, kWarps>::Box box;
    const int b = blockIdx.x / (unsigned)ctas, rank = blockIdx.x % (unsigned)ctas;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, vocab = (int)a.vocab;
    Exchange<3, kWarps> all(box, ctas, rank, a.status);
    const int32_t* draft = a.draft + (int64_t)b * a.n_max;
    const float* u = a.u + (int64_t)b * (a.n_max + 1);
    after_previous();
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
    all.ready();
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
    const int step = ((per + kBlock - 1) / kBlock + kNotes - 1) / kNotes * kBlock;      // elements between two notes
    // a lane's elements of a block, `apart` from each other, all loads under way at once; negative ones and NaN are 0
    auto load = [&](int i0, int apart, float (&pv)[kEach], float (&qv)[kEach]) {
        const bool whole = i0 + kBlock <= hi;
        i0 += apart == 1 ? lane * kEach : lane;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = i0 + apart * k;
            pv[k] = whole || i < hi ? w.p[i] : 0.f;
            qv[k] = w.q && (whole || i < hi) ? w.q[i] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k) pv[k] = fmaxf(pv[k], 0.f), qv[k] = fmaxf(qv[k], 0.f);
        if (w.off >= 0) {
#pragma unroll
            for (int k = 0; k < kEach; ++k)
                if (i0 + apart * k == w.off) qv[k] = 1.f;
        }
    };
    float pv[kEach], qv[kEach];
    uint64_t total, before, mine;                       // the row's, what is before this warp's stretch, the stretch's
    float mags;
    int notes;
    for (int turn = 0;; ++turn) {
        uint64_t sum = 0;
        float mag = 0.f;
        notes = 0;
        for (int i0 = lo; i0 < hi; ++notes) {
            for (const int to = min(i0 + step, hi); i0 < to; i0 += kBlock) {
                load(i0, 32, pv, qv);
                Parts parts;
#pragma unroll
                for (int k = 0; k < kEach; ++k) {
                    parts.add(pv[k], qv[k]);
                    mag += pv[k];
                }
                sum += parts.sum();
            }
            s_note[warp][notes][lane] = sum;
        }
        sum = warp_sum(sum);
        mag = warp_sum(mag);
        all.send({(uint32_t)sum, (uint32_t)(sum >> 32), __float_as_uint(mag)});
        total = before = 0, mags = 0.f, mine = sum;
        for (int i = lane; i < ctas * kWarps; i += 32) {
            const uint64_t part = all.word(0, i) | (uint64_t)all.word(1, i) << 32;
            total += part, mags += __uint_as_float(all.word(2, i));
            before += i < rank * kWarps + warp ? part : 0;
        }
        all.settle();
        total = warp_sum(total), before = warp_sum(before), mags = warp_sum(mags);
        if (total > 0 || turn == 1 || (!w.q && w.off < 0) || all.dead) break;
        w.q = nullptr, w.off = -1;                      // nothing left of p - q: p itself
    }
    next_may_start();
    // the first index whose running sum exceeds floor(u * total)
    const uint64_t border = __umul64hi(__float2ull_rz(draw * 0x1p64f), total);
    if (all.dead) {                                     // whose part may have been to find it
        if (lane == 0) out[kept] = -1;
    } else if (total == 0 || !(mags < 3.99f)) {         // no distribution
        if (rank == 0 && threadIdx.x == 0) out[kept] = -1;
    } else if (before <= border && border < before + mine) {
        // the notes say between which two of them; that is read again (from L2)
        uint64_t at = 0;
        if (lane < notes) {
#pragma unroll 8
            for (int k = 0; k < 32; ++k) at += s_note[warp][lane][(k + lane) % 32];
        }
        const int note = __ffs(__ballot_sync(~0u, lane < notes && before + at > border)) - 1;
        if (note > 0) before += __shfl_sync(~0u, at, note - 1);
        for (int i0 = lo + note * step; i0 < hi; i0 += kBlock) {
            load(i0, 1, pv, qv);
            uint64_t m[kEach], own = 0;
#pragma unroll
            for (int k = 0; k < kEach; ++k) m[k] = less(pv[k], qv[k]), own += m[k];
            uint64_t to = own;                          // of the lanes up to this one
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t t = __shfl_up_sync(~0u, to, o);
                if (lane >= o) to += t;
            }
            const unsigned over = __ballot_sync(~0u, before + to > border);
            if (over) {
                if (lane == __ffs(over) - 1) {
                    before += to - own;
                    int k = 0;
#pragma unroll
                    for (int j = 0; j + 1 < kEach; ++j) {
                        before += m[j];
                        k += before <= border;
                    }
                    out[kept] = i0 + kEach * lane + k;
                }
                break;
            }
            before += __shfl_sync(~0u, to, 31);
        }
    }
    all.leave();
}

// A cluster of `ctas` for each row.
template <typename... P, typename A>
int launch(void (*kern)(P...), int threads, int64_t rows, int ctas, cudaStream_t stream, const char** why, const A& a) {
    return launch_in_turn(kern, dim3((unsigned)(rows * ctas)), threads, 0, ctas, stream, why, a, ctas);
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
    // (64 requests of 131072: eight CTAs of 256 threads 22 us, four of 512 23, eight of 512 28)
    int ctas = 1;
    while (ctas < 8 && (int64_t)a.batch * 2 * ctas <= 4 * kSms && a.vocab >= 2 * ctas * 2048) ctas *= 2;
    return launch(k_spec_verify, kVerifyThreads, a.batch, ctas, stream, why, a);
}

}  // namespace ssm
