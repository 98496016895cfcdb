// attn_decode.cu -- one query token per request over the paged, possibly int8, cache (sm_103a).
//
//   s_j = c q . k_j (c = scale log2 e),  l = sum_j 2^(s_j - m),  o = sum_j 2^(s_j - m) v_j,  out = o / l
//
// Every cached byte is read once and used for the few query heads that share its kv head, so the
// cache's bytes bound the step (and launch latency, when there are few of them).  What the design
// has to do is keep enough of them in flight and the arithmetic out of their way:
//   * a warp takes 16 keys at a time (a page holds a whole number of such units) straight from
//     global memory into registers, 16 bytes a load, each byte by one lane; the values' loads are in
//     flight under the scores, the next keys' under the softmax and the second product;
//   * keys and values are the 16-row A operand of m16n8k16 tensor-core products and the (up to 8)
//     query heads of the kv head their 8 columns: S^T = K q^T, O^T = V^T P^T.  The reduction index of
//     each product may be permuted freely, so a lane's 16 loaded bytes are its operand elements as
//     they lie; only P^T crosses lanes, as transposed 8 x 8 matrices;
//   * int8 codes become fp16 exactly (bytes 0x64 and code + 128 are the half 1152 + code); the row
//     scales multiply the scores after the first product and enter the softmax weights before the
//     second;
//   * the long axis is cut into pieces, one CTA each; a second kernel joins the pieces' (m, l, o).
//
// Precision: scores, m, l and o are fp32.  With int8 rows the query is held in fp16 after scaling
// by a power of two (exact for bf16 queries within 2^-25 of their head's maximum) and the weights
// w_j = 2^(s_j + log2 scale_j - mw) in fp16 (11 bits; mw, the running reference of the exponent with
// the scale in it, keeps them in range whatever the rows' scales are).  With bf16 rows the weights
// are a bf16 pair hi + lo.  Both references are raised only when the running maximum has grown by
// more than 2^8, so rescaling o is rare.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace ssm {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kUnit = 16;               // keys a warp takes at a time
constexpr float kSlack = 8.0f;          // log2 of how far a weight may pass its reference
constexpr float kLift = 6.0f;           // fp16 weights carry a factor 2^6: at most 2^14
constexpr unsigned kBadIndex = 8u;      // SSM_DEV_BAD_INDEX

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_b16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 8 x 8 matrix of 16-bit elements, transposed across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Two int8 codes (bytes i and j of w ^ 0x80808080, chosen by sel against 0x64 bytes) as exact halves.
template <uint32_t sel>
__device__ __forceinline__ uint32_t halves(uint32_t flipped) {
    const uint32_t u = __byte_perm(flipped, 0x64646464u, sel);
    const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&u), __half2half2(__ushort_as_half(0x6480)));   // 1152
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t pack_h(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_b(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint4 ld16(const void* p, bool on) {
    return on ? __ldcs(reinterpret_cast<const uint4*>(p)) : make_uint4(0u, 0u, 0u, 0u);
}

// Pieces of the long axis.
struct Cut {
    int tokens, pieces;
};

// A request's length, kept inside the bound and the table.
__device__ __forceinline__ int length_of(const AttnDecodeArgs& a, int b, bool report) {
    const int64_t most = min((int64_t)a.max_len, (int64_t)a.n_table * a.c.page_size);
    int len = a.lens[b];
    if (len < 0 || len > most) {
        if (report) atomicOr(a.status, kBadIndex);
        len = len < 0 ? 0 : (int)most;
    }
    return len;
}

// DP: head_dim padded to 64 or 128.  NT: groups of 8 query heads a CTA serves.
template <bool I8, int DP, int NT, typename Tout>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2)
k_attn_decode(const AttnDecodeArgs a, const Cut cut) {
    constexpr int kHeads = 8 * NT;
    constexpr int kSteps = DP / 16;                     // products over the head's dimensions
    constexpr int kRowLoads = I8 ? DP / 64 : DP / 32;   // 16-byte loads a lane makes of a key row
    constexpr int kVLoads = I8 ? 1 : DP / 64;           // ... of a value row (8 bytes for int8, DP 64)
    __shared__ float s_m[kWarps][kHeads], s_l[kWarps][kHeads], s_w[kWarps][kHeads];
    __shared__ float s_o[kWarps][kHeads][DP];

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = blockIdx.z, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int group = a.n_q / a.c.n_kv, per_kv = (group + kHeads - 1) / kHeads;
    const int hk = (int)blockIdx.y / per_kv, h0 = hk * group + ((int)blockIdx.y % per_kv) * kHeads;
    const int nh = min(kHeads, (hk + 1) * group - h0);  // heads of this CTA
    const int len = length_of(a, b, blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0);
    const int begin = (int)blockIdx.x * cut.tokens, end = min(len, begin + cut.tokens);
    if (begin >= end && !(blockIdx.x == 0 && cut.pieces == 1)) return;
    const int dim = a.c.dim, psz = a.c.page_size;
    const float c = a.scale * kLog2e;

    // ---- the query heads as B operands: column n = lane / 4 is head h0 + 8 i + n
    uint32_t qb[NT][kSteps][2];
    float ch[NT][2];                                    // c (and the query's scaling undone) of heads 2t, 2t + 1
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const bool on = 8 * i + g < nh;
        const __nv_bfloat16* qp = reinterpret_cast<const __nv_bfloat16*>(a.q) + (int64_t)b * a.q_st +
                                  (int64_t)(h0 + 8 * i + (on ? g : 0)) * a.q_sh;
        float qmax = 0.f;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            // the four dimensions this lane's operand elements stand for in step s
            const int d = I8 ? 16 * (t + 4 * (s >> 2)) + 4 * (s & 3) : 8 * (t + 4 * (s >> 1)) + 4 * (s & 1);
            const uint2 w = on && d < dim ? *reinterpret_cast<const uint2*>(qp + d) : make_uint2(0u, 0u);
            qb[i][s][0] = w.x;
            qb[i][s][1] = w.y;
            qmax = fmaxf(qmax, fmaxf(fabsf(__uint_as_float(w.x << 16)), fabsf(__uint_as_float(w.x & 0xffff0000u))));
            qmax = fmaxf(qmax, fmaxf(fabsf(__uint_as_float(w.y << 16)), fabsf(__uint_as_float(w.y & 0xffff0000u))));
        }
        ch[i][0] = ch[i][1] = c;
        if constexpr (I8) {
            qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, 1));
            qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, 2));
            // 2^e with qmax 2^e in [2^10, 2^11); the exponent kept where 2^e and 2^-e are normal
            const int e = qmax > 0.f ? max(-100, min(100, 137 - (int)(__float_as_uint(qmax) >> 23))) : 0;
            const float up = __uint_as_float((uint32_t)(127 + e) << 23), down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t w = qb[i][s][k];
                    qb[i][s][k] = pack_h(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
                }
            ch[i][0] *= __shfl_sync(0xffffffffu, down, 8 * t);          // lane 4 (2t) holds head 2t's
            ch[i][1] *= __shfl_sync(0xffffffffu, down, 8 * t + 4);
        }
    }

    float o[NT][DP / 16][4];
    float m[NT][2], mw[NT][2], l[NT][2];                // of heads 2t, 2t + 1
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][k][e] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) m[i][e] = mw[i][e] = -INFINITY, l[i][e] = 0.f;
    }

    // the cache row of a unit's first key, or -1
    const int32_t* table = a.page_table + (int64_t)b * a.table_stride;
    auto row_of = [&](int j) -> int64_t {
        if (j >= end) return -1;
        const int page = table[j / psz];
        if (page < 0 || page >= a.c.n_pages) {
            if (lane == 0) atomicOr(a.status, kBadIndex);
            return -1;
        }
        return ((int64_t)page * a.c.n_kv + hk) * psz + j % psz;
    };
    constexpr int kE = I8 ? 1 : 2;
    const char* kbase = reinterpret_cast<const char*>(a.c.k);
    const char* vbase = reinterpret_cast<const char*>(a.c.v);
    uint4 kr[2][kRowLoads];                             // rows g and g + 8
    float ks[2] = {0.f, 0.f};
    auto load_keys = [&](int64_t row) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const char* p = kbase + (row + g + 8 * r) * dim * kE;
#pragma unroll
            for (int i = 0; i < kRowLoads; ++i) {
                const int at = 16 * (t + 4 * i);
                kr[r][i] = ld16(p + at, row >= 0 && at < dim * kE);
            }
            if constexpr (I8) ks[r] = row >= 0 ? __ldg(a.c.k_scale + row + g + 8 * r) : 0.f;
        }
    };

    int j = begin + kUnit * warp;
    int64_t row = row_of(j);
    load_keys(row);
    for (; j < end; j += kUnit * kWarps) {
        // ---- values of this unit, in flight: keys 2t, 2t + 1, 2t + 8, 2t + 9
        uint4 vr[4][kVLoads];
        float vs[2] = {0.f, 0.f};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int key = 2 * t + (r & 1) + 8 * (r >> 1);
            const bool on = row >= 0 && j + key < end;
            const char* p = vbase + (row + key) * dim * kE;
            if constexpr (I8 && DP == 64) {
                const uint2 w = on && 8 * g < dim ? __ldcs(reinterpret_cast<const uint2*>(p + 8 * g)) : make_uint2(0u, 0u);
                vr[r][0] = make_uint4(w.x, w.y, 0u, 0u);
            } else {
#pragma unroll
                for (int i = 0; i < kVLoads; ++i) vr[r][i] = ld16(p + 16 * (g + 8 * i), on && 16 * (g + 8 * i) < dim * kE);
            }
        }
        if constexpr (I8) {
#pragma unroll
            for (int r = 0; r < 2; ++r) vs[r] = row >= 0 && j + g + 8 * r < end ? __ldg(a.c.v_scale + row + g + 8 * r) : 0.f;
        }
        const int64_t next = row_of(j + kUnit * kWarps);

        // ---- scores: S^T = K q^T
        float s[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
#pragma unroll
        for (int st = 0; st < kSteps; ++st) {
            uint32_t af[4];
            if constexpr (I8) {
                const uint4 w0 = kr[0][st >> 2], w1 = kr[1][st >> 2];
                const uint32_t x0 = ((st & 3) == 0 ? w0.x : (st & 3) == 1 ? w0.y : (st & 3) == 2 ? w0.z : w0.w) ^ 0x80808080u;
                const uint32_t x1 = ((st & 3) == 0 ? w1.x : (st & 3) == 1 ? w1.y : (st & 3) == 2 ? w1.z : w1.w) ^ 0x80808080u;
                af[0] = halves<0x4140>(x0);
                af[1] = halves<0x4140>(x1);
                af[2] = halves<0x4342>(x0);
                af[3] = halves<0x4342>(x1);
#pragma unroll
                for (int i = 0; i < NT; ++i) mma_f16(s[i], af, qb[i][st][0], qb[i][st][1]);
            } else {
                const uint4 w0 = kr[0][st >> 1], w1 = kr[1][st >> 1];
                af[0] = st & 1 ? w0.z : w0.x;
                af[1] = st & 1 ? w1.z : w1.x;
                af[2] = st & 1 ? w0.w : w0.y;
                af[3] = st & 1 ? w1.w : w1.y;
#pragma unroll
                for (int i = 0; i < NT; ++i) mma_b16(s[i], af, qb[i][st][0], qb[i][st][1]);
            }
        }
        // ---- softmax weights; s[i][2 r + e]: key g + 8 r, head 2t + e
        bool see[2];
        float lv[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            see[r] = row >= 0 && j + g + 8 * r < end;
            lv[r] = I8 ? lg2(vs[r]) : 0.f;              // log2 of 0 is -inf: a row of zeros weighs nothing
        }
        bool grow = false;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float& x = s[i][2 * r + e];
                    x = see[r] ? x * (I8 ? ch[i][e] * ks[r] : ch[i][e]) : -INFINITY;
                    grow = grow || x > m[i][e] + kSlack || (I8 && x + lv[r] > mw[i][e] + kSlack);
                }
        load_keys(next);
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = fmaxf(s[i][e], s[i][2 + e]);
                    float y = I8 ? fmaxf(s[i][e] + lv[0], s[i][2 + e] + lv[1]) : x;
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) {
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                        if constexpr (I8) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
                    }
                    if constexpr (!I8) y = x;
                    const float mn = fmaxf(m[i][e], x), wn = fmaxf(mw[i][e], y);
                    // nothing yet: 2^(-inf - m) = 0 scales a zero
                    if (mn > -INFINITY) l[i][e] *= ex2(m[i][e] - mn);
                    const float f = wn > -INFINITY ? ex2(mw[i][e] - wn) : 1.f;
                    m[i][e] = mn;
                    mw[i][e] = wn;
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k) {
                        o[i][k][e] *= f;
                        o[i][k][2 + e] *= f;
                    }
                }
        }
        uint32_t pb[NT][2], pl[NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float p[2], w[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {           // a reference of -inf: nothing but -inf so far, weights 0
                    p[e] = see[r] ? ex2(s[i][2 * r + e] - (m[i][e] == -INFINITY ? 0.f : m[i][e])) : 0.f;
                    l[i][e] += p[e];
                    w[e] = p[e];
                    if constexpr (I8)
                        w[e] = see[r] ? ex2(s[i][2 * r + e] + lv[r] - ((mw[i][e] == -INFINITY ? 0.f : mw[i][e]) - kLift)) : 0.f;
                }
                if constexpr (I8) {
                    pb[i][r] = transpose8(pack_h(w[0], w[1]));
                    pl[i][r] = 0u;
                } else {
                    const uint32_t hi = pack_b(w[0], w[1]);
                    pb[i][r] = transpose8(hi);
                    pl[i][r] = transpose8(pack_b(w[0] - __uint_as_float(hi << 16), w[1] - __uint_as_float(hi & 0xffff0000u)));
                }
            }
        // ---- O^T += V^T P^T: product k's rows g and g + 8 are the dimensions d and d + 1 of the lane's bytes
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
            uint32_t af[4];
            if constexpr (I8) {
                uint32_t x[4];                          // the word of four dimensions in each of the four rows
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    x[r] = ((k >> 1) == 0 ? vr[r][0].x : (k >> 1) == 1 ? vr[r][0].y : (k >> 1) == 2 ? vr[r][0].z : vr[r][0].w) ^
                           0x80808080u;
                const uint32_t y0 = __byte_perm(x[0], x[1], k & 1 ? 0x7362 : 0x5140);   // d of both keys, d + 1 of both
                const uint32_t y1 = __byte_perm(x[2], x[3], k & 1 ? 0x7362 : 0x5140);
                af[0] = halves<0x4140>(y0);
                af[1] = halves<0x4342>(y0);
                af[2] = halves<0x4140>(y1);
                af[3] = halves<0x4342>(y1);
#pragma unroll
                for (int i = 0; i < NT; ++i) mma_f16(o[i][k], af, pb[i][0], pb[i][1]);
            } else {
                uint32_t x[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint4 v = vr[r][k >> 2];
                    x[r] = (k & 3) == 0 ? v.x : (k & 3) == 1 ? v.y : (k & 3) == 2 ? v.z : v.w;
                }
                af[0] = __byte_perm(x[0], x[1], 0x5410);
                af[1] = __byte_perm(x[0], x[1], 0x7632);
                af[2] = __byte_perm(x[2], x[3], 0x5410);
                af[3] = __byte_perm(x[2], x[3], 0x7632);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    mma_b16(o[i][k], af, pb[i][0], pb[i][1]);
                    mma_b16(o[i][k], af, pl[i][0], pl[i][1]);
                }
            }
        }
        row = next;
    }

    // ---- the warps' parts joined
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], d);
            const int hd = 8 * i + 2 * t + e;
            if (g == 0) {
                s_m[warp][hd] = m[i][e];
                s_l[warp][hd] = l[i][e];
                s_w[warp][hd] = I8 ? mw[i][e] - kLift : m[i][e];
            }
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) {
                const int d = I8 ? (DP == 64 ? 8 * g + 2 * k : 16 * g + 2 * k) : 8 * (g + 8 * (k >> 2)) + 2 * (k & 3);
                *reinterpret_cast<float2*>(&s_o[warp][hd][d]) = make_float2(o[i][k][e], o[i][k][2 + e]);
            }
        }
    __syncthreads();
    for (int x = threadIdx.x; x < nh * DP; x += kThreads) {
        const int hd = x / DP, d = x % DP;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][hd]);
        float L = 0.f, acc = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (s_m[w][hd] == -INFINITY) continue;      // no key of this warp was seen
            L += s_l[w][hd] * ex2(s_m[w][hd] - M);
            if (s_w[w][hd] > -INFINITY || s_w[w][hd] != s_w[w][hd]) acc += s_o[w][hd][d] * ex2(s_w[w][hd] - M);
        }
        const int64_t at = (int64_t)b * a.n_q + h0 + hd;
        if (cut.pieces == 1) {
            if (d < dim)
                reinterpret_cast<Tout*>(a.out)[(int64_t)b * a.o_st + (int64_t)(h0 + hd) * a.o_sh + d] =
                    from_f32<Tout>(M == -INFINITY ? 0.f : acc / L);
            if (a.lse && d == 0) a.lse[at] = M == -INFINITY ? -INFINITY : kLn2 * (M + log2f(L));
        } else {
            float* ws = reinterpret_cast<float*>(a.workspace);
            const int64_t piece = at * cut.pieces + blockIdx.x;
            ws[piece * DP + d] = acc;
            if (d == 0) {
                float2* ml = reinterpret_cast<float2*>(ws + (int64_t)gridDim.z * a.n_q * cut.pieces * DP);
                ml[piece] = make_float2(M, L);
            }
        }
    }
}

// Joins the pieces of one (request, head): out = sum_p o_p 2^(m_p - m) / sum_p l_p 2^(m_p - m).
template <int DP, typename Tout>
__global__ void __launch_bounds__(DP)
k_attn_decode_join(const AttnDecodeArgs a, const Cut cut) {
    const int h = blockIdx.x, b = blockIdx.y, d = threadIdx.x;
    const int len = length_of(a, b, false);
    const int n = (len + cut.tokens - 1) / cut.tokens;
    const int64_t at = (int64_t)b * a.n_q + h;
    const float* ws = reinterpret_cast<const float*>(a.workspace) + at * cut.pieces * DP + d;
    const float2* ml = reinterpret_cast<const float2*>(reinterpret_cast<const float*>(a.workspace) +
                                                       (int64_t)a.batch * a.n_q * cut.pieces * DP) + at * cut.pieces;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float M = -INFINITY, L = 0.f, acc = 0.f;
    for (int p = 0; p < n; ++p) M = fmaxf(M, ml[p].x);
#pragma unroll 8
    for (int p = 0; p < n; ++p) {
        const float2 x = ml[p];
        const float f = x.x == -INFINITY ? 0.f : ex2(x.x - M);
        L += x.y * f;
        acc += f == 0.f ? 0.f : ws[(int64_t)p * DP] * f;
    }
    if (d < a.c.dim)
        reinterpret_cast<Tout*>(a.out)[(int64_t)b * a.o_st + (int64_t)h * a.o_sh + d] =
            from_f32<Tout>(M == -INFINITY ? 0.f : acc / L);
    if (a.lse && d == 0) a.lse[at] = M == -INFINITY ? -INFINITY : kLn2 * (M + log2f(L));
}

// CTAs side by side for one request's long axis: one per kv head and group of 16 (or 8) query heads.
int lanes_of(int n_q, int n_kv) {
    const int group = n_q / n_kv, heads = group > 8 ? 16 : 8;
    return n_kv * ((group + heads - 1) / heads);
}

Cut cut_of(int batch, int n_q, int n_kv, int64_t max_len) {
    // Many CTAs of at least 512 keys, so that requests of different lengths fill the GPU evenly and the
    // join reads little; where that leaves fewer than two per resident slot (152 SMs x 3), pieces
    // down to 128 keys.
    const int64_t side = (int64_t)batch * lanes_of(n_q, n_kv);
    int64_t p = (3648 + side - 1) / side;
    const int64_t most = (max_len + 511) / 512;
    if (p > most) p = most;
    if (side * p < 912) {
        p = (912 + side - 1) / side;
        const int64_t fine = (max_len + 127) / 128;
        if (p > fine) p = fine;
    }
    Cut c;
    c.tokens = (int)(((max_len + p - 1) / p + 63) / 64 * 64);
    c.pieces = (int)((max_len + c.tokens - 1) / c.tokens);
    return c;
}

template <bool I8, int DP, int NT, typename Tout>
int launch(const AttnDecodeArgs& a, cudaStream_t stream, const char** why) {
    const Cut cut = cut_of(a.batch, a.n_q, a.c.n_kv, a.max_len);
    const dim3 grid((unsigned)cut.pieces, (unsigned)lanes_of(a.n_q, a.c.n_kv), (unsigned)a.batch);
    k_attn_decode<I8, DP, NT, Tout><<<grid, kThreads, 0, stream>>>(a, cut);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && cut.pieces > 1) {
        // launched while the pieces still run; it waits for them before it reads
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)a.n_q, (unsigned)a.batch);
        cfg.blockDim = dim3(DP);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, k_attn_decode_join<DP, Tout>, a, cut);
        if (e == cudaSuccess) e = cudaGetLastError();
    }
    if (e == cudaSuccess) return 0;
    *why = cudaGetErrorString(e);
    return -1;
}

template <bool I8, typename Tout>
int launch_shape(const AttnDecodeArgs& a, cudaStream_t stream, const char** why) {
    const bool wide = a.n_q / a.c.n_kv > 8;
    if (a.c.dim <= 64) return wide ? launch<I8, 64, 2, Tout>(a, stream, why) : launch<I8, 64, 1, Tout>(a, stream, why);
    return wide ? launch<I8, 128, 2, Tout>(a, stream, why) : launch<I8, 128, 1, Tout>(a, stream, why);
}

}  // namespace

size_t attn_decode_workspace(int batch, int n_q, int n_kv, int dim, int max_len) {
    const Cut c = cut_of(batch, n_q, n_kv, max_len);
    return c.pieces == 1 ? 0 : (size_t)batch * n_q * c.pieces * ((dim <= 64 ? 64 : 128) + 2) * sizeof(float);
}

int launch_attn_decode(const AttnDecodeArgs& a, bool cache_i8, bool out_bf16, cudaStream_t stream, const char** why) {
    if (cache_i8)
        return out_bf16 ? launch_shape<true, __nv_bfloat16>(a, stream, why) : launch_shape<true, float>(a, stream, why);
    return out_bf16 ? launch_shape<false, __nv_bfloat16>(a, stream, why) : launch_shape<false, float>(a, stream, why);
}

}  // namespace ssm
