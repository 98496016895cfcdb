// attn_decode.cu -- one query token per request over the paged, possibly int8, cache (sm_103a).
//
//   s_j = c q . k_j (c = scale log2 e),  l = sum_j 2^(s_j - m),  o = sum_j 2^(s_j - m) v_j,  out = o / l
//
// Every cached byte is read once and used for the few query heads that share its kv head, so the
// cache's bytes bound the step (and launch latency, when there are few of them).  What the design
// has to do is keep enough of them in flight and the arithmetic out of their way:
//   * a warp takes 16 keys at a time (a page holds a whole number of such units); its lanes copy
//     them to its own ring in shared memory with 16-byte asynchronous copies, several units ahead,
//     and no warp waits for another.  The 16-byte chunks of a 128-byte line are permuted by the row
//     (chunk ^ row % 8), so that the operand reads below meet no bank twice;
//   * keys and values are the 16-row A operand of m16n8k16 tensor-core products and the (up to 8)
//     query heads of the kv head their 8 columns: S^T = K q^T, O^T = V^T P^T (a tcgen05 tile of 128
//     rows would be all but empty, and int8 rows would have to be widened in shared memory first; the
//     tensor pipe is 11 to 14 % busy like this), the operands read as 8 x 8 matrices (the values'
//     transposed).  The order of the reduction index is free, so two int8 dimensions travel as one 16-bit
//     element;
//   * int8 codes become fp16 exactly, two at a time: code + 128 as the significand of 1024 + x for the
//     values (1152 subtracted), as a subnormal, x 2^-24, for the keys, whose 128 is taken off the
//     scores' starting value; the row scales multiply the scores after the first product and the
//     softmax weights before the second;
//   * the long axis is cut into pieces, one CTA each; a second kernel joins the pieces' (m, l, o), or, for
//     short calls, the cluster that the pieces form.
//
// Measured: 4 x 65536 tokens of 8 kv heads of 128, bf16: 168 us, 6.4 TB/s; the same in int8 112 us, 4.9 TB/s;
// 64 ragged requests up to 8192 tokens, int8: 72 us a call, 4.6 TB/s; one of 4096 tokens 9.5 us a call.  With
// int8 rows no unit is full (64 ragged requests: 0.60 instructions a cycle and scheduler, ALU pipe 59 %, DRAM
// 64 %): some 14 warps an SM go through each unit's chain of conversions, products and softmax one after
// the other, waiting for results and for the ALU more than for memory.
//
// Precision: scores, m, l and o are fp32.  With int8 rows the query is held in fp16 after scaling
// by a power of two (exact for bf16 queries within 2^-25 of their head's maximum) and the weights
// w_j = 2^(s_j - mw) scale_j in fp16 (11 bits; mw is a running reference of the exponent with the
// scale in it, so that they fit whatever the rows' scales are; below 2^-20 of the largest they lose
// bits, below 2^-31 they are zero, either way under 2^-31 of the largest each).  With bf16 rows the
// weights are a bf16 pair hi + lo, both positive, so that an infinite value keeps its sign.  The
// references are raised only when a weight would pass them by more than 2^8, so rescaling o is rare.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace ssm {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kUnit = 16;               // keys a warp takes at a time
constexpr float kSlack = 8.0f;          // log2 of how far a weight may pass its reference
constexpr float kLift = 6.0f;           // fp16 weights carry a factor 2^6 ...
constexpr float kMost = 16384.0f;       // ... and are at most 2^14
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

// Of the four codes in x, the bytes 0 and 2 (kHi false) or 1 and 3, exact in fp16: as (code + 128) 2^-24,
// or as the code itself.
template <bool kHi>
__device__ __forceinline__ uint32_t raised(uint32_t x) {
    return ((kHi ? x >> 8 : x) & 0x00ff00ffu) ^ 0x00800080u;
}
template <bool kHi>
__device__ __forceinline__ uint32_t halves(uint32_t x) {
    const uint32_t u = ((kHi ? x >> 8 : x) & 0x00ff00ffu) ^ 0x64806480u;
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

// Asynchronous copies to shared memory; `on` false writes zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(on ? 4 : 0) : "memory");
}
// Four 8 x 8 matrices of 16-bit elements, lane 8 i + r giving the address of matrix i's row r.
__device__ __forceinline__ void matrices(uint32_t (&x)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void matrices_t(uint32_t (&x)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ float lds4(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// A stage of a warp's ring: 16 key rows, 16 value rows, and (int8) their 16 + 16 scales.  A row of
// ROW bytes is ROW / 128 lines of 128 bytes (line i of all 16 rows together), or half a line.
template <bool I8, int DP>
struct Ring {
    static constexpr int kRow = DP * (I8 ? 1 : 2);
    static constexpr int kLine = kRow < 128 ? kRow : 128;
    static constexpr int kRows = kUnit * kRow;          // bytes of 16 rows
    static constexpr int kStage = 2 * kRows + (I8 ? 128 : 0);
    static constexpr int kStages = kStage > 4000 ? 3 : 4;
    // CTAs that share an SM (up to 8 query heads): by its 227 KB of shared memory 4 with int8 rows of 128
    // and with bf16 rows of 64, 2 with bf16 rows of 128, by its registers 4 with int8 rows of 64; 100 to 135
    // KB of copies are then in flight.
    static constexpr int kPer = kLine / 16;             // chunks of a line
    // byte offset of 16-byte chunk c of row r
    static __device__ __forceinline__ uint32_t at(int r, int c) {
        return (uint32_t)((c / kPer) * kUnit * kLine + r * kLine + ((c % kPer) ^ (kPer == 8 ? r & 7 : (r >> 1) & 3)) * 16);
    }
    // ... of chunk c + c0, c0 even, from that of chunk c < 2 (lines are 128-byte aligned)
    static __device__ __forceinline__ uint32_t step(uint32_t a, int c0) {
        return (a ^ (uint32_t)((c0 % kPer) * 16)) + (uint32_t)((c0 / kPer) * kUnit * kLine);
    }
};

// Pieces of the long axis; `cluster`: the pieces are the CTAs of a cluster and join there.
struct Cut {
    int tokens, pieces;
    bool cluster;
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

// The pieces' maxima and sums, after their outputs in the workspace.
template <int DP>
__device__ __forceinline__ float2* piece_sums(const AttnDecodeArgs& a, const Cut& cut, int64_t batch) {
    return reinterpret_cast<float2*>(reinterpret_cast<float*>(a.workspace) + batch * a.n_q * cut.pieces * DP);
}

// A sum of 0 is that of no key: nothing seen, output zeros, lse -inf.
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.f ? -INFINITY : kLn2 * (m + log2f(l)); }
__device__ __forceinline__ void store_out(float* p, float4 v, float l) {
    const float f = l == 0.f ? 0.f : 1.f / l;
    *reinterpret_cast<float4*>(p) = l == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
}
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float4 v, float l) {
    const float f = l == 0.f ? 0.f : 1.f / l;
    *reinterpret_cast<uint2*>(p) = l == 0.f ? make_uint2(0u, 0u) : make_uint2(pack_b(v.x * f, v.y * f), pack_b(v.z * f, v.w * f));
}

// DP: head_dim padded to 64 or 128.  NT: groups of 8 query heads a CTA serves.
template <bool I8, int DP, int NT, bool kCluster, typename Tout>
__global__ void __launch_bounds__(kThreads, NT == 1 ? (I8 ? 4 : DP == 64 ? 3 : 2) : 2)
k_attn_decode(const AttnDecodeArgs a, const Cut cut) {
    constexpr int kHeads = 8 * NT;
    constexpr int kSteps = DP / 16;                     // products over the head's dimensions
    using R = Ring<I8, DP>;
    constexpr int kE = I8 ? 1 : 2;
    extern __shared__ __align__(128) unsigned char smem[];      // the warps' rings, then their parts
    __shared__ float s_m[kWarps][kHeads], s_l[kWarps][kHeads], s_w[kWarps][kHeads];
    float(*s_o)[kHeads][DP + 4] = reinterpret_cast<float(*)[kHeads][DP + 4]>(smem);     // + 4: no bank twice

    if constexpr (!kCluster) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = blockIdx.z, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int group = a.n_q / a.c.n_kv, per_kv = (group + kHeads - 1) / kHeads;
    const int hk = (int)blockIdx.y / per_kv, h0 = hk * group + ((int)blockIdx.y % per_kv) * kHeads;
    const int nh = min(kHeads, (hk + 1) * group - h0);  // heads of this CTA
    const int len = length_of(a, b, blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0);
    const int begin = (int)blockIdx.x * cut.tokens, end = min(len, begin + cut.tokens);
    if (!kCluster && begin >= end && !(blockIdx.x == 0 && cut.pieces == 1)) return;
    const int dim = a.c.dim, psz = a.c.page_size;
    const float c = a.scale * kLog2e;

    // the cache row of each of this warp's units in turn, or -1: past the end, or a page outside the cache
    const int32_t* table = a.page_table + (int64_t)b * a.table_stride;
    constexpr int kStep = kUnit * kWarps;
    int at_j = begin + kUnit * warp, at_page = at_j / psz, at_row = at_j % psz;
    const int skip_page = kStep / psz, skip_row = kStep % psz;
    auto next_row = [&]() -> int64_t {
        if (at_j >= end) return -1;
        const int page = table[at_page], r = at_row;
        at_j += kStep;
        at_page += skip_page;
        at_row += skip_row;
        if (at_row >= psz) at_row -= psz, ++at_page;
        if (page < 0 || page >= a.c.n_pages) {
            if (lane == 0) atomicOr(a.status, kBadIndex);
            return -1;
        }
        return ((int64_t)page * a.c.n_kv + hk) * psz + r;
    };
    // the copies of the unit whose first row is `row` into ring stage `st` (none for row < 0; the
    // group is committed all the same, so that groups and units keep step)
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * R::kStages * R::kStage);
    constexpr int kChunks = R::kRow / 16, kPerPass = 32 / kChunks;       // chunks of a row, rows a pass of the warp copies
    const int ch16 = lane % kChunks, r0 = lane / kChunks;
    const bool in = 16 * ch16 < dim * kE;               // chunks past the head's dimensions are zeros
    const int64_t row_bytes = (int64_t)dim * kE, lane_off = in ? r0 * row_bytes + 16 * ch16 : 0, pass_bytes = kPerPass * row_bytes;
    auto fetch = [&](int64_t row, int j, int st) {
        if (row >= 0) {
            const uint32_t dst = ring + (uint32_t)(st * R::kStage);
            const char* kp = reinterpret_cast<const char*>(a.c.k) + row * row_bytes + lane_off;
            const char* vp = reinterpret_cast<const char*>(a.c.v) + row * row_bytes + lane_off;
            if (j + kUnit <= end && dim == DP) {        // whole rows, their places known to the compiler
#pragma unroll
                for (int r = 0; r < kUnit; r += kPerPass) {
                    copy16(dst + R::at(r0 + r, ch16), kp + r * R::kRow);
                    copy16(dst + R::kRows + R::at(r0 + r, ch16), vp + r * R::kRow);
                }
            } else {
#pragma unroll 1
                for (int r = 0; r < kUnit; r += kPerPass) {
                    // rows past the end are zeros: a value's weight is 0, but 0 x NaN is not
                    const bool on = in && j + r0 + r < end;
                    copy16(dst + R::at(r0 + r, ch16), on ? kp : reinterpret_cast<const char*>(a.c.k), on);
                    copy16(dst + R::kRows + R::at(r0 + r, ch16), on ? vp : reinterpret_cast<const char*>(a.c.v), on);
                    kp += pass_bytes, vp += pass_bytes;
                }
            }
            if constexpr (I8) {
                const int key = lane & 15;
                copy4(dst + 2 * R::kRows + 4 * lane, (lane < 16 ? a.c.k_scale : a.c.v_scale) + row + key, j + key < end);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    int j = at_j, stage = 0;
    int64_t rows[R::kStages];                           // of the units in the ring, the current one first
#pragma unroll
    for (int st = 0; st < R::kStages; ++st) {
        rows[st] = next_row();
        if (st + 1 < R::kStages) fetch(rows[st], j + st * kStep, st);
    }
    // this lane's rows of the operands' matrices: keys, matrix i = (key half i % 2, chunk i / 2); values
    // the same for int8, (chunk i % 2, key half i / 2) for bf16
    const uint32_t key_at = R::at((lane & 7) + (lane & 8), lane >> 4);
    const uint32_t val_at = I8 ? key_at : R::at((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1);

    // ---- the query heads as B operands: column n = lane / 4 is head h0 + 8 i + n
    uint32_t qb[NT][kSteps][2];
    float ch[NT][2];                                    // c (and the operands' scaling undone) of heads 2t, 2t + 1
    float s0[NT][2];                                    // where their scores start: the keys' 128 taken off
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const bool on = 8 * i + g < nh;
        const __nv_bfloat16* qp = reinterpret_cast<const __nv_bfloat16*>(a.q) + (int64_t)b * a.q_st +
                                  (int64_t)(h0 + 8 * i + (on ? g : 0)) * a.q_sh;
        ch[i][0] = ch[i][1] = c;
        s0[i][0] = s0[i][1] = 0.f;
        if constexpr (I8) {
            float qmax = 0.f;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int d = 16 * s + 4 * t;           // elements d, d + 2 and d + 1, d + 3
                const uint2 w = on && d < dim ? *reinterpret_cast<const uint2*>(qp + d) : make_uint2(0u, 0u);
                qb[i][s][0] = __byte_perm(w.x, w.y, 0x5410);
                qb[i][s][1] = __byte_perm(w.x, w.y, 0x7632);
                qmax = fmaxf(qmax, fmaxf(fabsf(__uint_as_float(w.x << 16)), fabsf(__uint_as_float(w.x & 0xffff0000u))));
                qmax = fmaxf(qmax, fmaxf(fabsf(__uint_as_float(w.y << 16)), fabsf(__uint_as_float(w.y & 0xffff0000u))));
            }
            qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, 1));
            qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, 2));
            // 2^e with qmax 2^e in [2^10, 2^11); the exponent kept where 2^e and 2^(24-e) are normal
            const int e = qmax > 0.f ? max(-90, min(90, 137 - (int)(__float_as_uint(qmax) >> 23))) : 0;
            const float up = __uint_as_float((uint32_t)(127 + e) << 23), down = __uint_as_float((uint32_t)(127 + 24 - e) << 23);
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t w = qb[i][s][k];
                    qb[i][s][k] = pack_h(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
                }
            // the product with a key of codes 0
            float zero[4] = {0.f, 0.f, 0.f, 0.f};
            const uint32_t key0[4] = {0x00800080u, 0x00800080u, 0x00800080u, 0x00800080u};
#pragma unroll
            for (int s = 0; s < kSteps; ++s) mma_f16(zero, key0, qb[i][s][0], qb[i][s][1]);
#pragma unroll
            for (int x = 0; x < 2; ++x) {               // lane 4 n holds head n's
                ch[i][x] *= __shfl_sync(0xffffffffu, down, 8 * t + 4 * x);
                s0[i][x] = -zero[x];
            }
        } else {
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int d = 16 * s + 2 * t;
                qb[i][s][0] = on && d < dim ? *reinterpret_cast<const uint32_t*>(qp + d) : 0u;
                qb[i][s][1] = on && d < dim ? *reinterpret_cast<const uint32_t*>(qp + d + 8) : 0u;
            }
        }
    }

    float o[NT][DP / 16][4];
    // of heads 2t, 2t + 1: references (mz: m, or 0 while m is -inf), fw = 2^(m - mw + kLift), sum
    float m[NT][2], mz[NT][2], mw[NT][2], fw[NT][2], l[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][k][e] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) m[i][e] = mw[i][e] = -INFINITY, mz[i][e] = 0.f, fw[i][e] = INFINITY, l[i][e] = 0.f;
    }

    for (; j < end; j += kStep) {
        // the unit kStages - 1 ahead goes into the stage that the last unit left
        int ahead = stage + R::kStages - 1;
        if (ahead >= R::kStages) ahead -= R::kStages;
        fetch(rows[R::kStages - 1], j + (R::kStages - 1) * kStep, ahead);
        asm volatile("cp.async.wait_group %0;" ::"n"(R::kStages - 1) : "memory");
        __syncwarp();
        const int64_t row = rows[0];
#pragma unroll
        for (int st = 0; st + 1 < R::kStages; ++st) rows[st] = rows[st + 1];
        rows[R::kStages - 1] = next_row();
        const uint32_t base = ring + (uint32_t)(stage * R::kStage);
        stage = stage + 1 == R::kStages ? 0 : stage + 1;
        if (row < 0) {                                  // a page outside the cache: nothing to see
            __syncwarp();
            continue;
        }
        float ks[2] = {1.f, 1.f}, vs[2] = {1.f, 1.f};
        if constexpr (I8) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                ks[r] = lds4(base + 2 * R::kRows + 4 * (g + 8 * r));
                ks[r] = fmaf(0.f, ks[r], ks[r]);        // +inf stands for a row that reads as NaN
                vs[r] = lds4(base + 2 * R::kRows + 64 + 4 * (g + 8 * r));
            }
        }
        uint32_t at[DP / 32];                           // int8 keys' places, and values' behind them
#pragma unroll
        for (int ld = 0; ld < DP / 32; ++ld) at[ld] = base + R::step(key_at, 2 * ld);
        // ---- scores: S^T = K q^T, in two chains of products
        float s[NT][4], s1[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[i][e] = s0[i][e & 1], s1[i][e] = 0.f;
        if constexpr (I8) {
#pragma unroll
            for (int ld = 0; ld < DP / 32; ++ld) {      // 32 dimensions: two chunks of 16
                uint32_t x[4];
                matrices(x, at[ld]);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t af[4] = {raised<false>(x[2 * u]), raised<false>(x[2 * u + 1]),
                                            raised<true>(x[2 * u]), raised<true>(x[2 * u + 1])};
#pragma unroll
                    for (int i = 0; i < NT; ++i)
                        mma_f16(u ? s1[i] : s[i], af, qb[i][2 * ld + u][0], qb[i][2 * ld + u][1]);
                }
            }
        } else {
#pragma unroll
            for (int st = 0; st < kSteps; ++st) {       // 16 dimensions: two chunks of 8
                uint32_t x[4];
                matrices(x, base + R::step(key_at, 2 * st));
#pragma unroll
                for (int i = 0; i < NT; ++i) mma_b16(st & 1 ? s1[i] : s[i], x, qb[i][st][0], qb[i][st][1]);
            }
        }
        // ---- softmax weights; s[i][2 r + e]: key g + 8 r, head 2t + e
        bool grow = false;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float& x = s[i][2 * r + e];
                    x = (x + s1[i][2 * r + e]) * (I8 ? ch[i][e] * ks[r] : ch[i][e]);
                    if (j + kUnit > end) x = j + g + 8 * r < end ? x : -INFINITY;
                    grow = grow || x > m[i][e] + kSlack;
                }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = fmaxf(s[i][e], s[i][2 + e]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                    x = fmaxf(m[i][e], x);
                    const float f = x > -INFINITY ? ex2(m[i][e] - x) : 1.f;     // nothing yet: 2^-inf scales a zero
                    l[i][e] *= f;
                    m[i][e] = x;
                    mz[i][e] = x > -INFINITY ? x : 0.f;         // nothing but -inf so far: weights 0
                    if constexpr (I8) {
                        fw[i][e] = ex2(x - mw[i][e] + kLift);
                    } else {
#pragma unroll
                        for (int k = 0; k < DP / 16; ++k) {
                            o[i][k][e] *= f;
                            o[i][k][2 + e] *= f;
                        }
                    }
                }
        }
        float w[NT][4];
        grow = false;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float p = ex2(s[i][2 * r + e] - mz[i][e]);
                    l[i][e] += p;
                    w[i][2 * r + e] = I8 ? p * (fw[i][e] * vs[r]) : p;
                    grow = grow || (I8 && !(w[i][2 * r + e] <= kMost));
                }
        if constexpr (I8) {
            if (__any_sync(0xffffffffu, grow)) {        // too large for fp16: a new reference of the weights
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float y = fmaxf(s[i][e] + lg2(vs[0]), s[i][2 + e] + lg2(vs[1]));
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
                        y = fmaxf(mw[i][e], y);
                        const float f = y > -INFINITY ? ex2(mw[i][e] - y) : 1.f;
                        mw[i][e] = y;
                        fw[i][e] = ex2(m[i][e] - y + kLift);
#pragma unroll
                        for (int k = 0; k < DP / 16; ++k) {
                            o[i][k][e] *= f;
                            o[i][k][2 + e] *= f;
                        }
#pragma unroll
                        for (int r = 0; r < 2; ++r)     // a row of zeros, or none seen: weight 0
                            w[i][2 * r + e] = s[i][2 * r + e] == -INFINITY || vs[r] == 0.f
                                                  ? 0.f
                                                  : ex2(s[i][2 * r + e] + lg2(vs[r]) - ((y == -INFINITY ? 0.f : y) - kLift));
                    }
            }
        }
        uint32_t pb[NT][2], pl[NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float w0 = w[i][2 * r], w1 = w[i][2 * r + 1];
                if constexpr (I8) {
                    pb[i][r] = transpose8(pack_h(w0, w1));
                    pl[i][r] = 0u;
                } else {
                    pb[i][r] = transpose8(high_parts(w0, w1));
                    pl[i][r] = transpose8(low_parts(w0, w1));
                }
            }
        // ---- O^T += V^T P^T
        if constexpr (I8) {
#pragma unroll
            for (int ld = 0; ld < DP / 32; ++ld) {
                uint32_t x[4];
                matrices_t(x, at[ld] + R::kRows);
#pragma unroll
                for (int u = 0; u < 2; ++u) {           // rows g and g + 8: dimensions 2g and 2g + 1 of the chunk
                    const uint32_t af[4] = {halves<false>(x[2 * u]), halves<true>(x[2 * u]),
                                            halves<false>(x[2 * u + 1]), halves<true>(x[2 * u + 1])};
#pragma unroll
                    for (int i = 0; i < NT; ++i) mma_f16(o[i][2 * ld + u], af, pb[i][0], pb[i][1]);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) {
                uint32_t x[4];
                matrices_t(x, base + R::kRows + R::step(val_at, 2 * k));
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    mma_b16(o[i][k], x, pb[i][0], pb[i][1]);
                    mma_b16(o[i][k], x, pl[i][0], pl[i][1]);
                }
            }
        }
        __syncwarp();                                   // every lane is done with the stage
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();                                    // the rings become the warps' parts

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
                if constexpr (I8) {
                    *reinterpret_cast<float2*>(&s_o[warp][hd][16 * k + 2 * g]) = make_float2(o[i][k][e], o[i][k][2 + e]);
                } else {
                    s_o[warp][hd][16 * k + g] = o[i][k][e];
                    s_o[warp][hd][16 * k + 8 + g] = o[i][k][2 + e];
                }
            }
        }
    __syncthreads();
    if (threadIdx.x < kHeads) {
        // one head's maximum and sum over the warps, and what its parts are multiplied by; a warp that saw
        // no key has m = -inf and counts 0
        const int hd = threadIdx.x;
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][hd]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const bool any = s_m[w][hd] > -INFINITY || s_m[w][hd] != s_m[w][hd] || s_l[w][hd] != s_l[w][hd];
            L += any ? s_l[w][hd] * ex2(s_m[w][hd] - M) : 0.f;
            s_w[w][hd] = any ? ex2(s_w[w][hd] - M) : 0.f;
        }
        s_m[0][hd] = M;
        s_l[0][hd] = L;
        const int64_t at = (int64_t)b * a.n_q + h0 + hd;
        if (!kCluster && hd < nh && cut.pieces > 1)
            piece_sums<DP>(a, cut, gridDim.z)[at * cut.pieces + blockIdx.x] = make_float2(M, L);
        if (!kCluster && hd < nh && cut.pieces == 1 && a.lse) a.lse[at] = lse_of(M, L);
    }
    __syncthreads();
    for (int x = threadIdx.x; x < nh * (DP / 4); x += kThreads) {
        const int hd = x / (DP / 4), d = 4 * (x % (DP / 4));
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float4 v = *reinterpret_cast<const float4*>(&s_o[w][hd][d]);
            const float f = s_w[w][hd];
            acc.x += v.x * f, acc.y += v.y * f, acc.z += v.z * f, acc.w += v.w * f;
        }
        if constexpr (kCluster) {
            *reinterpret_cast<float4*>(&s_o[0][hd][d]) = acc;        // read above by this thread alone
        } else if (cut.pieces > 1) {
            const int64_t piece = ((int64_t)b * a.n_q + h0 + hd) * cut.pieces + blockIdx.x;
            *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.workspace) + piece * DP + d) = acc;
        } else if (d < dim) {
            store_out(reinterpret_cast<Tout*>(a.out) + (int64_t)b * a.o_st + (int64_t)(h0 + hd) * a.o_sh + d, acc,
                      s_l[0][hd]);
        }
    }
    if constexpr (kCluster) {
        // the pieces' parts, read from the cluster's CTAs, which share the elements out
        auto cluster = cg::this_cluster();
        cluster.sync();
        for (int x = (int)cluster.block_rank() * kThreads + threadIdx.x; x < nh * (DP / 4); x += cut.pieces * kThreads) {
            const int hd = x / (DP / 4), d = 4 * (x % (DP / 4));
            float M = -INFINITY, L = 0.f;
            for (int p = 0; p < cut.pieces; ++p) M = fmaxf(M, *cluster.map_shared_rank(&s_m[0][hd], p));
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int p = 0; p < cut.pieces; ++p) {
                const float mp = *cluster.map_shared_rank(&s_m[0][hd], p), lp = *cluster.map_shared_rank(&s_l[0][hd], p);
                const float4 v = *reinterpret_cast<const float4*>(cluster.map_shared_rank(&s_o[0][hd][d], p));
                const float f = mp == -INFINITY && lp == 0.f ? 0.f : ex2(mp - M);      // a piece that saw no key
                L += lp * f;
                acc.x += v.x * f, acc.y += v.y * f, acc.z += v.z * f, acc.w += v.w * f;
            }
            const int64_t at = (int64_t)b * a.n_q + h0 + hd;
            if (d < dim)
                store_out(reinterpret_cast<Tout*>(a.out) + (int64_t)b * a.o_st + (int64_t)(h0 + hd) * a.o_sh + d, acc, L);
            if (a.lse && d == 0) a.lse[at] = lse_of(M, L);
        }
        cluster.sync();                                 // no CTA leaves while its part is read
    }
}

// Joins the pieces of each (request, head): out = sum_p o_p 2^(m_p - m) / sum_p l_p 2^(m_p - m).  W warps
// of a block of eight share one head's pieces, four dimensions a lane, so that a hundred pieces cost a
// few loads' latency and a few pieces no idle warps.
constexpr int kJoinWarps = 8;
template <int DP, int W, typename Tout>
__global__ void __launch_bounds__(32 * kJoinWarps)
k_attn_decode_join(const AttnDecodeArgs a, const Cut cut) {
    constexpr int kLanes = DP / 4, kRows = W * 32 / kLanes;     // lanes of a piece's row, rows side by side
    constexpr int kSides = kJoinWarps / W;                      // heads of a block
    __shared__ float s_max[kJoinWarps], s_sum[kSides][kRows];
    __shared__ float4 s_acc[kSides][kRows][kLanes];
    const int side = threadIdx.x / (32 * W), tid = threadIdx.x % (32 * W);
    const int h = blockIdx.x * kSides + side, b = blockIdx.y;
    const int sub = tid % kLanes, first = tid / kLanes;
    const int n = h < a.n_q ? (length_of(a, b, false) + cut.tokens - 1) / cut.tokens : 0;
    const int64_t at = (int64_t)b * a.n_q + h;
    const float4* rows = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.workspace) + at * cut.pieces * DP) + sub;
    const float2* ml = piece_sums<DP>(a, cut, a.batch) + at * cut.pieces;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float M = -INFINITY;
    for (int p = tid; p < n; p += 32 * W) M = fmaxf(M, ml[p].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    if constexpr (W > 1) {
        if ((tid & 31) == 0) s_max[tid >> 5] = M;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, s_max[w]);
    }
    float L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = first; p < n; p += kRows) {
        const float2 x = ml[p];
        const float4 v = rows[(int64_t)p * kLanes];
        const float f = x.x == -INFINITY && x.y == 0.f ? 0.f : ex2(x.x - M);      // a piece that saw no key
        L += x.y * f;
        acc.x += v.x * f, acc.y += v.y * f, acc.z += v.z * f, acc.w += v.w * f;
    }
    s_acc[side][first][sub] = acc;
    if (sub == 0) s_sum[side][first] = L;
    __syncthreads();
    if (tid < kLanes && h < a.n_q) {
        L = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const float4 v = s_acc[side][r][tid];
            L += s_sum[side][r];
            acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
        }
        if (4 * tid < a.c.dim)
            store_out(reinterpret_cast<Tout*>(a.out) + (int64_t)b * a.o_st + (int64_t)h * a.o_sh + 4 * tid, acc, L);
        if (a.lse && tid == 0) a.lse[at] = lse_of(M, L);
    }
}

// CTAs side by side for one request's long axis: one per kv head and group of 16 (or 8) query heads.
int lanes_of(int n_q, int n_kv) {
    const int group = n_q / n_kv, heads = group > 8 ? 16 : 8;
    return n_kv * ((group + heads - 1) / heads);
}

Cut cut_of(int batch, int n_q, int n_kv, int64_t max_len) {
    const int64_t side = (int64_t)batch * lanes_of(n_q, n_kv);
    Cut c;
    auto even = [&](int64_t p) {
        c.tokens = (int)(((max_len + p - 1) / p + 63) / 64 * 64);
        c.pieces = (int)((max_len + c.tokens - 1) / c.tokens);
    };
    // A short call: at most eight pieces of 64 keys or more, joined by their cluster without a second launch:
    // one request of 1024 keys 12.9 -> 10.9 us, nine of 4096 31 -> 27.  A request or two of 4096 keys on 8 kv
    // heads want more than 64 CTAs: there 17 us against 13.  608 CTAs are on the GPU at once with int8 rows (152
    // SMs x 4).  The rule does not see the rows' type, and bf16 rows of 128 take two turns from 304 on: 8
    // requests on 8 kv heads by clusters / by pieces and join: 512 keys 12.1 / 8.6 us, 1024 15.5 / 14.6, 2048 20.2 /
    // 21.9, 4096 30 / 32 (int8: 8.8 / 9.0, 11.4 / 12.3, 14.9 / 18.9, 22 / 25).
    if (max_len > 64 && side * 8 <= 608 && (max_len <= 2048 || (max_len <= 4096 && side * 8 >= 152))) {
        const int64_t p = (max_len + 63) / 64;
        even(p < 8 ? p : 8);
        c.cluster = true;
        return c;
    }
    c.cluster = false;
    // Many CTAs of at least 512 keys, so that requests of different lengths fill the GPU evenly and the
    // join reads little; where that leaves fewer than 912 (1.5 turns of the 608 that are on the GPU at once
    // with int8 rows, three of the 304 with bf16 rows of 128), pieces down to 128 keys.
    int64_t p = (3648 + side - 1) / side;
    const int64_t most = (max_len + 511) / 512;
    if (p > most) p = most;
    if (side * p < 912) {
        p = (912 + side - 1) / side;
        const int64_t fine = (max_len + 127) / 128;
        if (p > fine) p = fine;
    }
    even(p);
    return c;
}

template <bool I8, int DP, int NT, bool kCluster, typename Tout>
int launch(const AttnDecodeArgs& a, const Cut& cut, cudaStream_t stream, const char** why) {
    constexpr int kRing = kWarps * Ring<I8, DP>::kStages * Ring<I8, DP>::kStage, kParts = kWarps * 8 * NT * (DP + 4) * 4;
    constexpr int kSmem = kRing > kParts ? kRing : kParts;
    auto kern = k_attn_decode<I8, DP, NT, kCluster, Tout>;
    static ContextMemo attr_memo;
    if (!opt_in_dynamic_smem(attr_memo, kern, kSmem, why)) return -1;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)cut.pieces, (unsigned)lanes_of(a.n_q, a.c.n_kv), (unsigned)a.batch);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    if (kCluster) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)cut.pieces;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.numAttrs = 1;
    }
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, cut);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e == cudaSuccess && !kCluster && cut.pieces > 1) {
        // launched while the pieces still run; it waits for them before it reads
        const bool many = cut.pieces > 16;              // a warp joins up to 16 pieces in two rounds of loads
        cfg.gridDim = dim3((unsigned)(many ? a.n_q : (a.n_q + kJoinWarps - 1) / kJoinWarps), (unsigned)a.batch);
        cfg.blockDim = dim3(32 * kJoinWarps);
        cfg.dynamicSmemBytes = 0;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 1;
        e = many ? cudaLaunchKernelEx(&cfg, k_attn_decode_join<DP, kJoinWarps, Tout>, a, cut)
                 : cudaLaunchKernelEx(&cfg, k_attn_decode_join<DP, 1, Tout>, a, cut);
        if (e == cudaSuccess) e = cudaGetLastError();
    }
    if (e == cudaSuccess) return 0;
    *why = cudaGetErrorString(e);
    return -1;
}

template <bool I8, int DP, int NT, typename Tout>
int launch_cut(const AttnDecodeArgs& a, cudaStream_t stream, const char** why) {
    const Cut cut = cut_of(a.batch, a.n_q, a.c.n_kv, a.max_len);
    return cut.cluster ? launch<I8, DP, NT, true, Tout>(a, cut, stream, why) : launch<I8, DP, NT, false, Tout>(a, cut, stream, why);
}

template <bool I8, typename Tout>
int launch_shape(const AttnDecodeArgs& a, cudaStream_t stream, const char** why) {
    const bool wide = a.n_q / a.c.n_kv > 8;
    if (a.c.dim <= 64) return wide ? launch_cut<I8, 64, 2, Tout>(a, stream, why) : launch_cut<I8, 64, 1, Tout>(a, stream, why);
    return wide ? launch_cut<I8, 128, 2, Tout>(a, stream, why) : launch_cut<I8, 128, 1, Tout>(a, stream, why);
}

}  // namespace

size_t attn_decode_workspace(int batch, int n_q, int n_kv, int dim, int max_len) {
    const Cut c = cut_of(batch, n_q, n_kv, max_len);
    return c.pieces == 1 || c.cluster ? 0 : (size_t)batch * n_q * c.pieces * ((dim <= 64 ? 64 : 128) + 2) * sizeof(float);
}

int launch_attn_decode(const AttnDecodeArgs& a, bool cache_i8, bool out_bf16, cudaStream_t stream, const char** why) {
    if (cache_i8)
        return out_bf16 ? launch_shape<true, __nv_bfloat16>(a, stream, why) : launch_shape<true, float>(a, stream, why);
    return out_bf16 ? launch_shape<false, __nv_bfloat16>(a, stream, why) : launch_shape<false, float>(a, stream, why);
}

}  // namespace ssm
