// attn_prefill.cu -- causal attention over packed prompts with grouped heads on the sm_103a
// tensor cores (tcgen05).
//
// Row i of a sequence with Lq queries and Lk keys sees the keys j < see_i = min(Lk, i + Lk - Lq + 1).
// One pass over the keys in blocks of 128 carries, per row, a reference m of the scores, the sum l
// and the output o, all in fp32:
//   p_j = 2^(c (s_j - m)), c = scale log2(e);   l += sum p_j;   o += sum p_j v_j
// out = o / l, lse = ln 2 (c m + log2 l).  Any m gives the same quotient; it is raised to the
// running maximum only when that has grown by more than 2^8 (kSlack, in units of c s), so that p
// stays below 2^8 and o is seldom rescaled.  (The running softmax, the reference raised late, and two tiles in
// turn with P kept in TMEM are published methods; the code is written from the formulas.)  p is rounded to
// bf16 for the second product, as the tensor cores take it with bf16 values; l sums it unrounded.  For few
// rows p is a bf16 pair.
//
// Two dense products per block bound it: 2 x 128 x 128 x D multiply-adds on the tensor cores and
// 128 x 128 exponentials.  The design keeps the tensor cores fed while the exponentials run:
//   * a CTA owns 256 query rows of one head as two tiles of 128; while one tile's softmax runs, the
//     tensor cores work on the other's products;
//   * warps 0-3 and 4-7: the softmax of tile 0 and 1, a thread per row (TMEM lane), the row's 128
//     scores in registers; they write p over their scores in TMEM, where tcgen05.mma takes it as
//     its A operand, and rescale and store o;
//   * warp 8: TMA loads of the two query tiles and a ring of key and value blocks;
//   * warp 9: issues the MMAs: per block and tile o += P V, then the next block's S = Q K^T, the tiles
//     in turn (issued independently the tiles fall into step, and both softmaxes then run while the
//     tensor cores idle: 2.98 ms instead of 2.51 in the case below);
//   * warps 10-11: make the value rows of blocks that some row does not wholly see harmless: the
//     product multiplies an unseen value by 0, which a NaN or an infinity survives.  Rows past the
//     sequence are zeroed; non-finite values are zeroed and noted (the first key of each column
//     that holds +inf, -inf, NaN), and the rows that do see them get them back at the end.
// Where the items are few and the keys many, the CTAs of a cluster share an item's key blocks and join
// their (m, l, o) through distributed shared memory.
// TMEM: scores of tile t at column 128 t, output at 256 + 128 t; all 512 columns, one CTA per SM.
// The grid runs the longest rows first (the last tiles of every head and sequence), so the tail is short.
//
// Measured: 16384 tokens, 56 query and 8 kv heads of 128: 2.55 ms a call among hundreds, 1510 TFLOP/s, 0.80 of
// cuBLAS's bf16 rate in a burst and 0.89 of its rate in a loop of seconds, under the power cap as these calls
// are; 2.38 ms (CUDA events over a few calls with pauses), of which the products alone take 2.2, as Q K^T reads
// 128 bytes of shared memory a cycle, all there is.  8 packed prompts of 266 to 4096 tokens, 32 / 8 heads: 194
// us, half of it the starts and ends of short CTAs: the grid has 4096, for the longest prompt's tiles of every
// sequence, of which 2752 find no rows.
#include <cooperative_groups.h>
#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace ssm {
namespace {

namespace cg = cooperative_groups;

constexpr int kM = 128;                 // query rows per tile
constexpr int kN = 128;                 // keys per block
constexpr int kThreads = 384;
constexpr float kSlack = 8.0f;

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

template <int DP>                       // head_dim padded to 64 or 128
struct Geo {
    static constexpr int kTile = 128 * DP * 2;                  // bytes of 128 rows
    static constexpr int kSlots = DP == 128 ? 4 : 8;            // ring of key and value blocks
    static constexpr int kOffKV = 2 * kTile;
    // a split item's part, over the operands: [256][DP + 4] outputs, then [256] (maximum, sum)
    static constexpr int kOffSums = 256 * (DP + 4) * 4;
    static constexpr int kOffBar = kOffKV + kSlots * kTile;
    static_assert(kOffSums + 256 * 8 <= kOffKV + kSlots * kTile, "a part fits over the operands");
    // q_full[2], s_full[2], p_full[2], o_full[2], v_raw[4], v_ok[4], kv_full[slots], kv_empty[slots],
    // TMEM address
    static constexpr int kBars = 16 + 2 * kSlots;
    static constexpr int kOffBad = kOffBar + kBars * 8 + 16;    // first bad key per column: [3][DP]
    static constexpr int kSmem = kOffBad + 3 * DP * 4 + 1024;   // + slack to align to 1024
    // tcgen05.mma kind::f16 instruction descriptors: fp32 accumulator, bf16 operands, M = 128;
    // scores: N = 128, both K-major; output: N = DP, B (values) MN-major
    static constexpr uint32_t kIdescS = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kN >> 3) << 17) | (8u << 24);
    static constexpr uint32_t kIdescO =
        (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(DP >> 3) << 17) | (8u << 24);
};

// o += P V with P (bf16 pairs) in TMEM.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Descriptor of an MN-major tile with 128-byte swizzling (rows of 128 bytes run along K, groups of 8
// rows 1024 bytes apart, the second 64 columns 16 KB on).
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(16384u >> 4) << 16) | ((uint64_t)(1024u >> 4) << 32) |
           ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}

// 32 columns of this thread's TMEM lane, not waited for.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
// Orders the uses of 32 loaded registers after the wait before it.
__device__ __forceinline__ void pin32(uint32_t* r) {
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
          "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
          "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Pairs of fp32 in one 64-bit register: one instruction for two sums or multiply-adds.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// kPair: the weights as bf16 pairs hi + lo, both multiplied with the values and both positive where the weight
// is, so that an infinite value keeps its sign.
// kSplit: the CTAs of a cluster share the key blocks of an item and join their outputs through
// distributed shared memory.
template <int DP, bool kPair, bool kSplit, typename Tout>
__global__ void __launch_bounds__(kThreads, 1)
k_attn_prefill(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
               const __grid_constant__ CUtensorMap tm_v, const AttnPrefillArgs a) {
    using G = Geo<DP>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ int s_err, s_bad;
    const unsigned splits = kSplit ? cg::this_cluster().num_blocks() : 1u, rank = kSplit ? cg::this_cluster().block_rank() : 0u;
    const unsigned item = blockIdx.x / splits, items = gridDim.x / splits;
    const int h = (int)(item % (unsigned)a.n_q), b = (int)(item / (unsigned)a.n_q % (unsigned)a.batch);
    const int row0 = (int)((items - 1 - item) / ((unsigned)a.n_q * (unsigned)a.batch)) * 2 * kM;
    // the sequence's rows, kept inside the tensors whatever cu_q and cu_k hold
    const int q0 = min(max(a.cu_q[b], 0), (int)a.total_q);
    int k0 = min(max(a.cu_k[b], 0), (int)a.total_k);
    const int lq = min(min(a.cu_q[b + 1], (int)a.total_q) - q0, a.max_q);
    const int lq_all = min(a.cu_q[b + 1], (int)a.total_q) - q0;
    int lk = max(min(a.cu_k[b + 1], (int)a.total_k) - k0, 0);
    if (row0 >= lq) return;                              // the same for the whole block, and cluster
    int off = lk - lq_all;                         // row i sees keys < min(lk, i + off + 1)
    // blocks of keys that tile t's rows see
    auto blocks = [&](int t) -> int {
        const int r = row0 + t * kM;
        if (r >= lq) return 0;
        const int see = min(lk, min(lq - 1, r + kM - 1) + off + 1);
        return see <= 0 ? 0 : (see + kN - 1) / kN;
    };
    if constexpr (kSplit) {                              // this CTA's share: as if the keys began and ended there
        const int all = max(blocks(0), blocks(1)), from = (int)((int64_t)all * rank / splits) * kN;
        lk = min(lk, (int)((int64_t)all * (rank + 1) / splits) * kN) - from;
        k0 += from;
        off -= from;
    }
    const int n0 = blocks(0), n1 = blocks(1), nb = max(n0, n1);
    // the first block that some row of the CTA's tiles does not wholly see; as 256 neighbouring rows'
    // limits span at most 255 keys, at most three blocks are left from it on
    const int whole = min(lk, row0 + off + 1);
    const int mask_from = whole <= 0 ? 0 : whole / kN;

    unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + G::kOffBar);
    uint64_t* s_full = q_full + 2;
    uint64_t* p_full = s_full + 2;
    uint64_t* o_full = p_full + 2;
    uint64_t* v_raw = o_full + 2;       // [4], one use each: a value block to be cleaned has landed
    uint64_t* v_ok = v_raw + 4;         // [4], one use each: it is clean
    uint64_t* kv_full = v_ok + 4;
    uint64_t* kv_empty = kv_full + G::kSlots;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(kv_empty + G::kSlots);
    int* bad = reinterpret_cast<int*>(smem + G::kOffBad);       // [3][DP]: +inf, -inf, NaN

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        s_err = 0;
        s_bad = 0;
        for (int t = 0; t < 2; ++t) {
            mbar_init(&q_full[t], 1);
            mbar_init(&s_full[t], 1);
            mbar_init(&p_full[t], 4);           // one arrival per softmax warp
            mbar_init(&o_full[t], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&v_raw[i], 1);
            mbar_init(&v_ok[i], 2);             // one arrival per cleaning warp
        }
        for (int s = 0; s < G::kSlots; ++s) {
            mbar_init(&kv_full[s], 1);
            mbar_init(&kv_empty[s], 1);
        }
        fence_barrier_init();
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    for (int i = threadIdx.x; i < 3 * DP; i += kThreads) bad[i] = 0x7fffffff;
    if (warp == 9) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto expired = [&]() {
        s_err = 1;
        atomicOr(a.status, 1u);
    };

    if (warp < 8) {
        // ---- softmax of tile t: thread = row.  The softmax warps take registers from the four service
        // warps: 256 x 208 + 128 x 88 = 384 x 168, the launch's total.
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int t = warp >> 2, quarter = warp & 3;
        const int n = t ? n1 : n0;
        const int row = row0 + t * kM + 32 * quarter + lane;
        const int see = row < lq ? min(lk, row + off + 1) : 0;
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        const uint32_t ts = tmem + lanes + (uint32_t)(128 * t), to = tmem + lanes + 256u + (uint32_t)(128 * t);
        const float c = a.scale * kLog2e;
        // from this block on a row of this tile does not see all of it
        const int whole_t = min(lk, row0 + t * kM + off + 1), mask_t = whole_t <= 0 ? 0 : whole_t / kN;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(&s_full[t], (uint32_t)(j & 1)))) {
                expired();
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t r[128];
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld32_async(ts + 32u * q, r + 32 * q);
            tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < 4; ++q) pin32(r + 32 * q);
            if (j >= mask_t) {
#pragma unroll
                for (int i = 0; i < 128; ++i)
                    if (j * kN + i >= see) r[i] = 0xff800000u;          // -inf
            }
            float mq[8];                                 // eight chains side by side
#pragma unroll
            for (int i = 0; i < 8; ++i) mq[i] = __uint_as_float(r[i]);
#pragma unroll
            for (int i = 8; i < 128; i += 16)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    mq[e] = i + 8 < 128 ? fmaxf(fmaxf(mq[e], __uint_as_float(r[i + e])), __uint_as_float(r[i + 8 + e]))
                                        : fmaxf(mq[e], __uint_as_float(r[i + e]));
            const float mx = fmaxf(fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])),
                                   fmaxf(fmaxf(mq[4], mq[5]), fmaxf(mq[6], mq[7])));
            if (j == 0) {
                m = mx;
            } else {
                const bool up = (mx - m) * c > kSlack;
                if (__any_sync(0xffffffffu, up)) {
                    // o belongs to this thread between the previous product's end and the next one's start
                    if (!__all_sync(0xffffffffu, mbar_wait_bounded(&o_full[t], (uint32_t)((j - 1) & 1)))) {
                        expired();
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const float f = up ? ex2((m - mx) * c) : 1.f;
                    if (up) m = mx;
                    l *= f;
#pragma unroll 1
                    for (int q = 0; q < DP / 32; ++q) {
                        uint32_t o[32];
                        tmem_ld32_async(to + 32u * q, o);
                        tmem_wait_ld();
                        pin32(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_st32(to + 32u * q, o);
                    }
                }
            }
            const float mc = m == -INFINITY ? 0.f : m * c;       // nothing but -inf so far: p = 0
            const uint64_t c2 = pair(c, c), mc2 = pair(-mc, -mc);
            uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t p[32], p_lo[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    float x0, x1;
                    unpair(fma2(pair(__uint_as_float(r[64 * q + 2 * i]), __uint_as_float(r[64 * q + 2 * i + 1])), c2, mc2),
                           x0, x1);
                    x0 = ex2(x0);
                    x1 = ex2(x1);
                    sum[i & 3] = add2(sum[i & 3], pair(x0, x1));
                    p[i] = kPair ? high_parts(x0, x1) : pack_bf16(x0, x1);
                    if constexpr (kPair) p_lo[i] = low_parts(x0, x1);
                }
                tmem_st32(ts + 32u * q, p);
                if constexpr (kPair) tmem_st32(ts + 64u + 32u * q, p_lo);
            }
            float l0, l1;
            unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), l0, l1);
            l += l0 + l1;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[t]);
        }
        if (ok && n > 0 && !__all_sync(0xffffffffu, mbar_wait_bounded(&o_full[t], (uint32_t)((n - 1) & 1)))) {
            expired();
            ok = false;
        }
        tc_fence_after();
        const bool any_bad = *(volatile int*)&s_bad != 0;
        // 32 columns of this row's output, not yet divided, with the non-finite values that it sees
        auto columns = [&](int q, float (&v)[32]) {
            uint32_t o[32];
            __syncwarp();
            if (n > 0) {
                tmem_ld32_async(to + 32u * q, o);
                tmem_wait_ld();
                pin32(o);
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = l == 0.f ? 0.f : __uint_as_float(o[i]);
            if (any_bad) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int col = 32 * q + i;
                    if (bad[col] < see) v[i] += INFINITY;
                    if (bad[DP + col] < see) v[i] -= INFINITY;
                    if (bad[2 * DP + col] < see) v[i] = NAN;
                }
            }
        };
        if constexpr (kSplit) {
            // both tiles' products are done: the operands' shared memory becomes this CTA's part
            asm volatile("bar.sync 1, 256;" ::: "memory");
            const int r = t * kM + 32 * quarter + lane;
            float* part = reinterpret_cast<float*>(smem) + r * (DP + 4);
#pragma unroll 1
            for (int q = 0; q < DP / 32; ++q) {
                float v[32];
                columns(q, v);
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    *reinterpret_cast<float4*>(part + 32 * q + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
            reinterpret_cast<float2*>(smem + G::kOffSums)[r] = make_float2(l == 0.f ? -INFINITY : m * c, l);
        } else {
            const bool store = ok && s_err == 0 && row < lq;
            const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
            if (store && a.lse) a.lse[(int64_t)(q0 + row) * a.n_q + h] = l == 0.f ? -INFINITY : kLn2 * (m * c + log2f(l));
            Tout* out = reinterpret_cast<Tout*>(a.out) + (int64_t)(q0 + row) * a.o_st + (int64_t)h * a.o_sh;
#pragma unroll 1
            for (int q = 0; q < DP / 32; ++q) {
                float v[32];
                columns(q, v);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] *= inv;
#pragma unroll
                for (int g = 0; g < 4; ++g) {                // eight columns at a time, whole or not at all
                    if (!store || 32 * q + 8 * g >= a.dim) continue;
                    if constexpr (sizeof(Tout) == 2) {
                        *reinterpret_cast<uint4*>(out + 32 * q + 8 * g) =
                            make_uint4(pack_bf16(v[8 * g], v[8 * g + 1]), pack_bf16(v[8 * g + 2], v[8 * g + 3]),
                                       pack_bf16(v[8 * g + 4], v[8 * g + 5]), pack_bf16(v[8 * g + 6], v[8 * g + 7]));
                    } else {
                        reinterpret_cast<float4*>(out + 32 * q + 8 * g)[0] =
                            make_float4(v[8 * g], v[8 * g + 1], v[8 * g + 2], v[8 * g + 3]);
                        reinterpret_cast<float4*>(out + 32 * q + 8 * g)[1] =
                            make_float4(v[8 * g + 4], v[8 * g + 5], v[8 * g + 6], v[8 * g + 7]);
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 8 && lane == 0 && nb > 0) {
            // ---- TMA producer: the query tiles, then K_0, V_0, K_1, V_1, ... through the ring
            const int hk = h / (a.n_q / a.n_kv);
            for (int t = 0; t < 2; ++t) {
                if ((t ? n1 : n0) == 0) continue;
                mbar_arrive_expect_tx(&q_full[t], G::kTile);
                for (int c = 0; c < DP / 64; ++c)
                    tma_load_3d(smem + t * G::kTile + c * 16384, &tm_q, &q_full[t], 64 * c, h, q0 + row0 + t * kM);
            }
            int it = 0;
            for (; it < 2 * nb; ++it) {
                const int s = it % G::kSlots;
                if (it >= G::kSlots && !mbar_wait_bounded(&kv_empty[s], (uint32_t)((it / G::kSlots + 1) & 1))) {
                    expired();
                    break;
                }
                unsigned char* dst = smem + G::kOffKV + s * G::kTile;
                uint64_t* full = &kv_full[s];
                if ((it & 1) && (it >> 1) >= mask_from) {     // by way of the cleaning warps
                    mbar_arrive(full);
                    full = &v_raw[(it >> 1) - mask_from];
                }
                mbar_arrive_expect_tx(full, G::kTile);
                for (int c = 0; c < DP / 64; ++c)
                    tma_load_3d(dst + c * 16384, it & 1 ? &tm_v : &tm_k, full, 64 * c, hk, k0 + (it >> 1) * kN);
            }
            // tail: every load has landed and the MMAs' last releases have arrived before the CTA ends
            for (int u = max(0, it - G::kSlots); u < it; ++u) {
                const bool raw = (u & 1) && (u >> 1) >= mask_from;
                if (!mbar_wait_bounded(raw ? &v_raw[(u >> 1) - mask_from] : &kv_full[u % G::kSlots],
                                       raw ? 0u : (uint32_t)((u / G::kSlots) & 1)))
                    expired();
                if (!s_err && !mbar_wait_bounded(&kv_empty[u % G::kSlots], (uint32_t)((u / G::kSlots) & 1))) expired();
            }
            for (int t = 0; t < 2; ++t)
                if ((t ? n1 : n0) > 0 && !mbar_wait_bounded(&q_full[t], 0)) expired();
        } else if (warp == 9 && nb > 0) {
            // ---- MMA issuer: the whole warp walks the loop, so that descriptors stay in uniform registers
            // (32 products a block leave 64 cycles for each), one elected lane issues.
            // S_t(j + 1) is issued right behind O_t += P_t(j) V and overwrites the columns that hold P_t(j).  This
            // relies on a CTA's products running in the order of their issue: the PTX manual promises that
            // for products of one accumulator and shape, and these have two.  They do run in order: with a wait
            // for O_t's commit in between every output has the same bits (8 shapes, heads of 64 to 128, whole,
            // paired and split, 60 calls each), and a call takes 12 % longer (16384 tokens 2.56 -> 2.87 ms,
            // 2 x 2048 rows over 14337 keys 1054 -> 1188 us, ragged prompts 194 -> 212 us).  TMEM has no columns
            // for P beside 2 x 128 of scores and 2 x 128 of outputs.
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                if (ok && !__all_sync(0xffffffffu, mbar_wait_bounded(bar, parity))) {
                    ok = false;
                    expired();
                }
            };
            const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0), tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint64_t qd = smem_desc_sw128(base), kd = smem_desc_sw128(base + G::kOffKV), vd = smem_desc_mn(base + G::kOffKV);
            auto scores = [&](int t, int slot) {             // S_t = Q_t K^T
                if (elect_one()) {
                    const uint64_t q = qd + (uint64_t)(t * (G::kTile >> 4)), k = kd + (uint64_t)(slot * (G::kTile >> 4));
#pragma unroll
                    for (int s = 0; s < DP / 16; ++s) {      // dimensions past head_dim are zeros
                        const uint64_t at = (uint64_t)((s >> 2) * (16384 >> 4) + 2 * (s & 3));
                        mma_bf16(tm + (uint32_t)(128 * t), q + at, k + at, G::kIdescS, s != 0);
                    }
                    mma_commit(&s_full[t]);
                }
                __syncwarp();
            };
            auto output = [&](int t, int slot, bool first) { // O_t += P_t V
                if (elect_one()) {
                    const uint64_t v = vd + (uint64_t)(slot * (G::kTile >> 4));
#pragma unroll
                    for (int s = 0; s < kN / 16; ++s)        // 16 keys: 8 columns of P, 2048 bytes of V
                        mma_bf16_ts(tm + (uint32_t)(256 + 128 * t), tm + (uint32_t)(128 * t + 8 * s),
                                    v + (uint64_t)(s * (2048 >> 4)), G::kIdescO, s != 0 || !first);
                    if constexpr (kPair) {
#pragma unroll
                        for (int s = 0; s < kN / 16; ++s)    // the low parts, 64 columns on
                            mma_bf16_ts(tm + (uint32_t)(256 + 128 * t), tm + (uint32_t)(128 * t + 64 + 8 * s),
                                        v + (uint64_t)(s * (2048 >> 4)), G::kIdescO, 1);
                    }
                    mma_commit(&o_full[t]);
                }
                __syncwarp();
            };
            auto release = [&](int slot) {
                if (elect_one()) mma_commit(&kv_empty[slot]);
                __syncwarp();
            };
            wait(&kv_full[0], 0);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if ((t ? n1 : n0) == 0) continue;
                wait(&q_full[t], 0);
                tc_fence_after();
                if (ok) scores(t, 0);
            }
            if (ok) release(0);
            for (int j = 0; j < nb && ok; ++j) {
                const int vi = 2 * j + 1, ki = 2 * j + 2, vslot = vi % G::kSlots, kslot = ki % G::kSlots;
                wait(&kv_full[vslot], (uint32_t)((vi / G::kSlots) & 1));
                if (j >= mask_from) wait(&v_ok[j - mask_from], 0);
                if (j + 1 < nb) wait(&kv_full[kslot], (uint32_t)((ki / G::kSlots) & 1));
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int n = t ? n1 : n0;
                    if (j >= n) continue;
                    wait(&p_full[t], (uint32_t)(j & 1));
                    tc_fence_after();
                    if (ok) output(t, vslot, j == 0);
                    if (ok && j + 1 < n) scores(t, kslot);
                }
                if (ok) release(vslot);
                if (ok && j + 1 < nb) release(kslot);
            }
        } else if (warp >= 10) {
            // ---- value blocks that some row does not wholly see
            for (int j = mask_from; j < nb; ++j) {
                const int vi = 2 * j + 1;
                if (!__all_sync(0xffffffffu, mbar_wait_bounded(&v_raw[j - mask_from], 0))) {
                    expired();
                    break;
                }
                unsigned char* v = smem + G::kOffKV + (vi % G::kSlots) * G::kTile;
                const int rows = lk - j * kN;                // of this sequence; later ones are zeroed
                // rows before `seen` are seen by every row of both tiles and stay as they are; eight chunks of
                // 16 bytes are looked at together, as nearly all are fine
                const int seen = max(whole - j * kN, 0);
                constexpr int kAhead = 8;
                for (int i0 = threadIdx.x - 320; i0 < G::kTile / 16; i0 += 64 * kAhead) {
                    uint4 x[kAhead];
                    __nv_bfloat162 z = __float2bfloat162_rn(0.f);
                    bool past = false;
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) {
                        const int i = i0 + 64 * u, r = (i >> 3) & 127;
                        x[u] = make_uint4(0u, 0u, 0u, 0u);
                        if (r >= seen && r < rows) x[u] = reinterpret_cast<const uint4*>(v)[i];
                        past = past || r >= rows;
                    }
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) {
                        const uint32_t ws[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)      // x 0: a NaN for an infinity or a NaN, a zero otherwise
                            z = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&ws[e]), __float2bfloat162_rn(0.f), z);
                    }
                    if ((*reinterpret_cast<const uint32_t*>(&z) & 0x7fff7fffu) == 0u && !past) continue;
                    for (int u = 0; u < kAhead; ++u) {
                        const int i = i0 + 64 * u, r = (i >> 3) & 127;
                        uint4* p = reinterpret_cast<uint4*>(v) + i;
                        if (r >= rows) {
                            *p = make_uint4(0u, 0u, 0u, 0u);
                            continue;
                        }
                        if (r < seen) continue;
                        const uint4 y = *p;
                        uint32_t ws[4] = {y.x, y.y, y.z, y.w};
                        bool fine = true;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            fine = fine && (ws[e] & 0x7f80u) != 0x7f80u && (ws[e] & 0x7f800000u) != 0x7f800000u;
                        if (fine) continue;
                        const int col = (i >> 10) * 64 + ((i & 7) ^ (r & 7)) * 8;       // the swizzle undone
                        for (int e = 0; e < 8; ++e) {
                            const uint32_t b16 = (ws[e >> 1] >> (16 * (e & 1))) & 0xffffu;
                            if ((b16 & 0x7f80u) != 0x7f80u) continue;
                            const int kind = b16 == 0x7f80u ? 0 : (b16 == 0xff80u ? 1 : 2);
                            atomicMin(&bad[kind * DP + col + e], j * kN + r);
                            ws[e >> 1] &= e & 1 ? 0x0000ffffu : 0xffff0000u;
                        }
                        *p = make_uint4(ws[0], ws[1], ws[2], ws[3]);
                        s_bad = 1;
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&v_ok[j - mask_from]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if constexpr (kSplit) {
        // out = sum_p o_p 2^(m_p - m) / sum_p l_p 2^(m_p - m) over the cluster's parts; a warp per row, every
        // splits-th row of the item
        auto cluster = cg::this_cluster();
        cluster.sync();
        for (int r = (int)rank + (int)splits * warp; r < 2 * kM && row0 + r < lq; r += (int)splits * (kThreads / 32)) {
            float M = -INFINITY, L = 0.f;
            for (unsigned p = 0; p < splits; ++p)
                M = fmaxf(M, cluster.map_shared_rank(reinterpret_cast<float2*>(smem + G::kOffSums), p)[r].x);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (unsigned p = 0; p < splits; ++p) {
                const float2 ml = cluster.map_shared_rank(reinterpret_cast<float2*>(smem + G::kOffSums), p)[r];
                if (ml.y == 0.f) continue;               // it holds no key that this row sees
                const float f = ex2(ml.x - M);
                L += ml.y * f;
                if (4 * lane < DP) {
                    const float4 v = *reinterpret_cast<const float4*>(
                        cluster.map_shared_rank(reinterpret_cast<float*>(smem), p) + r * (DP + 4) + 4 * lane);
                    acc.x += v.x * f, acc.y += v.y * f, acc.z += v.z * f, acc.w += v.w * f;
                }
            }
            if (s_err) continue;
            const int64_t token = (int64_t)q0 + row0 + r;
            const float inv = L == 0.f ? 0.f : 1.f / L;
            if (lane == 0 && a.lse) a.lse[token * a.n_q + h] = L == 0.f ? -INFINITY : kLn2 * (M + log2f(L));
            if (4 * lane < a.dim) {
                Tout* out = reinterpret_cast<Tout*>(a.out) + token * a.o_st + (int64_t)h * a.o_sh + 4 * lane;
                if constexpr (sizeof(Tout) == 2)
                    *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
                else
                    *reinterpret_cast<float4*>(out) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
            }
        }
        cluster.sync();                                  // no CTA leaves while its part is read
    }
}

// Map over [tokens][heads][dim] bf16 with the given strides: boxes of 128 tokens x one head x 64
// elements, 128-byte swizzle; elements past dim and rows past the tensor read as zero.
bool make_map(CUtensorMap* m, const void* base, int64_t tokens, int heads, int dim, int64_t st, int64_t sh) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {(cuuint64_t)sh * 2, (cuuint64_t)st * 2};
    cuuint32_t box[3] = {64, 1, 128};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pairs of query tiles over all sequences.
int64_t tile_pairs(const AttnPrefillArgs& a) { return ((int64_t)a.max_q + 2 * kM - 1) / (2 * kM) * a.batch; }

template <int DP, bool kPair, bool kSplit, typename Tout>
int launch_dp(const AttnPrefillArgs& a, unsigned splits, cudaStream_t stream, const char** why) {
    CUtensorMap mq, mk, mv;
    // without keys nothing is loaded; the maps then stand over q
    const bool keys = a.total_k > 0;
    if (!make_map(&mq, a.q, a.total_q, a.n_q, a.dim, a.q_st, a.q_sh) ||
        !make_map(&mk, keys ? a.k : a.q, keys ? a.total_k : a.total_q, keys ? a.n_kv : a.n_q, a.dim,
                  keys ? a.k_st : a.q_st, keys ? a.k_sh : a.q_sh) ||
        !make_map(&mv, keys ? a.v : a.q, keys ? a.total_k : a.total_q, keys ? a.n_kv : a.n_q, a.dim,
                  keys ? a.v_st : a.q_st, keys ? a.v_sh : a.q_sh)) {
        *why = "cuTensorMapEncodeTiled failed (driver entry point missing or layout rejected)";
        return -1;
    }
    auto kern = k_attn_prefill<DP, kPair, kSplit, Tout>;
    static ContextMemo attr;
    if (!opt_in_dynamic_smem(attr, kern, Geo<DP>::kSmem, why)) return -1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tile_pairs(a) * a.n_q * splits));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Geo<DP>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute cluster[1];
    cluster[0].id = cudaLaunchAttributeClusterDimension;
    cluster[0].val.clusterDim.x = splits;
    cluster[0].val.clusterDim.y = cluster[0].val.clusterDim.z = 1;
    cfg.attrs = cluster;
    cfg.numAttrs = kSplit ? 1 : 0;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, mq, mk, mv, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e == cudaSuccess) return 0;
    *why = cudaGetErrorString(e);
    return -1;
}

template <int DP, typename Tout>
int launch_shape(const AttnPrefillArgs& a, cudaStream_t stream, const char** why) {
    int dev = 0, n_sm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n_sm < 1) {
        *why = "cudaGetDevice / multiprocessor count failed";
        return -1;
    }
    // Where the items leave half of the SMs or more without work and have 2048 keys or more on average, up
    // to eight CTAs share the keys of one, 512 or more each: 8 rows of 32 heads over 4008 keys 66 -> 27 us,
    // 1024 rows of 16 heads over 9024 keys 115 -> 76; with 1024 keys the join's 6 us are not won back (19 -> 25).
    const int64_t items = tile_pairs(a) * a.n_q, keys = a.total_k / a.batch;
    unsigned splits = 1;
    while (splits < 8 && 2 * splits * items <= n_sm && keys >= 2048 && keys >= 2 * splits * 512) splits *= 2;
    // Few rows (a short chunk, some tokens to verify) take microseconds of latency whatever the weights
    // are: there they keep 16 bits.  On whole prompts the second product would cost a third of the time.
    if (a.total_q * a.n_q <= 256) return launch_dp<DP, true, true, Tout>(a, splits, stream, why);
    if (splits > 1) return launch_dp<DP, false, true, Tout>(a, splits, stream, why);
    return launch_dp<DP, false, false, Tout>(a, 1, stream, why);
}

}  // namespace

int launch_attn_prefill(const AttnPrefillArgs& a, bool out_bf16, cudaStream_t stream, const char** why) {
    if (a.dim <= 64)
        return out_bf16 ? launch_shape<64, __nv_bfloat16>(a, stream, why) : launch_shape<64, float>(a, stream, why);
    return out_bf16 ? launch_shape<128, __nv_bfloat16>(a, stream, why) : launch_shape<128, float>(a, stream, why);
}

}  // namespace ssm
