// w4.cu -- weights of 4 bits with a scale (and a zero) per group: w4_quantize makes them, w4_linear multiplies
// the few rows of a decode step by them.
//
// w4_linear.  The weight is read once, so bytes of codes and scales over the copy rate are the floor; what it
// takes to stay near it is few instructions per weight.  A block of 16 rows of the weight is an m16n8k16 matrix
// instruction's A, 8 rows of x its B.  A warp owns a slice of the elements of every row, for which it holds x in
// registers for the whole call; rows of codes come by asynchronous copies into a ring of shared memory, are read as 8 x 8
// matrices of 16-bit words (which gives a lane eight consecutive codes of a row, the k of two instructions, x
// being held in the same order), and become bf16 numbers 16 + code in two operations for two codes.  The group's
// sum is multiplied by its scale in fp32.  The warps' sums of a block meet in shared memory; where a row of x is
// more than 16 warps hold, slices of the rows go to different CTAs and a second kernel adds their sums.
// Measured, in a graph: 1 x 4096 -> 16384, groups of 128 (34.7 MB), 11.9 us, of which the bytes are 5.1.  With N it is 4.8 us
// and 0.435 for every 1000 rows (4.9 TB/s, 0.72 of the copy rate; N = 768 takes 3.5, 77824 38.7).  Neither part is
// accounted for in full: no unit is busy (integer pipe 45 %, 0.48 instructions a cycle and scheduler), so it is waits,
// at the ring, at the warps' exchange and for the first loads.  8 x 8192 -> 4096, groups of 32 with zeros, 13.2 us,
// 6.3 of it fixed (four slices, so two kernels) and 1.7 for every 1000 rows (2.9 TB/s: a scale, a zero and eight
// multiply-adds for every two products); 1 x 1536 -> 768 3.1 us.  x with several scales a row reads them inside the group
// loop: 8 x 4096 -> 16384 12.8 us with one, 15.2 with four; 8 x 8192 -> 4096 in groups of 32 13.3 and 18.2.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "ssm.h"
#include "w4.cuh"

namespace ssm {
namespace {

// ------------------------------------------------------------------ quantisation
// A warp per group: a lane holds group / 32 consecutive elements, loaded one by one.  The weight is made once and kept, so
// this is the simple kernel: 50021 x 2560 bf16 in groups of 128 246 us, of 32 738 (1.3 and 0.5 TB/s of what it reads and
// writes; fp32 takes the same time, so a group's instructions are what counts, not its bytes).
template <typename Tin, int E>
__global__ void __launch_bounds__(256) k_w4_quantize(const W4Weight w, const Tin* W, int64_t ldw, int64_t n_groups) {
    const int64_t id = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
    if (id >= n_groups) return;
    const int lane = threadIdx.x % 32, per_row = w.K / w.group;
    const int64_t row = id / per_row;
    const int g = (int)(id % per_row);
    float v[E], lo = 0.f, hi = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        v[i] = to_f32(W[row * ldw + (int64_t)g * w.group + lane * E + i]);
        lo = fminf(lo, v[i]), hi = fmaxf(hi, v[i]);
    }
    for (int o = 16; o > 0; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(~0u, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(~0u, hi, o));
    }
    // (hi - lo) / 15 by halves, whose difference is always finite
    float s = w.zeros ? __fdiv_rn(fmaf(hi, 0.5f, -0.5f * lo), 7.5f) : __fdiv_rn(fmaxf(-lo, hi), 7.f);
    if (w.scale_bf16) s = __bfloat162float(__float2bfloat16_rn(s));
    float zero = 8.f, least = 1.f, most = 15.f;
    if (w.zeros) {
        least = 0.f;
        if (s > 0.f) zero = fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.f), 15.f);
    }
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const float c = s > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(v[i], s)) + zero, least), most) : 8.f;
        bits |= (uint32_t)c << (4 * i);
    }
    uint8_t* codes = const_cast<uint8_t*>(w.codes) + row * w.ldc + (int64_t)g * (w.group / 2);
    if (E == 1) {                                       // two lanes' elements make a byte
        bits |= __shfl_down_sync(~0u, bits, 1) << 4;
        if (lane % 2 == 0) codes[lane / 2] = (uint8_t)bits;
    } else if (E == 2) {
        codes[lane] = (uint8_t)bits;
    } else {
        reinterpret_cast<uint16_t*>(codes)[lane] = (uint16_t)bits;
    }
    if (lane == 0) {
        if (w.scale_bf16) reinterpret_cast<__nv_bfloat16*>(const_cast<void*>(w.scales))[row * w.lds + g] = __float2bfloat16_rn(s);
        else reinterpret_cast<float*>(const_cast<void*>(w.scales))[row * w.lds + g] = s;
        if (w.zeros) const_cast<uint8_t*>(w.zeros)[row * w.ldz + g] = (uint8_t)zero;
    }
}

// ------------------------------------------------------------------ the product
constexpr int kWarps = 16;                              // that compute
constexpr int kServe = 4;                               // that fetch the weight, sum the warps' parts up and store
constexpr int kThreads = 32 * (kWarps + kServe);
static_assert(32 * kServe == 8 * 16, "eight service threads for each of a stage's 16 rows");
constexpr int kRows = 16;                               // of the weight in a stage: a matrix instruction's M
constexpr int kCol = 20;                                // floats between columns of a part: 16 rows, no bank twice
constexpr int kMaxSmem = 227 * 1024;
constexpr int kMaxStages = 8;
constexpr int kSms = 152;

constexpr int kTiles = 2;                               // that a warp takes together: independent sums for the matrix pipe

// Of a kernel for 8 NT rows of x: the most chunks of 32 elements of a row that a warp holds x for (32 registers).
template <int NT> struct Shape {
    static constexpr int kChunks = 8 / NT;
    static constexpr int kPart = kTiles * NT * 8 * kCol, kOut = kTiles * NT * 128;
};

// How a call is cut up: the elements of a row into slices that a CTA's warps share out, the tiles of 16 rows of the
// weight into a range for each walker.  A CTA is a walker's, for one slice and one group of 8 NT rows of x.
struct W4Plan {
    int tiles, walkers, m_blocks, slices;
    int each, more;                                     // tiles of a walker; the first `more` walkers have one more
    int groups;                                         // of a row, in a slice
    int pitch_c, pitch_s, pitch_z, stage, stages;       // bytes of a row of codes, scales, zeros; of a stage
    int smem;
};

struct Bars {
    uint64_t full[kMaxStages], empty[kMaxStages];       // stages: copies there; read by all warps
    uint64_t part_full[2], part_empty[2];               // the warps' sums: written; read
};

// 16 bytes to shared memory, past the first level of cache.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives once this thread's copies so far are there.
__device__ __forceinline__ void arrive_after_copies(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two codes, 16 bits apart and at bit 3, as bf16 16 + code (16 has room for four bits below its leading one), in
// one operation: (w & mask) | 16.
__device__ __forceinline__ uint32_t two_codes(uint32_t w) {
    uint32_t v;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(v) : "r"(w), "r"(0x00780078u), "r"(0x41804180u));
    return v;
}
// A warp's slice of x: elements k .. of rows m, m + 8, ..., all loads in flight at once.  What is not there (rows
// from M on, chunks from n on) is loaded from the first place and counts as 0.
template <typename Q, int KC, int NT>
__device__ __forceinline__ void load_x(const W4LinearArgs& a, int m, int k, int n, uint32_t (&x)[KC][NT][4]) {
    constexpr int kSize = sizeof(Q) / 8;                // of an element
    Q q[KC][NT];
#pragma unroll
    for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const bool there = c < n && m + 8 * i < a.M;
            const int64_t at = there ? (int64_t)(m + 8 * i) * a.ldx + k + 32 * c : 0;
            q[c][i] = *reinterpret_cast<const Q*>(reinterpret_cast<const uint8_t*>(a.x) + at * kSize);
        }
#pragma unroll
    for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            x_pairs(q[c][i], x[c][i]);
            if (!(c < n && m + 8 * i < a.M)) x[c][i][0] = x[c][i][1] = x[c][i][2] = x[c][i][3] = 0;
        }
}

// Shared memory by its 32-bit address: a compute warp has no registers to spare for 64-bit ones.
__device__ __forceinline__ uint32_t ld_u8(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_u16(uint32_t at) {
    uint32_t v;
    asm volatile("{\n\t.reg .u16 h;\n\tld.shared.u16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_u32(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_f32x2(uint32_t at) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    return v;
}
// Of x's scales, inside the group loop: kept where it stands, else the loads of all groups are begun early and 16 rows spill.
__device__ __forceinline__ float ld_global(const float* at) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(at) : "memory");
    return v;
}
__device__ __forceinline__ void st_f32(uint32_t at, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory"); }
__device__ __forceinline__ void arrive_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// PG: chunks in a group.
template <int NT, int PG>
__global__ void __launch_bounds__(kThreads, 1) k_w4_linear(const W4LinearArgs a, const W4Plan plan, unsigned int* status) {
    using S = Shape<NT>;
    constexpr int KC = S::kChunks;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* const stages = smem;
    float* const red = reinterpret_cast<float*>(smem + plan.stages * plan.stage);          // [2][kWarps][kPart]
    float* const sums = red + 2 * kWarps * S::kPart;                                       // [kWarps][KC][8 NT]
    Bars& bars = *reinterpret_cast<Bars*>(sums + kWarps * KC * 8 * NT);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int slice = blockIdx.z, m0 = blockIdx.y * 8 * NT, walker = blockIdx.x;
    const int tile0 = walker * plan.each + min(walker, plan.more), tile1 = tile0 + plan.each + (walker < plan.more);
    // tiles of the turn that begins at one: two, but the last two by themselves, so that little is left to do once
    // the last data are there
    auto turn = [&](int tile) { return tile1 - tile > 2 ? kTiles : 1; };
    // this CTA's groups of a row
    const int g0 = slice * plan.groups, gn = min(plan.groups, a.w.K / (32 * PG) - g0);
    const int es = a.w.scale_bf16 ? 2 : 4, s_skip = g0 * es % 16, z_skip = g0 % 16;
    const int off_s = kRows * plan.pitch_c, off_z = off_s + kRows * plan.pitch_s;
    Waiter wait{status};

    if (threadIdx.x == 0) {
        for (int s = 0; s < plan.stages; ++s) mbar_init(&bars.full[s], 32 * kServe), mbar_init(&bars.empty[s], kWarps);
        for (int b = 0; b < 2; ++b) mbar_init(&bars.part_full[b], kWarps), mbar_init(&bars.part_empty[b], kServe);
    }
    fence_barrier_init();
    __syncthreads();
    after_previous();
    next_may_start();

    if (warp < kWarps) {
        // ---- the products
        const int g = lane / 4, t = lane % 4;
        // this warp's groups, dealt evenly over the warps and over the SM's four parts that issue for every fourth
        const int turn_of = warp % 4 * (kWarps / 4) + warp / 4;
        const int w0 = gn * turn_of / kWarps, wn = gn * (turn_of + 1) / kWarps - w0;
        uint32_t x[KC][NT][4];
        if (a.x_i8) load_x<uint2>(a, m0 + g, (g0 + w0) * PG * 32 + 8 * t, wn * PG, x);
        else load_x<uint4>(a, m0 + g, (g0 + w0) * PG * 32 + 8 * t, wn * PG, x);
        // The codes go in as 16 + code: a group's sum is that, less (16 + zero) times the sum of its x, which is
        // found the same way, as a product with ones.
        const uint32_t my_sums = smem_u32(sums + warp * (KC / PG) * 8 * NT) + 8 * t;
#pragma unroll
        for (int j = 0; j < KC / PG; ++j)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float one[4] = {};
#pragma unroll
                for (int c = j * PG; c < (j + 1) * PG; ++c) {
                    mma(one, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, x[c][n][0], x[c][n][1]);
                    mma(one, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, x[c][n][2], x[c][n][3]);
                }
                if (g == 0) st_f32(my_sums + (j * NT + n) * 32, one[0]), st_f32(my_sums + (j * NT + n) * 32 + 4, one[1]);
            }
        __syncwarp();
        const int x_block = a.w.K / (32 * PG) / a.x_blocks;  // groups
        const int row_at = (lane % 16) * plan.pitch_c + (w0 * PG + lane / 16) * 16;
        const int s_at = off_s + g * plan.pitch_s + s_skip + w0 * es, z_at = off_z + g * plan.pitch_z + z_skip + w0;
        uint32_t full_parity = 0, part_parity = 1;
        int s = 0, buf = 0;
        auto products = [&](auto many) {
            constexpr int RT = decltype(many)::value;
            uint32_t st[RT], done[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                wait(&bars.full[s], full_parity);
                st[r] = smem_u32(stages) + s * plan.stage, done[r] = smem_u32(&bars.empty[s]);
                if (++s == plan.stages) s = 0, full_parity ^= 1;
            }
            float acc[RT][NT][4] = {};
#pragma unroll
            for (int j = 0; j < KC / PG; ++j) {
                if (j >= wn) break;
                // a group's words, scales and zeros, all under way before the first is used
                uint32_t q[RT][(PG + 1) / 2][4], sb[RT][2], zb[RT][2] = {};
                float2 xs[NT];
#pragma unroll
                for (int c = 0; c < PG; c += 2)         // two chunks' words; of a group of one chunk the first counts
#pragma unroll
                    for (int r = 0; r < RT; ++r) ldmatrix4(q[r][c / 2], st[r] + row_at + (j * PG + c) * 16);
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const uint32_t sp = st[r] + s_at + j * es, zp = st[r] + z_at + j;
                    if (a.w.scale_bf16) sb[r][0] = ld_u16(sp) << 16, sb[r][1] = ld_u16(sp + 8 * plan.pitch_s) << 16;
                    else sb[r][0] = ld_u32(sp), sb[r][1] = ld_u32(sp + 8 * plan.pitch_s);
                    if (a.w.zeros) zb[r][0] = ld_u8(zp), zb[r][1] = ld_u8(zp + 8 * plan.pitch_z);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) xs[n] = ld_f32x2(my_sums + (j * NT + n) * 32);
                float part[RT][NT][4] = {};
#pragma unroll
                for (int c = 0; c < PG; ++c)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int r = 0; r < RT; ++r) {
                            const uint32_t u = q[r][c / 2][c % 2 * 2], v = q[r][c / 2][c % 2 * 2 + 1];
                            const uint32_t a0 = two_codes(h ? u >> 5 : u << 3), a1 = two_codes(h ? v >> 5 : v << 3);
                            const uint32_t a2 = two_codes(h ? u >> 9 : u >> 1), a3 = two_codes(h ? v >> 9 : v >> 1);
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma(part[r][n], a0, a1, a2, a3, x[j * PG + c][n][2 * h], x[j * PG + c][n][2 * h + 1]);
                        }
                // the group's sums times its scales
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const float s0 = __uint_as_float(sb[r][0]), s1 = __uint_as_float(sb[r][1]);
                    float z0 = 24.f, z1 = 24.f;
                    if (a.w.zeros) {                    // 16 + zero, as the codes
                        z0 = __uint_as_float(0x41800000u | (zb[r][0] & 15u) << 19);
                        z1 = __uint_as_float(0x41800000u | (zb[r][1] & 15u) << 19);
                    }
                    float(&p)[NT][4] = part[r];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        p[n][0] = fmaf(-z0, xs[n].x, p[n][0]), p[n][1] = fmaf(-z0, xs[n].y, p[n][1]);
                        p[n][2] = fmaf(-z1, xs[n].x, p[n][2]), p[n][3] = fmaf(-z1, xs[n].y, p[n][3]);
                        if (a.x_blocks > 1) {
                            const int m = m0 + 8 * n + 2 * t, blk = (g0 + w0 + j) / x_block;
                            const float x0 = m < a.M ? ld_global(a.x_scale + (int64_t)m * a.x_blocks + blk) : 0.f;
                            const float x1 = m + 1 < a.M ? ld_global(a.x_scale + (int64_t)(m + 1) * a.x_blocks + blk) : 0.f;
                            p[n][0] *= x0, p[n][1] *= x1, p[n][2] *= x0, p[n][3] *= x1;
                        }
                        acc[r][n][0] = fmaf(p[n][0], s0, acc[r][n][0]), acc[r][n][1] = fmaf(p[n][1], s0, acc[r][n][1]);
                        acc[r][n][2] = fmaf(p[n][2], s1, acc[r][n][2]), acc[r][n][3] = fmaf(p[n][3], s1, acc[r][n][3]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) {
#pragma unroll
                for (int r = 0; r < RT; ++r) arrive_at(done[r]);
            }
            wait(&bars.part_empty[buf], part_parity);
            uint32_t to = smem_u32(red + (buf * kWarps + warp) * S::kPart + 2 * t * kCol + g);
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int n = 0; n < NT; ++n, to += 8 * kCol * 4) {
                    st_f32(to, acc[r][n][0]), st_f32(to + kCol * 4, acc[r][n][1]);
                    st_f32(to + 32, acc[r][n][2]), st_f32(to + kCol * 4 + 32, acc[r][n][3]);
                }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.part_full[buf]);
            buf ^= 1, part_parity ^= buf == 0;
        };
        for (int tile = tile0; tile < tile1; tile += turn(tile)) {
            if (turn(tile) == kTiles) products(std::integral_constant<int, kTiles>());
            else products(std::integral_constant<int, 1>());
        }
    } else {
        const int me = threadIdx.x - 32 * kWarps;
        // ---- the copies: eight threads for each row of a stage, 128 bytes of it at a time
        const int row = me / 8, part8 = me % 8;
        const int pieces_c = gn * PG, pieces_s = (s_skip + gn * es + 15) / 16, pieces_z = a.w.zeros ? (z_skip + gn + 15) / 16 : 0;
        uint32_t empty_parity = 1;
        int load = tile0, ls = 0;                       // the next tile to load and its stage
        auto fetch = [&]() {
            wait(&bars.empty[ls], empty_parity);
            const int64_t n = (int64_t)load * kRows + row;
            if (n < a.w.N) {
                const uint32_t to = smem_u32(stages) + ls * plan.stage + part8 * 16;
                const uint8_t* c = a.w.codes + n * a.w.ldc + ((int64_t)g0 * PG + part8) * 16;
                const uint32_t tc = to + row * plan.pitch_c;
                int i = part8;
                for (; i + 24 < pieces_c; i += 32, c += 512) {
                    const uint32_t at = tc + (i - part8) * 16;
                    copy16(at, c), copy16(at + 128, c + 128), copy16(at + 256, c + 256), copy16(at + 384, c + 384);
                }
                for (; i < pieces_c; i += 8, c += 128) copy16(tc + (i - part8) * 16, c);
                const uint8_t* sc = reinterpret_cast<const uint8_t*>(a.w.scales) + (n * a.w.lds + g0) * es - s_skip;
                for (i = part8; i < pieces_s; i += 8) copy16(to + off_s + row * plan.pitch_s + (i - part8) * 16, sc + i * 16);
                for (i = part8; i < pieces_z; i += 8)
                    copy16(to + off_z + row * plan.pitch_z + (i - part8) * 16, a.w.zeros + n * a.w.ldz + g0 - z_skip + i * 16);
            }
            arrive_after_copies(&bars.full[ls]);
            ++load;
            if (++ls == plan.stages) ls = 0, empty_parity ^= 1;
        };
        // ---- the warps' sums
        uint32_t parity = 0;
        int buf = 0;
        for (int s = 0; s < plan.stages && load < tile1; ++s) fetch();
        const int columns = min(8 * NT, a.M - m0);      // rows of x
        for (int tile = tile0; tile < tile1; tile += turn(tile)) {
            // the tiles that take this turn's stages: after its products, before its sums
            for (int r = 0; r < turn(tile) && load < tile1; ++r) fetch();
            wait(&bars.part_full[buf], parity);
            const float* const parts = red + buf * kWarps * S::kPart;
            auto finish = [&](int r, int m, int row, float v) {
                const int64_t n = (int64_t)(tile + r) * kRows + row;
                if (n >= a.w.N) return;
                if (a.x_scale && a.x_blocks == 1) v *= a.x_scale[m0 + m];
                if (plan.slices > 1) a.parts[((int64_t)slice * a.M + m0 + m) * a.w.N + n] = v;
                else w4_store(a, m0 + m, n, v);
            };
            const int outs = turn(tile) * columns * kRows;
            if (outs <= 8 * kServe) {                   // few: four threads for each
                const int e = me / 4, col = e / kRows, r = col / columns;
                float v = 0.f;
                if (e < outs) {
                    const float* from = parts + (r * 8 * NT + col - r * columns) * kCol + e % kRows;
#pragma unroll
                    for (int w = 0; w < kWarps / 4; ++w) v += from[(me % 4 + 4 * w) * S::kPart];
                }
                v += __shfl_xor_sync(~0u, v, 1);
                v += __shfl_xor_sync(~0u, v, 2);
                if (e < outs && me % 4 == 0) finish(r, col - r * columns, e % kRows, v);
            } else {
                for (int e = me; e < outs; e += 32 * kServe) {
                    const int col = e / kRows, r = col >= columns;
                    const float* from = parts + (r * 8 * NT + col - r * columns) * kCol + e % kRows;
                    float p[kWarps], v = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) p[w] = from[w * S::kPart];
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) v += p[w];
                    finish(r, col - r * columns, e % kRows, v);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.part_empty[buf]);
            buf ^= 1, parity ^= buf == 0;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");            // also after a wait that expired
    }
}

// The slices' sums of an output, in their order.
__global__ void __launch_bounds__(256) k_w4_join(const W4LinearArgs a, int slices) {
    after_previous();
    next_may_start();
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (n >= a.w.N) return;
    const int m = blockIdx.y;
    float v = 0.f;
#pragma unroll 8
    for (int s = 0; s < slices; ++s) v += a.parts[((int64_t)s * a.M + m) * a.w.N + n];
    w4_store(a, m, n, v);
}

template <int NT>
W4Plan plan_of(int M, const W4Weight& w, int slices) {
    using S = Shape<NT>;
    const int es = w.scale_bf16 ? 2 : 4, groups = w.K / w.group;
    W4Plan p;
    p.tiles = (w.N + kRows - 1) / kRows;
    p.m_blocks = (M + 8 * NT - 1) / (8 * NT);
    p.groups = (groups + slices - 1) / slices;
    p.slices = (groups + p.groups - 1) / p.groups;      // none is empty
    p.walkers = kSms / (p.slices * p.m_blocks);
    if (p.walkers < 1) p.walkers = 1;
    if (p.walkers > p.tiles) p.walkers = p.tiles;
    p.each = p.tiles / p.walkers, p.more = p.tiles % p.walkers;
    // 16 bytes past a multiple of 128: rows of a column of words fall on different banks.  A slice may start
    // inside 16 bytes of scales or zeros, and two chunks' words are read together.
    p.pitch_c = (p.groups * w.group / 2 + 16 + 127) / 128 * 128 + 16;
    p.pitch_s = (p.groups * es + 32 + 127) / 128 * 128 + 16;
    p.pitch_z = w.zeros ? (p.groups + 32 + 127) / 128 * 128 + 16 : 0;
    p.stage = kRows * (p.pitch_c + p.pitch_s + p.pitch_z);
    const int fixed = (2 * kWarps * S::kPart + kWarps * S::kChunks * 8 * NT) * 4 + (int)sizeof(Bars);
    p.stages = (kMaxSmem - fixed) / p.stage;
    p.stages = p.stages > kMaxStages ? kMaxStages : p.stages / kTiles * kTiles;   // whole turns
    p.smem = p.stages * p.stage + fixed;
    return p;
}

// The slices with the least time by a simple count: a walker's most tiles, at an SM's share of the copy rate (44 bytes
// a nanosecond), and two microseconds for the second kernel that several slices need.
template <int NT>
W4Plan best_plan(int M, const W4Weight& w) {
    const int most = kWarps * (Shape<NT>::kChunks * 32 / w.group);
    W4Plan best{};
    int64_t least = 0;
    for (int slices = (w.K / w.group + most - 1) / most, i = 0; i < 6; ++slices, ++i) {
        const W4Plan p = plan_of<NT>(M, w, slices);
        const int64_t bytes = (int64_t)((p.tiles + p.walkers - 1) / p.walkers) * p.groups * (kRows * w.group / 2);
        const int64_t ns = bytes / 44 + (p.slices > 1 ? 2000 : 0);
        if (i == 0 || ns < least) best = p, least = ns;
    }
    return best;
}

template <int NT, int PG>
int linear(const W4LinearArgs& a, unsigned int* status, cudaStream_t stream, const char** why) {
    const W4Plan p = best_plan<NT>(a.M, a.w);
    auto kern = k_w4_linear<NT, PG>;
    static ContextMemo attr_memo;
    if (!opt_in_dynamic_smem(attr_memo, kern, kMaxSmem, why)) return -1;
    if (launch_in_turn(kern, dim3((unsigned)p.walkers, (unsigned)p.m_blocks, (unsigned)p.slices), kThreads, p.smem, 1, stream, why, a, p, status))
        return -1;
    return p.slices > 1 ? launch_w4_join(a, p.slices, stream, why) : 0;
}

template <int NT>
int linear_of(const W4LinearArgs& a, unsigned int* status, cudaStream_t stream, const char** why) {
    if (a.w.group == 32) return linear<NT, 1>(a, status, stream, why);
    if (a.w.group == 64) return linear<NT, 2>(a, status, stream, why);
    return linear<NT, 4>(a, status, stream, why);
}

int done(const char** why) {
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return 0;
    *why = cudaGetErrorString(e);
    return -1;
}

template <typename Tin>
int quantize(const W4Weight& w, const Tin* W, int64_t ldw, cudaStream_t stream, const char** why) {
    const int64_t n = (int64_t)w.N * (w.K / w.group), blocks = (n + 7) / 8;
    if (blocks >= (1LL << 31)) {
        *why = "the weight has too many groups";
        return -1;
    }
    if (w.group == 32) k_w4_quantize<Tin, 1><<<(unsigned)blocks, 256, 0, stream>>>(w, W, ldw, n);
    else if (w.group == 64) k_w4_quantize<Tin, 2><<<(unsigned)blocks, 256, 0, stream>>>(w, W, ldw, n);
    else k_w4_quantize<Tin, 4><<<(unsigned)blocks, 256, 0, stream>>>(w, W, ldw, n);
    return done(why);
}

}  // namespace

int launch_w4_quantize(const W4Weight& w, const void* W, int64_t ldw, bool in_bf16, cudaStream_t stream, const char** why) {
    return in_bf16 ? quantize(w, static_cast<const __nv_bfloat16*>(W), ldw, stream, why)
                   : quantize(w, static_cast<const float*>(W), ldw, stream, why);
}

int launch_w4_join(const W4LinearArgs& a, int slices, cudaStream_t stream, const char** why) {
    return launch_in_turn(k_w4_join, dim3((unsigned)((a.w.N + 255) / 256), (unsigned)a.M), 256, 0, 1, stream, why, a, slices);
}

// Whether a call goes to the tiles of w4_tiles.cu: from nine rows of x on where the weight is large.  They unpack it
// once for 64 rows and cost two or three kernels; here it is unpacked for every 16 rows, and sums of 16 columns
// are what a turn waits for.  One border does for all groups; measured (us in a graph, here / tiles, with zeros):
//                                groups of 128     of 64         of 32
//     9 rows,  4096 x 4096        10.4 /  9.8      10.6 / 10.7   11.9 / 13.3
//    16 rows,  8192 x 4096        12.7 / 14.8      14.0 / 16.2   16.1 / 21.9
//    16 rows, 16384 x 4096        31   / 21        32   / 23     34   / 34
//    16 rows, 50021 x 2560        89   / 35        91   / 39     94   / 61
//    17 rows,  2048 x 2048         5.1 /  6.8       5.5 /  7.2    5.9 /  7.9
//    17 rows,  4096 x 4096        11.9 /  9.9      12.5 / 10.6   15.2 / 13.3
//    64 rows,  2048 x 2048         7.2 /  8.1       7.7 /  8.6    9.2 / 10.3
//    64 rows,  4096 x 4096        20   / 12        21   / 13     25   / 16
//   128 rows,  2048 x 2048        10.4 / 11.4      10.8 /  9.4   13.7 / 11.1
static bool in_tiles(int M, const W4Weight& w) {
    const int64_t work = (int64_t)((M + 15) / 16) * w.N * w.K;
    return M > 16 ? work > (1 << 24) : M > 8 && work > 3 * (1 << 24);
}

size_t w4_linear_workspace(int M, const W4Weight& w) {
    if (in_tiles(M, w)) return w4_tiles_workspace(M, w);
    const int slices = M <= 8 ? best_plan<1>(M, w).slices : best_plan<2>(M, w).slices;
    return slices == 1 ? 0 : (size_t)slices * M * w.N * sizeof(float);
}

int launch_w4_linear(const W4LinearArgs& a, unsigned int* status, cudaStream_t stream, const char** why) {
    if (in_tiles(a.M, a.w)) return launch_w4_tiles(a, status, stream, why);
    return a.M <= 8 ? linear_of<1>(a, status, stream, why) : linear_of<2>(a, status, stream, why);
}

}  // namespace ssm
