// w4_tiles.cu -- w4_linear for more than a few rows of x and a large weight: tiles of 128 rows of the
// 4-bit weight against up to 64 rows of x on the 5th-generation tensor cores.
//
// With 64 rows the product costs a warp's matrix instructions several times what the weight's bytes take, and the
// codes would be unpacked once for every 16 rows of x.  Here they are unpacked once for 64: a thread has a row of
// the weight, turns its codes into bf16 whole numbers code - zero (exact) and writes them to TMEM, where they are
// the A operand; x, in the order in which a word's codes come out, is B in shared memory.  A group's sums are an
// accumulator of their own (four of them in turn), which other threads, a row each, multiply by the group's
// scale and add up in fp32 registers.  Eight warps unpack (56 integer operations and 32 subtractions for 64 codes of
// 32 rows), eight scale, one each issues copies of codes, copies of x and products.  Measured: 64 x 2560 -> 50021, groups
// of 128 with zeros (67 MB, 16 GFLOP) 35 us, 0.34 us a step of 128 x 128 codes, at 0.54 instructions a cycle and
// scheduler; bytes are 10 us of it, products 9, and a seventh is that 391 tiles are no multiple of 152 SMs.  What bounds it
// is the way of a step from warp to warp (copies, unpacking, products, scaling): with nothing but its waits, arrivals and
// commits left the loop took 33 us of then 38.  With twelve unpacking warps 39, with sixteen (spilling) 135; steps of 64
// elements 53.  Groups of 64, two accumulators to hand over in a step, 44 us, of 32, four of them, 72.  More rows of x
// unpack the weight again for every 64: 128 rows 64 us, 256 112.  Several scales a row of x are read inside the scaling loop:
// 96 us with four where one takes 36.
#include <type_traits>

#include "kernels.h"
#include "ssm.h"
#include "tcgen05.cuh"
#include "w4.cuh"

namespace ssm {
namespace {

constexpr int kRows = 128;                              // of the weight: an MMA's M
constexpr int kStep = 128;                              // elements of a step: 64 TMEM columns, two tiles of x
constexpr int kStageK = 256;                            // elements in a stage of codes: rows of 128 bytes
constexpr int kStageC = kRows * kStageK / 2;
constexpr int kCodeStages = 6;
constexpr int kSteps = 4;                               // under way: A operands in TMEM and x in shared memory
constexpr int kD = 4;                                   // accumulators in TMEM
constexpr int kSets = 2, kUnpack = 4 * kSets, kScale = 8;       // warps; then one each for codes, x and products
constexpr int kThreads = 32 * (kUnpack + kScale + 3);
static_assert(kSteps == kD, "a step that is a group has one barrier for both");

template <int MP> struct Geo {                          // rows of x: 32 or 64
    static constexpr int kStageX = MP * kStep * 2;
    static constexpr int kOffX = kCodeStages * kStageC;
    static constexpr int kOffBar = kOffX + kSteps * kStageX;
    static constexpr int kSmem = kOffBar + (2 * kCodeStages + 2 * kSteps + 2 * kD) * 8 + 16 + 1024;    // + to align
    static constexpr uint32_t kColD = kStep / 2 * kSteps;          // TMEM: A operands, then accumulators
    // fp32 accumulator, bf16 operands, M = 128, N = MP, both K-major
    static constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(MP >> 3) << 17) | (8u << 24);
};

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void mma_from_tmem(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
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
__device__ __forceinline__ uint4 ld_u128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
// Sixteen zeros of a row, where they stand in the loop: left to move, the load cost groups of 128 three hundredths (64 x 2560 ->
// 50021 36.0 us, so 34.9), and the same for scales costs groups of 64 a fiftieth.
__device__ __forceinline__ uint4 ld_global(const uint4* at) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(at));
    return v;
}
// bf16 128 + zero twice, of a group's zero
__device__ __forceinline__ uint32_t zero_pair(uint32_t z) { return (0x4300u | (z & 15u)) * 0x10001u; }
// Two codes, 16 bits apart, as bf16 128 + code (its last place is 1 there), less 128 + zero: exact.
__device__ __forceinline__ uint32_t less_zero(uint32_t w, uint32_t zero) {
    uint32_t v;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(v) : "r"(w), "r"(0x000f000fu), "r"(0x43004300u));
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), *reinterpret_cast<const __nv_bfloat162*>(&zero));
    return *reinterpret_cast<const uint32_t*>(&d);
}

// A position in a ring of stages and the parity of its turn.
struct Ring {
    int at = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        if (++at == kCodeStages) at = 0, parity ^= 1;
    }
};

struct Cut {                    // of a call
    int tiles, slices, m_blocks;
    int slice_k;                // elements of a row in a slice: a multiple of a stage's
};

// Steps, groups and stages are counted over all the tiles of a CTA: step r has A operand and x stage r % kSteps, in
// the turn r / kSteps; group q accumulator q % kD.
template <int MP, int GK>                               // rows of x, elements of a group
__global__ void __launch_bounds__(kThreads, 1)
k_w4_tiles(const __grid_constant__ CUtensorMap tm_codes, const __grid_constant__ CUtensorMap tm_x, const W4LinearArgs a,
           const Cut cut, unsigned int* status) {
    using G = Geo<MP>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* const c_full = reinterpret_cast<uint64_t*>(smem + G::kOffBar);
    uint64_t *const c_empty = c_full + kCodeStages, *const full = c_empty + kCodeStages;
    // where a step is a group, one commit tells both that its operands are used and that its sums are there
    uint64_t *const d_full = full + kSteps, *const used = GK == kStep ? d_full : d_full + kD, *const d_empty = d_full + kD + kSteps;
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(d_empty + kD);
    uint64_t* const done = d_empty + kD + 1;

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int m0 = blockIdx.y * MP, slice = blockIdx.z;
    const int k0 = slice * cut.slice_k, kn = min(cut.slice_k, a.w.K - k0);
    const int steps = (kn + kStep - 1) / kStep, groups = kn / GK, j0 = k0 / GK;
    Waiter wait{status};

    if (threadIdx.x == 0) {
        for (int i = 0; i < kCodeStages; ++i) mbar_init(&c_full[i], 1), mbar_init(&c_empty[i], kUnpack);
        for (int i = 0; i < kSteps; ++i) mbar_init(&full[i], 4 + 1), mbar_init(&used[i], 1);      // operand and x
        for (int i = 0; i < kD; ++i) {
            if (GK != kStep) mbar_init(&d_full[i], 1);
            mbar_init(&d_empty[i], kScale);
        }
        mbar_init(done, 1);
        fence_barrier_init();
        prefetch_tmap(&tm_codes);
        prefetch_tmap(&tm_x);
    }
    if (warp == kUnpack + kScale) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    after_previous();                                   // x in its order comes from the kernel before
    next_may_start();

    if (warp < kUnpack) {
        // ---- codes to operands: a row of the weight each; the sets of four warps take the steps in turn
        const uint32_t set = warp / 4, row = 32 * (warp % 4) + lane;
        const uint32_t lanes = (uint32_t)(32 * (warp % 4)) << 16;
        Ring cs;
        uint32_t r = 0;
        for (int tile = blockIdx.x; tile < cut.tiles; tile += gridDim.x) {
            const int64_t n = min((int64_t)tile * kRows + row, (int64_t)a.w.N - 1);
            // a row's zeros, 16 groups at a time, the next ones under way: one byte of a row at a time would be a
            // load of 32 sectors, and its wait, for every step
            const uint4* const zeros = reinterpret_cast<const uint4*>(a.w.zeros + n * a.w.ldz);
            auto zeros_at = [&](int block) { return a.w.zeros && block * 16 < a.w.K / GK ? ld_global(zeros + block) : make_uint4(0, 0, 0, 0); };
            int z_block = j0 / 16;
            uint4 z_now = zeros_at(z_block), z_next = zeros_at(z_block + 1);
            auto zero_of = [&](int j) {
                const uint32_t w = j % 16 < 4 ? z_now.x : j % 16 < 8 ? z_now.y : j % 16 < 12 ? z_now.z : z_now.w;
                return zero_pair(w >> (j % 4 * 8));
            };
            for (int s0 = 0; s0 < steps; s0 += kStageK / kStep, cs.next()) {
                wait(&c_full[cs.at], cs.parity);
                const uint32_t at = smem_u32(smem) + cs.at * kStageC + row * 128;
                for (int i = 0; i < kStageK / kStep && s0 + i < steps; ++i, ++r) {
                    if (r % kSets != set) continue;
                    const uint32_t buf = r % kSteps;
                    // 64 bytes of the row: four 16-byte pieces, where the 128-byte swizzle put them
                    uint4 pieces[4];
#pragma unroll
                    for (int h = 0; h < 4; ++h) pieces[h] = ld_u128(at + (((4 * i + h) ^ (row & 7)) << 4));
#pragma unroll
                    for (int h = 0; h < 2; ++h) {           // 64 elements at a time
                        uint32_t z0 = 0x43084308u, z1 = z0;
                        if (a.w.zeros) {                    // a step's groups are of one block of 16
                            const int j = j0 + ((s0 + i) * kStep + 64 * h) / GK;
                            if (j / 16 != z_block) z_block = j / 16, z_now = z_next, z_next = zeros_at(z_block + 1);
                            z0 = zero_of(j), z1 = GK == 32 ? zero_of(j + 1) : z0;
                        }
                        const uint4 p = pieces[2 * h], q = pieces[2 * h + 1];
                        const uint32_t words[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
                        uint32_t v[32];
#pragma unroll
                        for (int w = 0; w < 8; ++w)
#pragma unroll
                            for (int k = 0; k < 4; ++k) v[4 * w + k] = less_zero(words[w] >> (4 * k), w < 4 ? z0 : z1);
                        if (h == 0) {                       // half of the step is ready before its operand is free
                            wait(&used[buf], r / kSteps & 1 ^ 1);
                            tc_fence_after();
                        }
                        __syncwarp();
                        tmem_st32(tmem + lanes + (uint32_t)(kStep / 2) * buf + 32u * h, v);
                    }
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[buf]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&c_empty[cs.at]);
            }
        }
    } else if (warp < kUnpack + kScale) {
        // ---- a group's sums times its scale, and the outputs: a row of the weight and half of x's rows each
        constexpr int kMine = MP / 2;
        const int row = 32 * (warp % 4) + lane, c0 = (warp - kUnpack) / 4 * kMine;
        const uint32_t from = tmem + ((uint32_t)(32 * (warp % 4)) << 16) + G::kColD + c0;
        uint32_t q = 0;
        const int x_block = a.w.K / GK / a.x_blocks;    // groups
        for (int tile = blockIdx.x; tile < cut.tiles; tile += gridDim.x) {
            const int64_t n = (int64_t)tile * kRows + row, n_in = min(n, (int64_t)a.w.N - 1);
            // a row's scales, 16 bytes at a time, the next ones under way: one at a time would be a load of 32
            // sectors, and its wait, for every group (that took twice the time of all the rest)
            const uint4* const scales = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(a.w.scales) + n_in * a.w.lds * (a.w.scale_bf16 ? 2 : 4));
            const int shift = a.w.scale_bf16 ? 3 : 2, per = 1 << shift;     // scales in 16 bytes
            auto scales_at = [&](int block) { return block << shift < a.w.K / GK ? scales[block] : make_uint4(0, 0, 0, 0); };
            uint4 next = scales_at(j0 >> shift);
            float2 acc[kMine / 2] = {};                 // of two columns
            for (int block = j0 >> shift; block << shift < j0 + groups; ++block) {
                const uint4 now = next;
                next = scales_at(block + 1);
                const int to_k = min(j0 + groups - (block << shift), per);
#pragma unroll 1
                for (int k = max(j0 - (block << shift), 0); k < to_k; ++k, ++q) {
                    const int i = a.w.scale_bf16 ? k / 2 : k;               // the same for all threads
                    const uint32_t word = i & 2 ? (i & 1 ? now.w : now.z) : (i & 1 ? now.y : now.x);
                    const float scale = __uint_as_float(!a.w.scale_bf16 ? word : k % 2 ? word & 0xffff0000u : word << 16);
                    const uint32_t buf = q % kD;
                    wait(&d_full[buf], q / kD & 1);
                    tc_fence_after();
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < kMine; c += 16) {
                        float d[16];
                        tmem_ld16(from + MP * buf + c, d);
                        if (c + 16 == kMine) {              // all read: the accumulator is free again
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&d_empty[buf]);
                        }
                        if (a.x_blocks > 1) {
                            const float* xs = a.x_scale + ((block << shift) + k) / x_block;
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (m0 + c0 + c + i < a.M) d[i] *= xs[(int64_t)(m0 + c0 + c + i) * a.x_blocks];
                        }
#pragma unroll
                        for (int i = 0; i < 16; i += 2)
                            acc[(c + i) / 2] = __ffma2_rn(make_float2(d[i], d[i + 1]), make_float2(scale, scale), acc[(c + i) / 2]);
                    }
                }
            }
            if (n < a.w.N) {
                const int rows = min(kMine, a.M - m0 - c0);
                if (a.x_scale && a.x_blocks == 1) {
#pragma unroll
                    for (int i = 0; i < kMine; ++i)
                        if (i < rows) (i % 2 ? acc[i / 2].y : acc[i / 2].x) *= a.x_scale[m0 + c0 + i];
                }
                auto put = [&](auto* to, int64_t stride) {
#pragma unroll
                    for (int i = 0; i < kMine; ++i, to += stride)
                        if (i < rows) *to = from_f32<std::remove_pointer_t<decltype(to)>>(i % 2 ? acc[i / 2].y : acc[i / 2].x);
                };
                if (cut.slices > 1) put(a.parts + ((int64_t)slice * a.M + m0 + c0) * a.w.N + n, a.w.N);
                else if (a.out_bf16) put(reinterpret_cast<__nv_bfloat16*>(a.out) + (int64_t)(m0 + c0) * a.ldo + n, a.ldo);
                else put(reinterpret_cast<float*>(a.out) + (int64_t)(m0 + c0) * a.ldo + n, a.ldo);
            }
        }
    } else if (warp == kUnpack + kScale) {
        // ---- copies of codes.  Here and below the whole warp walks the loop, so that what an instruction wants in
        // uniform registers stays there, and one elected lane issues, nothing more after a wait that expired.  In the end it
        // waits for what it issued last: who reads it has waited for it, but goes on where that wait expired, and the CTA must
        // not end before its copies.
        before_copies();
        Ring cs;
        uint32_t issued = 0;
        const int stages = (steps + kStageK / kStep - 1) / (kStageK / kStep);
        for (int tile = blockIdx.x; tile < cut.tiles; tile += gridDim.x)
            for (int i = 0; i < stages; ++i, cs.next()) {
                wait(&c_empty[cs.at], cs.parity ^ 1);
                if (elect_one() && !wait.dead) {
                    mbar_arrive_expect_tx(&c_full[cs.at], kStageC);
                    tma_load_2d(smem + cs.at * kStageC, &tm_codes, &c_full[cs.at], k0 / 2 + i * (kStageK / 2), tile * kRows);
                    ++issued;
                }
                __syncwarp();
            }
        Waiter last{status};
        for (uint32_t i = issued < kCodeStages ? 0 : issued - kCodeStages; i < issued; ++i) last(&c_full[i % kCodeStages], i / kCodeStages & 1);
    } else if (warp == kUnpack + kScale + 1) {
        // ---- copies of x
        before_copies();
        uint32_t r = 0, issued = 0;
        for (int tile = blockIdx.x; tile < cut.tiles; tile += gridDim.x)
            for (int s = 0; s < steps; ++s, ++r) {
                const uint32_t buf = r % kSteps;
                wait(&used[buf], r / kSteps & 1 ^ 1);
                if (elect_one() && !wait.dead) {
                    mbar_arrive_expect_tx(&full[buf], G::kStageX);
                    for (int h = 0; h < 2; ++h)
                        tma_load_2d(smem + G::kOffX + buf * G::kStageX + h * (G::kStageX / 2), &tm_x, &full[buf], k0 + s * kStep + 64 * h, m0);
                    ++issued;
                }
                __syncwarp();
            }
        Waiter last{status};
        for (uint32_t i = issued < kSteps ? 0 : issued - kSteps; i < issued; ++i) last(&full[i % kSteps], i / kSteps & 1);
    } else {
        // ---- products
        const uint32_t tm = __shfl_sync(~0u, tmem, 0);
        const uint64_t xd = smem_desc_sw128(__shfl_sync(~0u, smem_u32(smem), 0) + G::kOffX);
        uint32_t r = 0, q = 0;
        for (int tile = blockIdx.x; tile < cut.tiles; tile += gridDim.x)
            for (int s = 0; s < steps; ++s, ++r) {
                const uint32_t buf = r % kSteps;
                wait(&full[buf], r / kSteps & 1);
                const uint64_t b = xd + (uint64_t)(buf * (G::kStageX >> 4));
                // the step's groups, each an accumulator's: products of 16 elements, the first of which starts it
                constexpr int kGroups = kStep / GK, kCount = GK / 16;
#pragma unroll
                for (int h = 0; h < kGroups; ++h) {
                    if (kGroups > 1 && s * kGroups + h >= groups) break;
                    wait(&d_empty[q % kD], q / kD & 1 ^ 1);
                    tc_fence_after();
                    if (elect_one() && !wait.dead) {
#pragma unroll
                        for (int k = h * kCount; k < (h + 1) * kCount; ++k)
                            mma_from_tmem(tm + G::kColD + MP * (q % kD), tm + (uint32_t)(kStep / 2) * buf + 8u * k,
                                          b + (uint64_t)(k / 4 * (G::kStageX >> 5) + 2 * (k % 4)), G::kIdesc, k != h * kCount);
                        mma_commit(&d_full[q % kD]);
                    }
                    __syncwarp();
                    ++q;
                }
                if (GK != kStep) {
                    if (elect_one() && !wait.dead) mma_commit(&used[buf]);
                    __syncwarp();
                }
            }
        // the last commits have arrived before the CTA ends; where the loop ended early, one for all that was issued
        for (uint32_t i = r < kSteps ? 0 : r - kSteps; i < r; ++i) wait(&used[i % kSteps], i / kSteps & 1);
        if (__any_sync(~0u, wait.dead)) {
            if (elect_one()) mma_commit(done);
            __syncwarp();
            Waiter last{status};
            last(done, 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kUnpack + kScale) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// x as bf16, every eight elements in the order 0 4 1 5 2 6 3 7 in which a word's codes come out; rows from M on are 0.
__global__ void __launch_bounds__(256) k_w4_order(const W4LinearArgs a, uint4* to, int64_t vecs) {
    after_previous();
    next_may_start();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= vecs) return;
    const int per_row = a.w.K / 8, m = (int)(i / per_row), k = (int)(i % per_row) * 8;
    uint32_t r[4] = {};
    if (m < a.M) {
        if (a.x_i8) x_pairs(*reinterpret_cast<const uint2*>(reinterpret_cast<const int8_t*>(a.x) + m * a.ldx + k), r);
        else x_pairs(*reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.x) + m * a.ldx + k), r);
    }
    to[i] = make_uint4(r[0], r[1], r[2], r[3]);
}

bool encode(CUtensorMap* m, CUtensorMapDataType type, int size, const void* base, uint64_t inner, uint64_t rows, uint64_t stride,
            uint32_t box_inner, uint32_t box_rows) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {inner, rows}, strides[1] = {stride * size};
    cuuint32_t box[2] = {box_inner, box_rows}, one[2] = {1, 1};
    return enc(m, type, 2, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kSms = 152;

int rows_of(int M) { return M <= 32 ? 32 : 64; }

// Slices of the rows where the tiles alone leave SMs idle, by the CTA with most work, and for the second kernel two
// microseconds and the slices' sums at 4 TB/s.  A step takes 0.35 us with groups of 128, which is 24 bytes of codes a
// nanosecond, more with the two or four accumulators of groups of 64 or 32: 20, 12.  64 x 4096 -> 8192, groups of 128:
// one slice 19.4 us, two 16.  Counted at 24, groups of 32 and 64 had one slice for 128 x 2048 -> 2048: 20.8 and 13.3 us,
// now 11.1 and 9.4; 20 x 5120 -> 13824 in groups of 32 40.9, now 36.3; 48 other sizes measured the same.
Cut cut_of(int M, const W4Weight& w) {
    Cut best{};
    int64_t least = 0;
    const int stages = (w.K + kStageK - 1) / kStageK, rate = w.group == 32 ? 12 : w.group == 64 ? 20 : 24;
    for (int s = 1; s <= 32 && s <= stages; ++s) {
        Cut c;
        c.tiles = (w.N + kRows - 1) / kRows;
        c.m_blocks = (M + rows_of(M) - 1) / rows_of(M);
        c.slice_k = (stages + s - 1) / s * kStageK;
        c.slices = (w.K + c.slice_k - 1) / c.slice_k;
        int walkers = kSms / (c.m_blocks * c.slices);
        walkers = walkers < 1 ? 1 : walkers > c.tiles ? c.tiles : walkers;
        const int64_t bytes = (int64_t)((c.tiles + walkers - 1) / walkers) * c.slice_k * (kRows / 2);
        const int64_t ns = bytes / rate + (c.slices > 1 ? 2000 + (int64_t)c.slices * M * w.N * 8 / 4000 : 0);
        if (s == 1 || ns < least) best = c, least = ns;
    }
    return best;
}

int64_t padded(int M) { return (int64_t)(M + rows_of(M) - 1) / rows_of(M) * rows_of(M); }

template <int MP, int GK>
int launch(const W4LinearArgs& a, unsigned int* status, cudaStream_t stream, const char** why) {
    using G = Geo<MP>;
    const Cut cut = cut_of(a.M, a.w);
    uint4* const x = reinterpret_cast<uint4*>(a.parts);         // x in its order, then the slices' sums
    W4LinearArgs b = a;
    b.parts = reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(a.parts) + padded(a.M) * a.w.K * 2);
    CUtensorMap mc, mx;
    if (!encode(&mc, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.w.codes, a.w.K / 2, a.w.N, a.w.ldc, kStageK / 2, kRows) ||
        !encode(&mx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x, a.w.K, padded(a.M), a.w.K, kStep / 2, MP)) {
        *why = "cuTensorMapEncodeTiled failed (driver entry point missing or layout rejected)";
        return -1;
    }
    auto kern = k_w4_tiles<MP, GK>;
    static ContextMemo attr_memo;
    if (!opt_in_dynamic_smem(attr_memo, kern, G::kSmem, why)) return -1;
    const int64_t vecs = padded(a.M) * a.w.K / 8;
    if (launch_in_turn(k_w4_order, dim3((unsigned)((vecs + 255) / 256)), 256, 0, 1, stream, why, a, x, vecs)) return -1;
    int walkers = kSms / (cut.m_blocks * cut.slices);
    walkers = walkers < 1 ? 1 : walkers > cut.tiles ? cut.tiles : walkers;
    if (launch_in_turn(kern, dim3((unsigned)walkers, (unsigned)cut.m_blocks, (unsigned)cut.slices), kThreads, G::kSmem, 1, stream, why, mc, mx,
                       b, cut, status))
        return -1;
    return cut.slices > 1 ? launch_w4_join(b, cut.slices, stream, why) : 0;
}

}  // namespace

size_t w4_tiles_workspace(int M, const W4Weight& w) {
    const Cut c = cut_of(M, w);
    return (size_t)padded(M) * w.K * 2 + (c.slices > 1 ? (size_t)c.slices * M * w.N * sizeof(float) : 0);
}

int launch_w4_tiles(const W4LinearArgs& a, unsigned int* status, cudaStream_t stream, const char** why) {
    const bool few = rows_of(a.M) == 32;
    if (a.w.group == 32) return few ? launch<32, 32>(a, status, stream, why) : launch<64, 32>(a, status, stream, why);
    if (a.w.group == 64) return few ? launch<32, 64>(a, status, stream, why) : launch<64, 64>(a, status, stream, why);
    return few ? launch<32, 128>(a, status, stream, why) : launch<64, 128>(a, status, stream, why);
}

}  // namespace ssm
