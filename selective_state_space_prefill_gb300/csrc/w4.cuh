// w4.cuh -- what the two kernels of w4_linear share: x in the order in which codes come out of a word, bounded
// waits, outputs.
#pragma once

#include "common.cuh"
#include "kernels.h"
#include "ssm.h"

namespace ssm {

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float i8_at(uint32_t w, int i) { return (float)(int8_t)(w >> (8 * i)); }

// Eight consecutive elements of x as the pairs (0, 4), (1, 5), (2, 6), (3, 7), as the codes come out of a word.
__device__ __forceinline__ void x_pairs(uint4 q, uint32_t (&r)[4]) {
    r[0] = __byte_perm(q.x, q.z, 0x5410), r[1] = __byte_perm(q.x, q.z, 0x7632);
    r[2] = __byte_perm(q.y, q.w, 0x5410), r[3] = __byte_perm(q.y, q.w, 0x7632);
}
__device__ __forceinline__ void x_pairs(uint2 q, uint32_t (&r)[4]) {    // whole numbers up to 128: exact in bf16
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = bf16_pair(i8_at(q.x, i), i8_at(q.y, i));
}
// Waits that give up after two seconds, report it and are not waited for again: every loop still ends.  The timer
// takes longer to read than most waits, so it is not looked at before 4096 tries.
struct Waiter {
    unsigned int* status;
    uint64_t limit_ns = 2000000000ull;
    bool dead = false;
    __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
        if (dead) return;
        uint64_t t0 = 0;
        for (uint32_t spin = 0; !mbar_try_wait(bar, parity); ++spin)
            if ((spin & 4095u) == 4095u) {
                const uint64_t now = globaltimer_ns();
                if (t0 == 0) t0 = now;
                if (now - t0 > limit_ns) {
                    dead = true;
                    atomicOr(status, (unsigned)SSM_DEV_WAIT_TIMEOUT);
                    return;
                }
            }
    }
};

__device__ __forceinline__ void w4_store(const W4LinearArgs& a, int m, int64_t n, float v) {
    if (a.out_bf16) reinterpret_cast<__nv_bfloat16*>(a.out)[(int64_t)m * a.ldo + n] = __float2bfloat16_rn(v);
    else reinterpret_cast<float*>(a.out)[(int64_t)m * a.ldo + n] = v;
}

// The slices' sums of every output, added up by a kernel that is launched while they still come (w4.cu).
int launch_w4_join(const W4LinearArgs& a, int slices, cudaStream_t stream, const char** why);
// More rows of x than k_w4_linear is for (w4_tiles.cu); its workspace holds x as well.
size_t w4_tiles_workspace(int M, const W4Weight& w);
int launch_w4_tiles(const W4LinearArgs& a, unsigned int* status, cudaStream_t stream, const char** why);

}  // namespace ssm
