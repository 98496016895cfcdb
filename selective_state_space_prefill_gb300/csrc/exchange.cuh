// exchange.cuh -- what the CTAs of a thread-block cluster tell each other (spec.cu).
#pragma once

#include <cooperative_groups.h>

#include "common.cuh"
#include "ssm.h"

namespace ssm {

// What the warps of a row's CTAs tell each other, at most twice: each writes its words into the shared memory of every
// CTA of the cluster, in 64 bits of which the upper half is the word and the lower half says that it is there, and
// reads the others' from its own.  A word and its mark come as one, so nothing has to be ordered, and nobody waits
// for anything but the words.  (A barrier of the cluster, and reads from the others behind it, waits for all that the
// SM has under way, two microseconds where four CTAs of it write: 512 x 131072 95 us so, 86 with words; 64 x 32000 7.5
// and 5.0.  Words of every warp instead of every CTA, polled by all: 107, 6.7.)
//
// Who may leave: the two exchanges have slots of their own, and a CTA that has all words of the last one is written to by
// nobody.  A wait that expires says nothing of the sender, who may have been held up and write later (the limit is one
// of time).  So a warp that gave up (`dead`, the same in all its lanes after settle()) sends no more, as those who have
// what they need may be gone, and leave() keeps its CTA until all other threads of the cluster have left or given up
// too: all their waits are bounded.
constexpr int kMostCtas = 8;
template <int kWords, int kWarps> struct Exchange {
    struct Box {                                        // in shared memory
        uint64_t slot[2][kWords][kMostCtas * kWarps];
    };
    Box& box;
    int ctas, rank;
    unsigned int* status;
    uint64_t limit_ns;
    int turn = 0;
    bool dead = false;

    // By all threads; ready() before the first words are sent.
    __device__ __forceinline__ Exchange(Box& box, int ctas, int rank, unsigned int* status, uint64_t limit_ns = 2000000000ull)
        : box(box), ctas(ctas), rank(rank), status(status), limit_ns(limit_ns) {
        for (int i = threadIdx.x; i < 2 * kWords * kMostCtas * kWarps; i += blockDim.x) (&box.slot[0][0][0])[i] = 0;
        if (ctas > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    }
    __device__ __forceinline__ void ready() {
        if (ctas > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
        else __syncthreads();
    }
    // A warp's words (the CTA's where kWarps is 1), the same in all lanes.
    __device__ __forceinline__ void send(const uint32_t (&words)[kWords]) {
        const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
        if (lane < ctas && warp < kWarps && !dead) {
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
                uint64_t* to = &box.slot[turn][w][rank * kWarps + warp];
                if (ctas > 1) to = cooperative_groups::this_cluster().map_shared_rank(to, lane);
                *reinterpret_cast<volatile uint64_t*>(to) = (uint64_t)words[w] << 32 | 1u;
            }
        }
        ++turn;
    }
    // A word of the last exchange by warp and CTA; gives up after two seconds, like all waits here.
    __device__ __forceinline__ uint32_t word(int w, int from) {
        const volatile uint64_t* at = &box.slot[turn - 1][w][from];
        uint64_t v = *at, t0 = 0;
        for (uint32_t spin = 0; v == 0 && !dead; ++spin) {
            if ((spin & 4095u) == 4095u) {
                const uint64_t now = globaltimer_ns();
                if (t0 == 0) t0 = now;
                if (now - t0 > limit_ns) {
                    dead = true;
                    atomicOr(status, (unsigned)SSM_DEV_WAIT_TIMEOUT);
                }
            }
            v = *at;
        }
        return (uint32_t)(v >> 32);
    }
    // By all lanes, once they have their words: what one of them gave up, the warp gives up.
    __device__ __forceinline__ void settle() { dead = __any_sync(~0u, dead); }
    // The last thing that a thread does.
    __device__ __forceinline__ void leave() {
        if (dead && ctas > 1) asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    }
};

}  // namespace ssm
