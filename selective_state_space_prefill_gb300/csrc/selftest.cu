// selftest.cu -- diagnostic kernels that let a caller watch the library's bounded waits
// fail safely: each waits for what nobody does, through the same bounded wait that the
// library's kernels use, and reports the expiry in the device status word
// (SSM_DEV_WAIT_TIMEOUT) before returning normally.  No trap, no fault, no unbounded spin.
#include "common.cuh"
#include "exchange.cuh"
#include "kernels.h"
#include "w4.cuh"

namespace ssm {
namespace {

__global__ void k_expire_wait(unsigned int* status, uint64_t limit_ns) {
    __shared__ __align__(8) uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);                 // one arrival expected; none ever comes
        fence_barrier_init();
    }
    __syncthreads();
    if (threadIdx.x == 0 && !mbar_wait_bounded(&bar, 0u, limit_ns)) atomicOr(status, 1u);
}

// The waits of the 4-bit projections: the second one is not waited for.
__global__ void k_expire_waiter(unsigned int* status, uint64_t limit_ns) {
    __shared__ __align__(8) uint64_t bar;
    after_previous();
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_barrier_init();
    }
    __syncthreads();
    Waiter wait{status, limit_ns};
    wait(&bar, 0);
    wait(&bar, 0);
}

// The exchange between the CTAs of a cluster: each waits for a word of the other that is never sent, and stays until
// both have given up.
__global__ void k_expire_exchange(unsigned int* status, uint64_t limit_ns, int ctas) {
    __shared__ Exchange<1, 1>::Box box;
    Exchange<1, 1> all(box, ctas, blockIdx.x % (unsigned)ctas, status, limit_ns);
    after_previous();
    all.ready();
    ++all.turn;
    all.word(0, (all.rank + 1) % ctas);
    all.settle();
    all.leave();
}

}  // namespace

int launch_expire_wait(int which, unsigned int* status, uint64_t limit_ns, cudaStream_t stream, const char** why) {
    if (which == 1) return launch_in_turn(k_expire_waiter, dim3(1), 32, 0, 1, stream, why, status, limit_ns);
    if (which == 2) return launch_in_turn(k_expire_exchange, dim3(2), 64, 0, 2, stream, why, status, limit_ns, 2);
    k_expire_wait<<<1, 32, 0, stream>>>(status, limit_ns);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        *why = cudaGetErrorString(e);
        return -1;
    }
    return 0;
}

}  // namespace ssm
