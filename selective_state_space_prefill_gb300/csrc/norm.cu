// norm.cu -- norm_rms: residual addition and root-mean-square norm over groups of a row's channels, with an
// output in bf16, fp32, or int8 with a scale per row and group.
//
// Bytes in and out over the copy rate are the floor.  A row's group stays in registers between its uses (mean of
// squares, maximum, output), so that everything is read and written once: a thread holds up to V vectors of eight
// channels, all loads in flight before the first is used.  Small groups are a warp's, several to a CTA, without a
// barrier; larger ones a CTA's of 64 .. 1024 threads, with as few vectors a thread as that allows for few rows
// (latency) and four for many (loads in flight, fewer threads at the barriers).  Measured: 8192 x 5120 fp32 in 8
// groups to bf16 38 us (6.6 TB/s, 0.97 of the copy rate), 16384 x 7168 with an fp32 residual 201 us (7.0 TB/s);
// one row of 1536 1.6 us in a graph, which is a launch and a load.
#include "common.cuh"
#include "kernels.h"
#include "ssm.h"

namespace ssm {
namespace {

constexpr int kSms = 152;

// Eight channels.
template <typename T> struct Vec;
template <> struct Vec<__nv_bfloat16> {
    uint4 q;
    __device__ __forceinline__ void load(const void* p, int64_t at) {
        q = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p) + at);
    }
    __device__ __forceinline__ void get(float* v) const {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
};
template <> struct Vec<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const void* p, int64_t at) {
        const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + at);
        a = q[0], b = q[1];
    }
    __device__ __forceinline__ void get(float* v) const {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
};
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float* v) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
// round_half_even(y * inv) within [-127, 127]; a NaN gives 0
__device__ __forceinline__ uint32_t code(float y, float inv) {
    const float c = y * inv;
    return c == c ? (uint32_t)__float2int_rn(fminf(fmaxf(c, -127.f), 127.f)) & 0xffu : 0u;
}

// The sum or maximum over a group's threads: a warp, or a CTA of W warps.
template <int W, bool kMax>
__device__ __forceinline__ float across(float v, float* s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float w = __shfl_xor_sync(~0u, v, o);
        v = kMax ? fmaxf(v, w) : v + w;
    }
    if (W == 1) return v;
    if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = v;
    __syncthreads();
    const int lane = threadIdx.x % 32;
    v = lane < W ? s[lane] : 0.f;                       // a sum of squares and a maximum of magnitudes start at 0
#pragma unroll
    for (int o = W > 16 ? 16 : W > 8 ? 8 : W > 4 ? 4 : W > 2 ? 2 : 1; o > 0; o >>= 1) {
        const float w = __shfl_xor_sync(~0u, v, o);
        v = kMax ? fmaxf(v, w) : v + w;
    }
    return __shfl_sync(~0u, v, 0);
}

// The mean of squares (with eps) of a group whose squares leave fp32's range, from its r (a thread's `count` in t, which
// come back scaled) times a power of two that brings the larger of r and the root of eps near 1.  Groups of zeros
// without eps and infinities keep the mean they have.  A call, with r in local memory, as it is hardly ever made: inlined it
// took registers from every form, 16384 x 7168 fp32 101 us -> 109.
template <int W>
__device__ __noinline__ float mean_again(float* t, int count, int n, float eps, float mean, float* s_max, float* s_sum) {
    float most = 0.f;
#pragma unroll 1
    for (int i = 0; i < count; ++i) most = fmaxf(most, fabsf(t[i]));
    most = fmaxf(across<W, true>(most, s_max), sqrtf(eps));
    if (most > 0.f && most < INFINITY) {
        const float by = __int_as_float((254 - min(__float_as_int(most) >> 23, 253)) << 23);    // 2^127 .. 2^-126
        float sum = 0.f;
#pragma unroll 1
        for (int i = 0; i < count; ++i) t[i] *= by, sum = fmaf(t[i], t[i], sum);
        mean = across<W, false>(sum, s_sum) / n + eps * by * by;
    }
    if (W > 1) __syncthreads();                         // the maximum's place is used again
    return mean;
}

// Blocks an SM that the registers of a form with int8 out are kept to (0: the compiler's choice, which would be one less):
// 64 a thread, or 80 for fp32 x and residual and, up to 8192 channels, for an fp32 residual of bf16 x (4096 x 8192 60 us,
// with 64 and spills 65; with fp32 x alone 64 are right: 16384 x 7168 105 us, with more 116).
template <typename Tx, typename Tr, typename To, int W, int V>
constexpr int blocks_per_sm() {
    if (V == 1 || sizeof(To) != 1 || W == 32) return 0;
    return (sizeof(Tr) == 4 && (sizeof(Tx) == 4 || W <= 8) ? 768 : 1024) / (W == 1 ? 128 : 32 * W);
}

// W warps for a group (1: four groups to a CTA), V vectors a thread.
template <typename Tx, typename Tr, typename To, int W, int V>
__global__ void __launch_bounds__(W == 1 ? 128 : 32 * W, blocks_per_sm<Tx, Tr, To, W, V>()) k_norm_rms(const NormArgs a) {
    constexpr bool kI8 = sizeof(To) == 1;
    constexpr int kStep = 8 * 32 * W;                   // channels of a group between a thread's vectors
    __shared__ float s_sum[W], s_max[W];
    const int n = a.width / a.n_groups, tid = W == 1 ? threadIdx.x % 32 : threadIdx.x;
    const unsigned unit = W == 1 ? blockIdx.x * 4 + threadIdx.x / 32 : blockIdx.x;
    const unsigned row = unit / (unsigned)a.n_groups, group = unit - row * (unsigned)a.n_groups;
    if (W == 1 && row >= a.n_rows) return;
    const int c0 = group * n, first = 8 * tid;
    after_previous();
    next_may_start();
    Vec<Tx> x[V];
    Vec<Tr> r[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (first + i * kStep < n) {
            x[i].load(a.x, row * a.x_st + c0 + first + i * kStep);
            if (a.residual) r[i].load(a.residual, row * a.res_st + c0 + first + i * kStep);
        }
    float v[V][8], sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (first + i * kStep < n) {
            x[i].get(v[i]);
            if (a.residual) {
                float w[8];
                r[i].get(w);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[i][k] += w[k];
                if (a.residual_out) store8(reinterpret_cast<Tr*>(a.residual_out) + row * a.ro_st + c0 + first + i * kStep, v[i]);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) sum = fmaf(v[i][k], v[i][k], sum);
        }
    float mean = across<W, false>(sum, s_sum) / n + a.eps;
    // Squares lose places below 2^-126, are gone below 2^-149, and pass fp32's range: a mean below 2^-100 (at which what is
    // lost is 2^-49 of it) or infinite is taken again.  All threads of a group agree on that.
    if (!(mean >= 0x1p-100f && mean < INFINITY) && mean == mean) {
        float t[V * 8];
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) t[i * 8 + k] = first + i * kStep < n ? v[i][k] : 0.f;
        mean = mean_again<W>(t, V * 8, n, a.eps, mean, s_max, s_sum);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) v[i][k] = t[i * 8 + k];
    }
    const float f = rsqrtf(mean);
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (first + i * kStep < n) {
            float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
            if (a.weight) {
                Vec<float> q;
                q.load(a.weight, c0 + first + i * kStep);
                q.get(w);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[i][k] = v[i][k] * f * w[k];
                if (kI8) amax = fmaxf(amax, fabsf(v[i][k]));
            }
            if constexpr (!kI8) store8(reinterpret_cast<To*>(a.out) + row * a.out_st + c0 + first + i * kStep, v[i]);
        }
    if constexpr (kI8) {
        amax = across<W, true>(amax, s_max);
        if (tid == 0) a.out_scale[(int64_t)row * a.n_groups + group] = __fdiv_rn(amax, 127.f);
        const float inv = amax > 0.f ? __fdiv_rn(127.f, amax) : 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (first + i * kStep < n) {
                uint32_t q[2] = {0, 0};
#pragma unroll
                for (int k = 0; k < 8; ++k) q[k / 4] |= code(v[i][k], inv) << (8 * (k % 4));
                *reinterpret_cast<uint2*>(reinterpret_cast<int8_t*>(a.out) + row * a.out_st + c0 + first + i * kStep) = make_uint2(q[0], q[1]);
            }
    }
}

template <typename Tx, typename Tr, typename To, int W, int V>
int go(const NormArgs& a, cudaStream_t stream, const char** why) {
    const int64_t units = a.n_rows * a.n_groups;
    return launch_in_turn(k_norm_rms<Tx, Tr, To, W, V>, dim3((unsigned)(W == 1 ? (units + 3) / 4 : units)), W == 1 ? 128 : 32 * W, 0, 1,
                          stream, why, a);
}

template <typename Tx, typename Tr, typename To>
int launch(const NormArgs& a, cudaStream_t stream, const char** why) {
    const int vecs = a.width / a.n_groups / 8;
    const bool few = a.n_rows * a.n_groups <= 2 * kSms;
    if (vecs <= 32) return go<Tx, Tr, To, 1, 1>(a, stream, why);
    if (vecs <= 128 && !few) return go<Tx, Tr, To, 1, 4>(a, stream, why);
    if (few) {                                          // a vector a thread, as far as 1024 threads go
        if (vecs <= 64) return go<Tx, Tr, To, 2, 1>(a, stream, why);
        if (vecs <= 128) return go<Tx, Tr, To, 4, 1>(a, stream, why);
        if (vecs <= 256) return go<Tx, Tr, To, 8, 1>(a, stream, why);
        if (vecs <= 512) return go<Tx, Tr, To, 16, 1>(a, stream, why);
        if (vecs <= 1024) return go<Tx, Tr, To, 32, 1>(a, stream, why);
    } else {
        if (vecs <= 256) return go<Tx, Tr, To, 2, 4>(a, stream, why);
        if (vecs <= 512) return go<Tx, Tr, To, 4, 4>(a, stream, why);
        if (vecs <= 1024) return go<Tx, Tr, To, 8, 4>(a, stream, why);
    }
    if (vecs <= 2048) return go<Tx, Tr, To, 16, 4>(a, stream, why);
    return go<Tx, Tr, To, 32, 4>(a, stream, why);
}

template <typename Tx, typename Tr>
int launch_out(const NormArgs& a, cudaStream_t stream, const char** why) {
    if (a.out_type == SSM_I8) return launch<Tx, Tr, int8_t>(a, stream, why);
    if (a.out_type == SSM_BF16) return launch<Tx, Tr, __nv_bfloat16>(a, stream, why);
    return launch<Tx, Tr, float>(a, stream, why);
}

}  // namespace

int launch_norm_rms(const NormArgs& a, cudaStream_t stream, const char** why) {
    if (a.in_type == SSM_BF16)
        return a.res_type == SSM_BF16 ? launch_out<__nv_bfloat16, __nv_bfloat16>(a, stream, why) : launch_out<__nv_bfloat16, float>(a, stream, why);
    return a.res_type == SSM_BF16 ? launch_out<float, __nv_bfloat16>(a, stream, why) : launch_out<float, float>(a, stream, why);
}

}  // namespace ssm
