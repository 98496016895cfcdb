// norm.cu -- norm_rms: residual addition and root-mean-square norm over groups of a row's channels, with an
// output in bf16, fp32, or int8 with a scale per row and group.
//
// A first form: one CTA per row and group, the fp32 sum r in shared memory between its three uses (mean of
// squares, maximum, output).
#include "common.cuh"
#include "kernels.h"
#include "ssm.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void load8(const void* p, int64_t at, bool bf16, float* v) {
    if (bf16) {
        const uint4 q = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p) + at);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
        const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + at);
        const float4 a = q[0], b = q[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(void* p, int64_t at, bool bf16, const float* v) {
    if (bf16) {
        *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p) + at) =
            make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
    } else {
        float4* q = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + at);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}
// round_half_even(y * inv) within [-127, 127]; a NaN gives 0
__device__ __forceinline__ uint32_t code(float y, float inv) {
    const float c = y * inv;
    return c == c ? (uint32_t)__float2int_rn(fminf(fmaxf(c, -127.f), 127.f)) & 0xffu : 0u;
}

template <bool kMax>
__device__ float across(float v, float* s) {
    for (int o = 16; o > 0; o >>= 1) {
        const float w = __shfl_xor_sync(~0u, v, o);
        v = kMax ? fmaxf(v, w) : v + w;
    }
    __syncthreads();
    if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = v;
    __syncthreads();
    v = s[0];
    for (int i = 1; i < kThreads / 32; ++i) v = kMax ? fmaxf(v, s[i]) : v + s[i];
    return v;
}

__global__ void __launch_bounds__(kThreads) k_norm_rms(const NormArgs a) {
    extern __shared__ float s_r[];
    __shared__ float s_part[kThreads / 32];
    const int64_t row = blockIdx.x / a.n_groups;
    const int group = blockIdx.x % a.n_groups, n = a.width / a.n_groups, c0 = group * n;
    float sum = 0.f;
    for (int c = 8 * threadIdx.x; c < n; c += 8 * kThreads) {
        float v[8], w[8];
        load8(a.x, row * a.x_st + c0 + c, a.in_type == SSM_BF16, v);
        if (a.residual) {
            load8(a.residual, row * a.res_st + c0 + c, a.res_type == SSM_BF16, w);
            for (int i = 0; i < 8; ++i) v[i] += w[i];
            if (a.residual_out) store8(a.residual_out, row * a.ro_st + c0 + c, a.res_type == SSM_BF16, v);
        }
        for (int i = 0; i < 8; ++i) sum = fmaf(v[i], v[i], sum), s_r[c + i] = v[i];
    }
    const float f = rsqrtf(across<false>(sum, s_part) / n + a.eps);
    float amax = 0.f;
    if (a.out_type == SSM_I8) {
        for (int c = 8 * threadIdx.x; c < n; c += 8 * kThreads)
            for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(s_r[c + i] * f * (a.weight ? a.weight[c0 + c + i] : 1.f)));
        amax = across<true>(amax, s_part);
        if (threadIdx.x == 0) a.out_scale[row * a.n_groups + group] = __fdiv_rn(amax, 127.f);
    }
    const float inv = amax > 0.f ? __fdiv_rn(127.f, amax) : 0.f;
    for (int c = 8 * threadIdx.x; c < n; c += 8 * kThreads) {
        float y[8];
        for (int i = 0; i < 8; ++i) y[i] = s_r[c + i] * f * (a.weight ? a.weight[c0 + c + i] : 1.f);
        if (a.out_type == SSM_I8) {
            uint32_t q[2] = {0, 0};
            for (int i = 0; i < 8; ++i) q[i / 4] |= code(y[i], inv) << (8 * (i % 4));
            *reinterpret_cast<uint2*>(reinterpret_cast<int8_t*>(a.out) + row * a.out_st + c0 + c) = make_uint2(q[0], q[1]);
        } else {
            store8(a.out, row * a.out_st + c0 + c, a.out_type == SSM_BF16, y);
        }
    }
}

}  // namespace

int launch_norm_rms(const NormArgs& a, cudaStream_t stream, const char** why) {
    static ContextMemo attr_memo;
    if (!opt_in_dynamic_smem(attr_memo, k_norm_rms, 32768 * 4, why)) return -1;
    k_norm_rms<<<(unsigned)(a.n_rows * a.n_groups), kThreads, a.width / a.n_groups * 4, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return 0;
    *why = cudaGetErrorString(e);
    return -1;
}

}  // namespace ssm
