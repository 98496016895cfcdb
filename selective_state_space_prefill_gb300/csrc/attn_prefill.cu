// attn_prefill.cu -- causal attention over packed prompts with grouped heads (sm_103a).
//
// Row i of a sequence with Lq queries and Lk keys sees the keys j <= i + Lk - Lq.  One pass over
// them carries the running maximum m and sum l of the softmax:
//   m' = max(m, s_j); l = l e^(m-m') + e^(s_j-m'); o = o e^(m-m') + e^(s_j-m') v_j
// and out = o / l, lse = m + ln l.
//
// A warp owns one (row, head) and its lanes the head's dimensions, so each key costs a warp sum.
#include "common.cuh"
#include "kernels.h"

namespace ssm {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float4 load4(const void* base, int64_t at, bool on) {
    if (!on) return make_float4(0.f, 0.f, 0.f, 0.f);
    const uint2 w = *reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(base) + at);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}

template <typename Tout>
__global__ void __launch_bounds__(kThreads)
k_attn_prefill(const AttnPrefillArgs a) {
    const int b = blockIdx.z, h = blockIdx.y, lane = threadIdx.x & 31;
    const int i = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t q0 = a.cu_q[b], k0 = a.cu_k[b];
    const int64_t lq = min((int64_t)a.cu_q[b + 1], a.total_q) - q0, lk = min((int64_t)a.cu_k[b + 1], a.total_k) - k0;
    if (i >= lq || i >= a.max_q || q0 < 0 || k0 < 0) return;
    const int d = 4 * lane, hk = h / (a.n_q / a.n_kv);
    const bool on = d < a.dim;
    float4 q = load4(a.q, (q0 + i) * a.q_st + h * a.q_sh + d, on);
    const float s2 = a.scale * kLog2e;
    const int64_t see = min(lk, i + lk - lq + 1);
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int64_t j = 0; j < see; ++j) {
        const float4 k = load4(a.k, (k0 + j) * a.k_st + hk * a.k_sh + d, on);
        const float4 v = load4(a.v, (k0 + j) * a.v_st + hk * a.v_sh + d, on);
        float s = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        s *= s2;                                     // in units of log 2
        const float m2 = fmaxf(m, s), r = ex2(m - m2), p = ex2(s - m2);
        m = m2;
        l = l * r + p;
        o.x = o.x * r + p * v.x;
        o.y = o.y * r + p * v.y;
        o.z = o.z * r + p * v.z;
        o.w = o.w * r + p * v.w;
    }
    const float inv = see > 0 ? 1.f / l : 0.f;
    if (on) {
        Tout* out = reinterpret_cast<Tout*>(a.out) + (q0 + i) * a.o_st + h * a.o_sh + d;
        out[0] = from_f32<Tout>(o.x * inv);
        out[1] = from_f32<Tout>(o.y * inv);
        out[2] = from_f32<Tout>(o.z * inv);
        out[3] = from_f32<Tout>(o.w * inv);
    }
    if (a.lse && lane == 0) a.lse[(q0 + i) * a.n_q + h] = see > 0 ? m * kLn2 + logf(l) : -INFINITY;
}

}  // namespace

int launch_attn_prefill(const AttnPrefillArgs& a, bool out_bf16, cudaStream_t stream, const char** why) {
    const dim3 grid((unsigned)((a.max_q + 3) / 4), (unsigned)a.n_q, (unsigned)a.batch);
    if (out_bf16) k_attn_prefill<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(a);
    else k_attn_prefill<float><<<grid, kThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return 0;
    *why = cudaGetErrorString(e);
    return -1;
}

}  // namespace ssm
