// attn_decode.cu -- one query token per request over the paged, possibly int8, cache (sm_103a).
//
// The softmax runs in one pass with a running maximum and sum; an int8 row's scale multiplies its
// score (keys) or its weight (values).  A block owns one (request, query head); its warps take
// every fourth key and join their maxima, sums and outputs at the end.
#include "common.cuh"
#include "kernels.h"

namespace ssm {
namespace {

constexpr int kWarps = 4;
constexpr unsigned kBadIndex = 8u;      // SSM_DEV_BAD_INDEX

template <bool I8>
__device__ __forceinline__ float4 row4(const void* base, const float* scale, int64_t row, int dim, int d, bool on) {
    if (!on) return make_float4(0.f, 0.f, 0.f, 0.f);
    if constexpr (I8) {
        const char4 c = *reinterpret_cast<const char4*>(reinterpret_cast<const int8_t*>(base) + row * dim + d);
        const float s = scale[row];
        return make_float4(c.x * s, c.y * s, c.z * s, c.w * s);
    } else {
        const uint2 w = *reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(base) + row * dim + d);
        return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                           __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
    }
}

template <bool I8, typename Tout>
__global__ void __launch_bounds__(kWarps * 32)
k_attn_decode(const AttnDecodeArgs a) {
    __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][128];
    const int h = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int hk = h / (a.n_q / a.c.n_kv), d = 4 * lane;
    const bool on = d < a.c.dim;
    const int64_t most = min((int64_t)a.max_len, (int64_t)a.n_table * a.c.page_size);
    int64_t len = a.lens[b];
    if (len < 0 || len > most) {
        if (threadIdx.x == 0) atomicOr(a.status, kBadIndex);
        len = len < 0 ? 0 : most;
    }
    const __nv_bfloat16* qp = reinterpret_cast<const __nv_bfloat16*>(a.q) + b * a.q_st + h * a.q_sh + d;
    float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on) q = make_float4(to_f32(qp[0]), to_f32(qp[1]), to_f32(qp[2]), to_f32(qp[3]));
    const float s2 = a.scale * kLog2e;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int64_t j = warp; j < len; j += kWarps) {
        const int page = a.page_table[b * a.table_stride + j / a.c.page_size];
        if (page < 0 || page >= a.c.n_pages) {
            if (lane == 0) atomicOr(a.status, kBadIndex);
            continue;
        }
        const int64_t row = ((int64_t)page * a.c.n_kv + hk) * a.c.page_size + j % a.c.page_size;
        const float4 k = row4<I8>(a.c.k, a.c.k_scale, row, a.c.dim, d, on);
        const float4 v = row4<I8>(a.c.v, a.c.v_scale, row, a.c.dim, d, on);
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
    if (lane == 0) s_m[warp] = m, s_l[warp] = l;
    *reinterpret_cast<float4*>(&s_o[warp][d]) = o;
    __syncthreads();
    m = -INFINITY;
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_m[w]);
    l = 0.f;
    float acc = 0.f;
    for (int w = 0; w < kWarps; ++w) {
        const float f = s_m[w] == -INFINITY ? 0.f : ex2(s_m[w] - m);
        l += f * s_l[w];
        acc += f * s_o[w][threadIdx.x];
    }
    if (threadIdx.x < a.c.dim)
        reinterpret_cast<Tout*>(a.out)[b * a.o_st + h * a.o_sh + threadIdx.x] = from_f32<Tout>(l > 0.f ? acc / l : 0.f);
    if (a.lse && threadIdx.x == 0) a.lse[(int64_t)b * a.n_q + h] = l > 0.f ? m * kLn2 + logf(l) : -INFINITY;
}

}  // namespace

size_t attn_decode_workspace(int, int, int, int, int) { return 0; }

int launch_attn_decode(const AttnDecodeArgs& a, bool cache_i8, bool out_bf16, cudaStream_t stream, const char** why) {
    const dim3 grid((unsigned)a.n_q, (unsigned)a.batch);
    if (cache_i8) {
        if (out_bf16) k_attn_decode<true, __nv_bfloat16><<<grid, kWarps * 32, 0, stream>>>(a);
        else k_attn_decode<true, float><<<grid, kWarps * 32, 0, stream>>>(a);
    } else {
        if (out_bf16) k_attn_decode<false, __nv_bfloat16><<<grid, kWarps * 32, 0, stream>>>(a);
        else k_attn_decode<false, float><<<grid, kWarps * 32, 0, stream>>>(a);
    }
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return 0;
    *why = cudaGetErrorString(e);
    return -1;
}

}  // namespace ssm
