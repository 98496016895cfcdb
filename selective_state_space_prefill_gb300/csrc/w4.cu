// w4.cu -- weights of 4 bits with a scale (and a zero) per group: w4_quantize makes them, w4_linear multiplies
// the few rows of a decode step by them.
//
// A first form of w4_linear: a warp per output element, eight weights of a lane at a time.
#include "common.cuh"
#include "kernels.h"
#include "ssm.h"

namespace ssm {
namespace {

__device__ __forceinline__ float scale_at(const W4Weight& w, int64_t at) {
    return w.scale_bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(w.scales)[at])
                        : reinterpret_cast<const float*>(w.scales)[at];
}

// ------------------------------------------------------------------ quantisation
// A warp per group: a lane holds group / 32 consecutive elements.  Read once, at the rate of memory; the
// weight is made once and kept.
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
    float s = w.zeros ? __fdiv_rn(hi - lo, 15.f) : __fdiv_rn(fmaxf(-lo, hi), 7.f);
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
__global__ void __launch_bounds__(256) k_w4_linear(const W4LinearArgs a) {
    const int64_t id = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
    if (id >= (int64_t)a.M * a.w.N) return;
    const int64_t m = id / a.w.N, n = id % a.w.N;
    const int lane = threadIdx.x % 32, per_block = a.w.K / a.x_blocks;
    float sum = 0.f;
    for (int k = 8 * lane; k < a.w.K; k += 256) {
        const uint32_t c = *reinterpret_cast<const uint32_t*>(a.w.codes + n * a.w.ldc + k / 2);
        const int g = k / a.w.group;
        const float zero = a.w.zeros ? (float)(a.w.zeros[n * a.w.ldz + g] & 15) : 8.f;
        float part = 0.f;
        for (int i = 0; i < 8; ++i) {
            const float x = a.x_i8 ? (float)reinterpret_cast<const int8_t*>(a.x)[m * a.ldx + k + i]
                                   : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.x)[m * a.ldx + k + i]);
            part = fmaf((float)((c >> (4 * i)) & 15) - zero, x, part);
        }
        float s = scale_at(a.w, n * a.w.lds + g);
        if (a.x_scale) s *= a.x_scale[m * a.x_blocks + k / per_block];
        sum = fmaf(part, s, sum);
    }
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (lane != 0) return;
    if (a.out_bf16) reinterpret_cast<__nv_bfloat16*>(a.out)[m * a.ldo + n] = __float2bfloat16_rn(sum);
    else reinterpret_cast<float*>(a.out)[m * a.ldo + n] = sum;
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

int launch_w4_linear(const W4LinearArgs& a, cudaStream_t stream, const char** why) {
    k_w4_linear<<<(unsigned)(((int64_t)a.M * a.w.N + 7) / 8), 256, 0, stream>>>(a);
    return done(why);
}

}  // namespace ssm
