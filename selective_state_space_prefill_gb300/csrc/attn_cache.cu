// attn_cache.cu -- rotary positions, the paged key/value cache's writer and its reader (sm_103a).
//
// These are the attention block's counterparts of the state cache of "Scaling State-Space Models
// on Multiple GPUs with Tensor Parallelism", Methodology 3 (prefill fills a cache that decode
// continues from), for the hybrid families the pages name (Overview: Zamba).
//
//   k_attn_rope_table   cos/sin of every position, angles in fp64
//   k_attn_append       rotate q and k, write k and v (bf16, or int8 with a scale per row)
//   k_attn_read         cache rows back to packed tokens
//
// All three are elementwise over rows: the bytes moved bound them (and launch latency, for a few
// tokens).
#include "common.cuh"
#include "kernels.h"

namespace ssm {
namespace {

constexpr unsigned kBadIndex = 8u;      // SSM_DEV_BAD_INDEX

// ------------------------------------------------------------------ rope table
__global__ void k_attn_rope_table(const AttnRopeArgs a) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= a.n_pos * a.half) return;
    double s, c;
    sincos((double)(i / a.half) * a.inv_freq[i % a.half], &s, &c);
    a.cos[i] = (float)(a.scale * c);
    a.sin[i] = (float)(a.scale * s);
}

// ------------------------------------------------------------------ append
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// (a c - b s) and (b c + a s) with the products rounded before the sum: the same bits as an
// elementwise evaluation, so that int8 codes do not depend on a contraction.
__device__ __forceinline__ float rot_first(float a, float b, float c, float s) {
    return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
__device__ __forceinline__ float rot_second(float a, float b, float c, float s) {
    return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

// code = rne(x * inv) in [-127, 127]; the conversion sends a NaN to 0.
__device__ __forceinline__ uint32_t code8(float x, float inv) {
    int q = __float2int_rn(__fmul_rn(x, inv));
    q = q < -127 ? -127 : (q > 127 ? 127 : q);
    return (uint32_t)(q & 255);
}

constexpr int kAppendThreads = 256;

// LPR lanes hold a row of up to 4 * LPR elements, four each.  grid.x: tokens; grid.y: groups of
// rows_per_block of the token's n_q + 2 n_kv rows (q heads, then k heads, then v heads).
template <bool I8, int LPR>
__global__ void __launch_bounds__(kAppendThreads)
k_attn_append(const AttnAppendArgs a, int rows_per_block) {
    constexpr int kRows = kAppendThreads / LPR;
    const int64_t t = blockIdx.x;
    const int sub = threadIdx.x % LPR;
    const int e = 4 * sub;
    const int D = a.c.dim, half = a.rot / 2, nkv = a.c.n_kv;
    const int slot = a.slots[t];
    if (slot == -1) return;
    const int pos = a.rot ? a.positions[t] : 0;
    if (slot < 0 || slot >= a.c.n_pages * a.c.page_size || (a.rot && (pos < 0 || pos >= a.n_pos))) {
        if (threadIdx.x == 0) atomicOr(a.status, kBadIndex);
        return;
    }
    // this lane's cosines and sines, the same for every head
    float4 c4 = make_float4(1.f, 1.f, 1.f, 1.f), s4 = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool turned = e < a.rot;
    const bool first = e < half;                     // half layout: this lane holds the pairs' first elements
    if (turned) {
        const float *cr = a.cos + (int64_t)pos * half, *sr = a.sin + (int64_t)pos * half;
        if (a.interleaved) {
            c4.x = cr[e / 2], c4.z = cr[e / 2 + 1], s4.x = sr[e / 2], s4.z = sr[e / 2 + 1];
        } else {
            const int i = first ? e : e - half;
            c4 = *reinterpret_cast<const float4*>(cr + i);
            s4 = *reinterpret_cast<const float4*>(sr + i);
        }
    }
    const int partner = first ? sub + half / 4 : sub - half / 4;
    const int page = slot / a.c.page_size, off = slot % a.c.page_size;
    const int rows = a.n_q + 2 * nkv;
    const int r_end = min(rows, ((int)blockIdx.y + 1) * rows_per_block);
    for (int r0 = (int)blockIdx.y * rows_per_block; r0 < r_end; r0 += kRows) {
        const int r = r0 + threadIdx.x / LPR;
        const bool on = r < r_end && e < D;
        const int kind = r < a.n_q ? 0 : (r < a.n_q + nkv ? 1 : 2);         // q, k, v
        const int h = kind == 0 ? r : (kind == 1 ? r - a.n_q : r - a.n_q - nkv);
        const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(kind == 0 ? a.q : (kind == 1 ? a.k : a.v)) +
                                   t * (kind == 0 ? a.q_st : (kind == 1 ? a.k_st : a.v_st)) +
                                   (int64_t)h * (kind == 0 ? a.q_sh : (kind == 1 ? a.k_sh : a.v_sh)) + e;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (on) x = load4(src);
        float4 y = x;
        if (a.rot) {                                  // the same branch for the whole block: shuffles inside
            if (a.interleaved) {
                if (turned && kind < 2)
                    y = make_float4(rot_first(x.x, x.y, c4.x, s4.x), rot_second(x.x, x.y, c4.x, s4.x),
                                    rot_first(x.z, x.w, c4.z, s4.z), rot_second(x.z, x.w, c4.z, s4.z));
            } else {
                const int src_lane = turned ? partner : sub;
                float4 o;
                o.x = __shfl_sync(0xffffffffu, x.x, src_lane, LPR);
                o.y = __shfl_sync(0xffffffffu, x.y, src_lane, LPR);
                o.z = __shfl_sync(0xffffffffu, x.z, src_lane, LPR);
                o.w = __shfl_sync(0xffffffffu, x.w, src_lane, LPR);
                if (turned && kind < 2)
                    y = first ? make_float4(rot_first(x.x, o.x, c4.x, s4.x), rot_first(x.y, o.y, c4.y, s4.y),
                                            rot_first(x.z, o.z, c4.z, s4.z), rot_first(x.w, o.w, c4.w, s4.w))
                              : make_float4(rot_second(o.x, x.x, c4.x, s4.x), rot_second(o.y, x.y, c4.y, s4.y),
                                            rot_second(o.z, x.z, c4.z, s4.z), rot_second(o.w, x.w, c4.w, s4.w));
            }
        }
        if (on && kind == 0)
            store4(reinterpret_cast<__nv_bfloat16*>(a.q_out) + t * a.qo_st + (int64_t)h * a.qo_sh + e, y);
        if (on && kind == 1 && a.k_out)
            store4(reinterpret_cast<__nv_bfloat16*>(a.k_out) + t * a.ko_st + (int64_t)h * a.ko_sh + e, y);
        const int64_t row = ((int64_t)page * nkv + h) * a.c.page_size + off;
        void* cache = const_cast<void*>(kind == 1 ? a.c.k : a.c.v);
        if constexpr (I8) {
            // fmaxf passes over a NaN; the leading zero stands for a row of nothing else
            float m = on ? fmaxf(fmaxf(fmaxf(fmaxf(0.f, fabsf(y.x)), fabsf(y.y)), fabsf(y.z)), fabsf(y.w)) : 0.f;
#pragma unroll
            for (int d = LPR / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d, LPR));
            if (on && kind > 0) {
                const float inv = m > 0.f ? __fdiv_rn(127.f, m) : 0.f;
                const uint32_t w = code8(y.x, inv) | code8(y.y, inv) << 8 | code8(y.z, inv) << 16 | code8(y.w, inv) << 24;
                *reinterpret_cast<uint32_t*>(reinterpret_cast<int8_t*>(cache) + row * D + e) = w;
                if (sub == 0) const_cast<float*>(kind == 1 ? a.c.k_scale : a.c.v_scale)[row] = __fdiv_rn(m, 127.f);
            }
        } else {
            if (on && kind > 0) store4(reinterpret_cast<__nv_bfloat16*>(cache) + row * D + e, y);
        }
    }
}

// ------------------------------------------------------------------ read
constexpr int kReadThreads = 256;
constexpr int kReadTokens = 16;         // tokens per block

// The last b with cu[b] <= t, b < n, by the calling warp: 32 pivots a round.
__device__ __forceinline__ int find_sequence(const int32_t* cu, int n, int64_t t) {
    int lo = 0, hi = n;
    const int lane = threadIdx.x & 31;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int p = lo + lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, p < hi && cu[p] <= t);
        if (below == 0) break;
        lo += (__popc(below) - 1) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

__device__ __forceinline__ void store8(float* p, const float v[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float v[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool I8, typename Tout>
__global__ void __launch_bounds__(kReadThreads)
k_attn_read(const AttnReadArgs a) {
    __shared__ int64_t s_slot[kReadTokens];          // cache row of the token's head 0, or -1
    const int64_t t0 = (int64_t)blockIdx.x * kReadTokens;
    if (threadIdx.x < 32) {
        int b = find_sequence(a.cu_len, a.batch, t0);
        const int64_t t = t0 + threadIdx.x;
        if (threadIdx.x < kReadTokens) {
            int64_t slot = -1;
            if (t < a.n_tokens) {
                while (b + 1 < a.batch && a.cu_len[b + 1] <= t) ++b;
                const int64_t p = t - a.cu_len[b] + (a.first ? a.first[b] : 0);
                const int64_t pi = p / a.c.page_size;
                const int page = p >= 0 && pi < a.n_table ? a.page_table[b * a.table_stride + pi] : -1;
                if (page < 0 || page >= a.c.n_pages) atomicOr(a.status, kBadIndex);
                else slot = (int64_t)page * a.c.n_kv * a.c.page_size + p % a.c.page_size;
            }
            s_slot[threadIdx.x] = slot;
        }
    }
    __syncthreads();
    const int D = a.c.dim, cpr = D / 8, per_token = a.c.n_kv * cpr;      // 8-element chunks
    for (int i = threadIdx.x; i < kReadTokens * per_token; i += kReadThreads) {
        const int tk = i / per_token, rest = i % per_token, h = rest / cpr, e = (rest % cpr) * 8;
        const int64_t slot = s_slot[tk];
        if (slot < 0) continue;
        const int64_t row = slot + (int64_t)h * a.c.page_size;
        const int64_t o = ((t0 + tk) * a.c.n_kv + h) * D + e;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            float x[8];
            if constexpr (I8) {
                const uint2 w = __ldcs(reinterpret_cast<const uint2*>(reinterpret_cast<const int8_t*>(kv ? a.c.v : a.c.k) + row * D + e));
                const float s = (kv ? a.c.v_scale : a.c.k_scale)[row];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[j] = __fmul_rn((float)(int8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3))), s);
            } else {
                const uint4 w = __ldcs(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(kv ? a.c.v : a.c.k) + row * D + e));
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[2 * j] = __uint_as_float(ws[j] << 16);
                    x[2 * j + 1] = __uint_as_float(ws[j] & 0xffff0000u);
                }
            }
            store8(reinterpret_cast<Tout*>(kv ? a.v_out : a.k_out) + o, x);
        }
    }
}

int launched(const char** why) {
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return 0;
    *why = cudaGetErrorString(e);
    return -1;
}

}  // namespace

int launch_attn_rope_table(const AttnRopeArgs& a, cudaStream_t stream, const char** why) {
    const int64_t n = a.n_pos * a.half;
    k_attn_rope_table<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(a);
    return launched(why);
}

int launch_attn_append(const AttnAppendArgs& a, bool cache_i8, cudaStream_t stream, const char** why) {
    const int rows = a.n_q + 2 * a.c.n_kv;
    const int lpr = a.c.dim > 64 ? 32 : 16;
    const int per_pass = kAppendThreads / lpr;
    // few tokens: a row per lane group, so that the rows run side by side; many: a block per token
    const int rows_per_block = a.n_tokens < 1024 ? per_pass : (rows + per_pass - 1) / per_pass * per_pass;
    const dim3 grid((unsigned)a.n_tokens, (unsigned)((rows + rows_per_block - 1) / rows_per_block));
    if (cache_i8) {
        if (lpr == 32) k_attn_append<true, 32><<<grid, kAppendThreads, 0, stream>>>(a, rows_per_block);
        else k_attn_append<true, 16><<<grid, kAppendThreads, 0, stream>>>(a, rows_per_block);
    } else {
        if (lpr == 32) k_attn_append<false, 32><<<grid, kAppendThreads, 0, stream>>>(a, rows_per_block);
        else k_attn_append<false, 16><<<grid, kAppendThreads, 0, stream>>>(a, rows_per_block);
    }
    return launched(why);
}

int launch_attn_read(const AttnReadArgs& a, bool cache_i8, bool out_bf16, cudaStream_t stream, const char** why) {
    const unsigned grid = (unsigned)((a.n_tokens + kReadTokens - 1) / kReadTokens);
    if (cache_i8) {
        if (out_bf16) k_attn_read<true, __nv_bfloat16><<<grid, kReadThreads, 0, stream>>>(a);
        else k_attn_read<true, float><<<grid, kReadThreads, 0, stream>>>(a);
    } else {
        if (out_bf16) k_attn_read<false, __nv_bfloat16><<<grid, kReadThreads, 0, stream>>>(a);
        else k_attn_read<false, float><<<grid, kReadThreads, 0, stream>>>(a);
    }
    return launched(why);
}

}  // namespace ssm
