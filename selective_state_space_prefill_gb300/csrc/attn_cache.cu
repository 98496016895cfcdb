// attn_cache.cu -- rotary positions, the paged key/value cache's writer and its reader (sm_103a).
//
// These are the attention block's counterparts of the state cache of "Scaling State-Space Models
// on Multiple GPUs with Tensor Parallelism", Methodology 3 (prefill fills a cache that decode
// continues from), for the hybrid families the pages name (Overview: Zamba).
//
//   k_attn_rope_table cos/sin of every position, angles in fp64
//   k_attn_append       rotate q and k, write k and v (bf16, or int8 with a scale per row)
//   k_attn_read       cache rows back to packed tokens
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

__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// W 32-bit words (2 W bf16 elements) to and from memory in one access.
template <int W>
struct Words;
template <>
struct Words<2> {
    static __device__ __forceinline__ void load(uint32_t* w, const void* p) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        w[0] = x.x, w[1] = x.y;
    }
    static __device__ __forceinline__ void store(void* p, const uint32_t* w) {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
};
template <>
struct Words<4> {
    static __device__ __forceinline__ void load(uint32_t* w, const void* p) {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    }
    static __device__ __forceinline__ void store(void* p, const uint32_t* w) {
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

constexpr int kAppendThreads = 256;

// A row of up to EPL * LPR elements lies on LPR lanes, EPL consecutive ones each, in registers from
// the load to the store; a pair's other element comes by a shuffle (half layout: from the lane half /
// EPL away, so half must be a multiple of EPL) or lies beside it (interleaved).  grid.x: tokens;
// grid.y: groups of rows_per_block of the token's n_q + 2 n_kv rows (q heads, then k heads, then v
// heads).  The next row's load is in flight while a row is worked on.
template <bool I8, int EPL, int LPR>
__global__ void __launch_bounds__(kAppendThreads)
k_attn_append(const AttnAppendArgs a, int rows_per_block) {
    constexpr int kRows = kAppendThreads / LPR, W = EPL / 2;
    const int64_t t = blockIdx.x;
    const int sub = threadIdx.x % LPR, e = EPL * sub;
    const int D = a.c.dim, half = a.rot / 2, nkv = a.c.n_kv;
    const int rows = a.n_q + 2 * nkv;
    const int r_end = min(rows, ((int)blockIdx.y + 1) * rows_per_block);
    int r = (int)blockIdx.y * rows_per_block + threadIdx.x / LPR;
    const __nv_bfloat16* qp = reinterpret_cast<const __nv_bfloat16*>(a.q) + t * a.q_st + e;
    const __nv_bfloat16* kp = reinterpret_cast<const __nv_bfloat16*>(a.k) + t * a.k_st + e;
    const __nv_bfloat16* vp = reinterpret_cast<const __nv_bfloat16*>(a.v) + t * a.v_st + e;
    const bool mine = e < D;
    auto load = [&](int r, uint32_t* w) {
        const __nv_bfloat16* p = r < a.n_q ? qp + r * a.q_sh
                                           : (r < a.n_q + nkv ? kp + (r - a.n_q) * a.k_sh : vp + (r - a.n_q - nkv) * a.v_sh);
        if (mine && r < r_end) Words<W>::load(w, p);
    };
    uint32_t x[W] = {}, nx[W] = {};
    const int slot = a.slots[t];
    const int pos = a.rot ? a.positions[t] : 0;
    if (slot != -1) load(r, x);
    if (slot == -1) return;
    if (slot < 0 || slot >= a.c.n_pages * a.c.page_size || (a.rot && (pos < 0 || pos >= a.n_pos))) {
        if (threadIdx.x == 0) atomicOr(a.status, kBadIndex);
        return;
    }
    // this lane's cosines and sines, the same for every head; half layout: one a element, interleaved: one a pair
    const bool turned = e < a.rot;
    const bool first = e < half;                     // half layout: this lane holds the pairs' first elements
    float cs[EPL], sn[EPL];
    if (turned) {
        const float *cr = a.cos + (int64_t)pos * half, *sr = a.sin + (int64_t)pos * half;
        if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < EPL / 2; ++i) cs[i] = cr[e / 2 + i], sn[i] = sr[e / 2 + i];
        } else {
            const int at = first ? e : e - half;
#pragma unroll
            for (int i = 0; i < EPL; i += 4) {
                const float4 c4 = *reinterpret_cast<const float4*>(cr + at + i), s4 = *reinterpret_cast<const float4*>(sr + at + i);
                cs[i] = c4.x, cs[i + 1] = c4.y, cs[i + 2] = c4.z, cs[i + 3] = c4.w;
                sn[i] = s4.x, sn[i + 1] = s4.y, sn[i + 2] = s4.z, sn[i + 3] = s4.w;
            }
        }
    }
    const int other = turned ? (first ? sub + half / EPL : sub - half / EPL) : sub;
    const int64_t row0 = (int64_t)(slot / a.c.page_size) * nkv * a.c.page_size + slot % a.c.page_size;
    __nv_bfloat16* qo = reinterpret_cast<__nv_bfloat16*>(a.q_out) + t * a.qo_st + e;
    __nv_bfloat16* ko = reinterpret_cast<__nv_bfloat16*>(a.k_out) + t * a.ko_st + e;

    // every lane of the block takes the same number of turns: the shuffles are the whole warp's
    for (int r0 = (int)blockIdx.y * rows_per_block; r0 < r_end; r0 += kRows, r += kRows) {
        load(r + kRows, nx);
        const bool on = mine && r < r_end;
        const int kind = r < a.n_q ? 0 : (r < a.n_q + nkv ? 1 : 2);         // q, k, v
        const int h = kind == 0 ? r : (kind == 1 ? r - a.n_q : r - a.n_q - nkv);
        float y[EPL];
#pragma unroll
        for (int i = 0; i < W; ++i) y[2 * i] = lo_f32(x[i]), y[2 * i + 1] = hi_f32(x[i]);
        if (a.rot) {                                  // the same branch for the whole block
            if (a.interleaved) {
                if (turned && kind < 2)
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        const float u = y[2 * i], v = y[2 * i + 1];
                        y[2 * i] = rot_first(u, v, cs[i], sn[i]);
                        y[2 * i + 1] = rot_second(u, v, cs[i], sn[i]);
                    }
            } else {
                uint32_t o[W];
#pragma unroll
                for (int i = 0; i < W; ++i) o[i] = __shfl_sync(0xffffffffu, x[i], other, LPR);
                if (turned && kind < 2)
#pragma unroll
                    for (int i = 0; i < EPL; ++i) {
                        const float z = i & 1 ? hi_f32(o[i / 2]) : lo_f32(o[i / 2]);
                        y[i] = first ? rot_first(y[i], z, cs[i], sn[i]) : rot_second(z, y[i], cs[i], sn[i]);
                    }
            }
        }
        uint32_t out[W];
#pragma unroll
        for (int i = 0; i < W; ++i) out[i] = pack2(y[2 * i], y[2 * i + 1]);
        if (on && kind == 0) Words<W>::store(qo + h * a.qo_sh, out);
        if (on && kind == 1 && a.k_out) Words<W>::store(ko + h * a.ko_sh, out);
        const int64_t row = row0 + (int64_t)h * a.c.page_size;
        if constexpr (I8) {
            // fmaxf passes over a NaN; the leading zero stands for a row of nothing else
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) m = fmaxf(m, fabsf(y[i]));
            if (!on) m = 0.f;
#pragma unroll
            for (int d = LPR / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
            if (on && kind > 0) {
                const float inv = m > 0.f ? __fdiv_rn(127.f, m) : 0.f;
                uint32_t codes[EPL / 4];
#pragma unroll
                for (int i = 0; i < EPL / 4; ++i)
                    codes[i] = code8(y[4 * i], inv) | code8(y[4 * i + 1], inv) << 8 | code8(y[4 * i + 2], inv) << 16 |
                               code8(y[4 * i + 3], inv) << 24;
                int8_t* p = reinterpret_cast<int8_t*>(const_cast<void*>(kind == 1 ? a.c.k : a.c.v)) + row * D + e;
                if constexpr (EPL == 8) *reinterpret_cast<uint2*>(p) = make_uint2(codes[0], codes[1]);
                else *reinterpret_cast<uint32_t*>(p) = codes[0];
                if (sub == 0) const_cast<float*>(kind == 1 ? a.c.k_scale : a.c.v_scale)[row] = __fdiv_rn(m, 127.f);
            }
        } else {
            if (on && kind > 0)
                Words<W>::store(reinterpret_cast<__nv_bfloat16*>(const_cast<void*>(kind == 1 ? a.c.k : a.c.v)) + row * D + e, out);
        }
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = nx[i];
    }
}

// ------------------------------------------------------------------ read
constexpr int kReadThreads = 256;
constexpr int kReadAhead = 4;           // chunks of 8 elements a thread has in flight, for k and for v
constexpr int kReadTokens = 32;         // most tokens per block

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
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float v[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}

// n / d for n * d < 2^32, with magic = ceil(2^32 / d): the error n (magic d - 2^32) / 2^32 d is below 1 / d.
__device__ __forceinline__ uint32_t quotient(uint32_t n, uint32_t magic, uint32_t d) { return d == 1 ? n : __umulhi(n, magic); }

struct ReadShape {
    uint32_t tokens;                    // of a block
    uint32_t row_chunks, row_magic;     // chunks of 8 elements of a row
    uint32_t tok_chunks, tok_magic;     // ... of a token's kv heads
};

// A block takes a few consecutive tokens: one warp finds their sequences and pages, then every thread
// moves chunks of 8 elements, the loads of several rows in flight together.
template <bool I8, typename Tout>
__global__ void __launch_bounds__(kReadThreads)
k_attn_read(const AttnReadArgs a, const ReadShape s) {
    __shared__ int64_t s_slot[kReadTokens];          // cache row of the token's head 0, or -1
    const int64_t t0 = (int64_t)blockIdx.x * s.tokens;
    if (threadIdx.x < 32) {
        int b = find_sequence(a.cu_len, a.batch, t0);
        const int64_t t = t0 + threadIdx.x;
        int64_t slot = -1;
        if (threadIdx.x < s.tokens && t < a.n_tokens) {
            while (b + 1 < a.batch && a.cu_len[b + 1] <= t) ++b;
            const int64_t p = t - a.cu_len[b] + (a.first ? a.first[b] : 0);
            const uint32_t p32 = (uint32_t)p, pi = p32 / (uint32_t)a.c.page_size;
            const int page = p >= 0 && p < (1LL << 31) && pi < (uint32_t)a.n_table ? a.page_table[b * a.table_stride + pi] : -1;
            if (page < 0 || page >= a.c.n_pages) atomicOr(a.status, kBadIndex);
            else slot = (int64_t)page * a.c.n_kv * a.c.page_size + p32 % (uint32_t)a.c.page_size;
        }
        s_slot[threadIdx.x] = slot;
    }
    __syncthreads();
    const int D = a.c.dim;
    const uint32_t total = s.tokens * s.tok_chunks;
    constexpr int W = I8 ? 2 : 4;
    for (uint32_t i0 = threadIdx.x; i0 < total; i0 += kReadAhead * kReadThreads) {
        uint32_t w[kReadAhead][2][W];
        float sc[kReadAhead][2];
        int64_t to[kReadAhead];                      // where the chunk goes, or -1
#pragma unroll
        for (int u = 0; u < kReadAhead; ++u) {
            const uint32_t i = i0 + u * kReadThreads;
            to[u] = -1;
            if (i >= total) continue;
            const uint32_t tk = quotient(i, s.tok_magic, s.tok_chunks), c = i - tk * s.tok_chunks;
            const uint32_t h = quotient(c, s.row_magic, s.row_chunks), e = (c - h * s.row_chunks) * 8;
            const int64_t slot = s_slot[tk];
            if (slot < 0) continue;
            to[u] = (t0 + tk) * (int64_t)s.tok_chunks * 8 + c * 8;
            const int64_t row = slot + (int64_t)h * a.c.page_size, at = row * D + e;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const void* base = kv ? a.c.v : a.c.k;
                if constexpr (I8) {
                    const uint2 x = __ldcs(reinterpret_cast<const uint2*>(reinterpret_cast<const int8_t*>(base) + at));
                    w[u][kv][0] = x.x, w[u][kv][1] = x.y;
                    sc[u][kv] = __ldg((kv ? a.c.v_scale : a.c.k_scale) + row);
                } else {
                    const uint4 x = __ldcs(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(base) + at));
                    w[u][kv][0] = x.x, w[u][kv][1] = x.y, w[u][kv][2] = x.z, w[u][kv][3] = x.w;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kReadAhead; ++u) {
            if (to[u] < 0) continue;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                Tout* p = reinterpret_cast<Tout*>(kv ? a.v_out : a.k_out) + to[u];
                if constexpr (!I8 && sizeof(Tout) == 2) {
                    Words<4>::store(p, w[u][kv]);    // the row itself
                } else {
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if constexpr (I8) v[j] = __fmul_rn((float)(int8_t)(w[u][kv][j >> 2] >> (8 * (j & 3))), sc[u][kv]);
                        else v[j] = j & 1 ? hi_f32(w[u][kv][j >> 1]) : lo_f32(w[u][kv][j >> 1]);
                    }
                    store8(p, v);
                }
            }
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

template <bool I8, int EPL, int LPR>
static void append(const AttnAppendArgs& a, cudaStream_t stream) {
    const int rows = a.n_q + 2 * a.c.n_kv, per_pass = kAppendThreads / LPR;
    // few tokens: a row per lane group, so that the rows run side by side; many: a block per token, which
    // reads the token's slot, position, cosines and sines once
    const int rows_per_block = a.n_tokens < 1024 ? per_pass : (rows + per_pass - 1) / per_pass * per_pass;
    const dim3 grid((unsigned)a.n_tokens, (unsigned)((rows + rows_per_block - 1) / rows_per_block));
    k_attn_append<I8, EPL, LPR><<<grid, kAppendThreads, 0, stream>>>(a, rows_per_block);
}

template <bool I8>
static void append_shape(const AttnAppendArgs& a, cudaStream_t stream) {
    // eight elements (16 bytes) a lane, unless a pair's halves are not whole lanes of eight apart
    const bool eight = a.interleaved || a.rot % 16 == 0;
    if (a.c.dim <= 64) {
        if (eight) append<I8, 8, 8>(a, stream);
        else append<I8, 4, 16>(a, stream);
    } else {
        if (eight) append<I8, 8, 16>(a, stream);
        else append<I8, 4, 32>(a, stream);
    }
}

int launch_attn_append(const AttnAppendArgs& a, bool cache_i8, cudaStream_t stream, const char** why) {
    if (cache_i8) append_shape<true>(a, stream);
    else append_shape<false>(a, stream);
    return launched(why);
}

int launch_attn_read(const AttnReadArgs& a, bool cache_i8, bool out_bf16, cudaStream_t stream, const char** why) {
    ReadShape s;
    auto magic = [](uint32_t d) { return (uint32_t)(((1ull << 32) + d - 1) / d); };
    s.row_chunks = (uint32_t)a.c.dim / 8;
    s.row_magic = magic(s.row_chunks);
    s.tok_chunks = s.row_chunks * (uint32_t)a.c.n_kv;                    // at most 4096 x 16
    s.tok_magic = magic(s.tok_chunks);
    const uint32_t want = kReadAhead * kReadThreads / s.tok_chunks;      // one turn of every thread
    s.tokens = want < 1 ? 1 : (want > (uint32_t)kReadTokens ? (uint32_t)kReadTokens : want);
    const unsigned grid = (unsigned)((a.n_tokens + s.tokens - 1) / s.tokens);
    if (cache_i8) {
        if (out_bf16) k_attn_read<true, __nv_bfloat16><<<grid, kReadThreads, 0, stream>>>(a, s);
        else k_attn_read<true, float><<<grid, kReadThreads, 0, stream>>>(a, s);
    } else {
        if (out_bf16) k_attn_read<false, __nv_bfloat16><<<grid, kReadThreads, 0, stream>>>(a, s);
        else k_attn_read<false, float><<<grid, kReadThreads, 0, stream>>>(a, s);
    }
    return launched(why);
}

}  // namespace ssm
