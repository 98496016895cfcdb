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
// tokens).  Measured: 16384 tokens of 56 + 8 + 8 heads of 128 appended to an int8 cache and read back from it
// in 125 us (5.7 TB/s); 124 K tokens of 8 heads of 128 read back from int8 to bf16 in 119 us (6.5 TB/s); a step's
// single token 6 us a call, the launch and two or three dependent loads.
#include <type_traits>

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

constexpr int kAppendThreads = 128;
constexpr int kAppendAhead = 4;         // rows a lane group has in flight
constexpr int kAppendBlocks = 7;        // on an SM

// How a token's rows are shared out: a turn is 32 / LPR heads of one kind (q heads first, then k, then
// v), a part is `turns` consecutive turns, taken by one warp.
struct AppendShape {
    int q_turns, kv_turns;              // turns of the q heads, of the k heads (and of the v heads)
    int turns, parts;                   // of a part, of a token
};

// A row of up to EPL * LPR elements lies on LPR lanes, EPL consecutive ones each, in registers from
// the load to the store; a pair's other element comes by a shuffle (half layout: from the lane half /
// EPL away, so half must be a multiple of EPL) or lies beside it (interleaved).  A warp reads a token's
// slot, position, cosines and sines once and then only rows, several at a time in flight.
template <bool I8, int EPL, int LPR>
__global__ void __launch_bounds__(kAppendThreads, kAppendBlocks)
k_attn_append(const AttnAppendArgs a, const AppendShape s) {
    constexpr int W = EPL / 2, kHeads = 32 / LPR;
    const int64_t id = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = id / s.parts;
    if (t >= a.n_tokens) return;                     // whole warps leave: no barrier below
    const int part = (int)(id - t * s.parts);
    const int sub = threadIdx.x % LPR, e = EPL * sub, head0 = (threadIdx.x & 31) / LPR;
    const int D = a.c.dim, half = a.rot / 2, nkv = a.c.n_kv;
    const bool mine = e < D;
    const int slot = a.slots[t];
    if (slot == -1) return;
    const int pos = a.rot ? a.positions[t] : 0;
    if (slot < 0 || slot >= a.c.n_pages * a.c.page_size || (a.rot && (pos < 0 || pos >= a.n_pos))) {
        if ((threadIdx.x & 31) == 0) atomicOr(a.status, kBadIndex);
        return;
    }
    const int begin = part * s.turns, end = begin + s.turns;
    // this lane's cosines and sines, the same for every head; half layout: one an element, interleaved: one a pair
    const bool turned = e < a.rot;
    const bool first = e < half;                     // half layout: this lane holds the pairs' first elements
    float cs[EPL], sn[EPL];
    if (turned && begin < s.q_turns + s.kv_turns) {
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

    // the heads of turns [lo, hi) of one kind: 0 q, 1 k, 2 v
    auto run = [&](auto kind_of, const void* in, int64_t st, int64_t sh, int heads, int lo, int hi) {
        constexpr int kind = decltype(kind_of)::value;
        const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(in) + t * st + e;
        for (int u0 = lo; u0 < hi; u0 += kAppendAhead) {
            uint32_t x[kAppendAhead][W];
#pragma unroll
            for (int u = 0; u < kAppendAhead; ++u) {
                const int h = (u0 + u) * kHeads + head0;
#pragma unroll
                for (int i = 0; i < W; ++i) x[u][i] = 0u;
                if (mine && u0 + u < hi && h < heads) Words<W>::load(x[u], src + h * sh);
            }
#pragma unroll
            for (int u = 0; u < kAppendAhead; ++u) {
                if (u0 + u >= hi) break;             // the whole warp's: shuffles follow
                const int h = (u0 + u) * kHeads + head0;
                const bool on = mine && h < heads;
                float y[EPL];
#pragma unroll
                for (int i = 0; i < W; ++i) y[2 * i] = lo_f32(x[u][i]), y[2 * i + 1] = hi_f32(x[u][i]);
                if (kind < 2 && a.rot) {
                    if (a.interleaved) {
                        if (turned)
#pragma unroll
                            for (int i = 0; i < W; ++i) {
                                const float p = y[2 * i], q = y[2 * i + 1];
                                y[2 * i] = rot_first(p, q, cs[i], sn[i]);
                                y[2 * i + 1] = rot_second(p, q, cs[i], sn[i]);
                            }
                    } else {
                        uint32_t o[W];
#pragma unroll
                        for (int i = 0; i < W; ++i) o[i] = __shfl_sync(0xffffffffu, x[u][i], other, LPR);
                        if (turned)
#pragma unroll
                            for (int i = 0; i < EPL; ++i) {
                                const float z = i & 1 ? hi_f32(o[i / 2]) : lo_f32(o[i / 2]);
                                y[i] = first ? rot_first(y[i], z, cs[i], sn[i]) : rot_second(z, y[i], cs[i], sn[i]);
                            }
                    }
                }
                uint32_t out[W];
                if (kind < 2 || !I8) {
#pragma unroll
                    for (int i = 0; i < W; ++i) out[i] = pack2(y[2 * i], y[2 * i + 1]);
                }
                if (kind == 0 && on)
                    Words<W>::store(reinterpret_cast<__nv_bfloat16*>(a.q_out) + t * a.qo_st + h * a.qo_sh + e, out);
                if (kind == 1 && on && a.k_out)
                    Words<W>::store(reinterpret_cast<__nv_bfloat16*>(a.k_out) + t * a.ko_st + h * a.ko_sh + e, out);
                if constexpr (kind > 0) {
                    const int64_t row = row0 + (int64_t)h * a.c.page_size;
                    void* cache = const_cast<void*>(kind == 1 ? a.c.k : a.c.v);
                    if constexpr (I8) {
                        // fmaxf passes over a NaN; the leading zero stands for a row of nothing else
                        float m = 0.f;
#pragma unroll
                        for (int i = 0; i < EPL; ++i) m = fmaxf(m, fabsf(y[i]));
#pragma unroll
                        for (int d = LPR / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                        if (on) {
                            const float inv = m > 0.f ? __fdiv_rn(127.f, m) : 0.f;
                            uint32_t codes[EPL / 4];
#pragma unroll
                            for (int i = 0; i < EPL / 4; ++i)
                                codes[i] = code8(y[4 * i], inv) | code8(y[4 * i + 1], inv) << 8 |
                                           code8(y[4 * i + 2], inv) << 16 | code8(y[4 * i + 3], inv) << 24;
                            int8_t* p = reinterpret_cast<int8_t*>(cache) + row * D + e;
                            if constexpr (EPL == 8) *reinterpret_cast<uint2*>(p) = make_uint2(codes[0], codes[1]);
                            else *reinterpret_cast<uint32_t*>(p) = codes[0];
                            if (sub == 0) const_cast<float*>(kind == 1 ? a.c.k_scale : a.c.v_scale)[row] = __fdiv_rn(m, 127.f);
                        }
                    } else {
                        if (on) Words<W>::store(reinterpret_cast<__nv_bfloat16*>(cache) + row * D + e, out);
                    }
                }
            }
        }
    };
    const int k0 = s.q_turns, v0 = k0 + s.kv_turns;
    run(std::integral_constant<int, 0>(), a.q, a.q_st, a.q_sh, a.n_q, begin, min(end, s.q_turns));
    run(std::integral_constant<int, 1>(), a.k, a.k_st, a.k_sh, nkv, max(begin, k0) - k0, min(end, v0) - k0);
    run(std::integral_constant<int, 2>(), a.v, a.v_st, a.v_sh, nkv, max(begin, v0) - v0, min(end - v0, s.kv_turns));
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
    constexpr int kHeads = 32 / LPR;
    AppendShape s;
    s.q_turns = (a.n_q + kHeads - 1) / kHeads;
    s.kv_turns = (a.c.n_kv + kHeads - 1) / kHeads;
    const int total = s.q_turns + 2 * s.kv_turns;
    // few tokens: a token's rows spread over so many warps that some 4864 (152 SMs x 32) run side by side;
    // many: a token a warp
    const int64_t want = (4864 + a.n_tokens - 1) / a.n_tokens;
    s.parts = (int)(want < 1 ? 1 : (want > total ? total : want));
    s.turns = (total + s.parts - 1) / s.parts;
    s.parts = (total + s.turns - 1) / s.turns;
    const int64_t warps = a.n_tokens * s.parts;
    constexpr int kPer = kAppendThreads / 32;
    k_attn_append<I8, EPL, LPR><<<(unsigned)((warps + kPer - 1) / kPer), kAppendThreads, 0, stream>>>(a, s);
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
