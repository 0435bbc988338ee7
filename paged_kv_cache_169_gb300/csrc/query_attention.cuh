// paged_query_attention: what its kernels share.  Row i of a sequence with n new tokens and context c
// stands at p = c - n + i and sees positions [lo, hi) (row_range); with x = scale q.k_j its scores are
// t_j = cap tanh(x / cap) - slope |p - j|, and out = sum_j softmax(t)_j v_j.
#pragma once

#include <math_constants.h>

#include "int4.cuh"
#include "pool_types.cuh"
#include "query_parts.h"

namespace kvp {

struct QueryArgs {
    const char* q;
    char* out;
    int64_t q_stride, out_stride;      // bytes between tokens
    const int32_t *query_start, *tables, *lens;
    const float* slopes;
    const int2* ranges;
    const char *kpool, *vpool;
    const float *kscale, *vscale;
    int num_tokens, max_queries, max_blocks, batch, ctx_limit, window;
    int H, G, B, log_b, num_blocks;    // K/V heads, query heads per K/V head, block size and its logarithm
    float scale, cap;                  // cap 0: none
    int splits;                        // parts of an item's keys in the tensor-core kernel; above 1, joined afterwards:
    float2* part_ml;                   // [part][row][query head] (QueryParts): base in log2 units, sum of weights
    float* part_o;                     // and the weighted sums, [D]
    int64_t part_rows;
    bool part_by_sequence;
    int* err;
};

// Longest context and most rows of a call: positions are exact in float32 there.
constexpr int kMaxQueryTokens = 1 << 24;

constexpr float kLog2e = 1.4426950408889634f;

#ifdef __CUDACC__

// 16 bytes global -> shared, or zeros (nothing is read)
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const char* src, bool read) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(read ? 16 : 0) : "memory");
}

// A sequence's rows of q (first, n) and its context; n 0 where it is left out.
struct QuerySeq { int first, n, ctx; };

__device__ __forceinline__ QuerySeq query_seq(const QueryArgs& a, int s, bool report) {
    QuerySeq r;
    r.first = a.query_start[s];
    const int end = a.query_start[s + 1];
    const int c = a.lens[s];
    r.n = end - r.first;
    r.ctx = c < 0 ? 0 : c > a.ctx_limit ? a.ctx_limit : c;
    if (r.first < 0 || end < r.first || end > a.num_tokens || r.n > a.max_queries) {
        if (report) atomicOr(a.err, KV_DEVERR_QUERY);
        r.n = 0;
    } else if (report && r.n > 0 && (r.ctx != c || r.n > c)) {
        atomicOr(a.err, KV_DEVERR_CONTEXT);
    }
    return r;
}

// Positions [x, y) that row i of sequence q sees; (0, 0) where it sees none.
__device__ __forceinline__ int2 row_range(const QueryArgs& a, const QuerySeq& q, int i) {
    const int p = q.ctx - q.n + i;
    int2 r = make_int2(0, p + 1);
    if (a.ranges) r = a.ranges[q.first + i];
    r.x = max(r.x, 0);
    if (a.window > 0) r.x = max(r.x, p - a.window + 1);
    r.y = min(r.y, q.ctx);
    return r.x < r.y ? r : make_int2(0, 0);
}

// A block id of a table; one outside the pool is reported and read as block 0.
__device__ __forceinline__ int checked_block(const QueryArgs& a, int id) {
    if (static_cast<unsigned>(id) < static_cast<unsigned>(a.num_blocks)) return id;
    atomicOr(a.err, KV_DEVERR_BLOCK_ID);
    return 0;
}
// The physical block of position j of sequence s.
__device__ __forceinline__ int query_block(const QueryArgs& a, int s, int j) {
    return checked_block(a, a.tables[static_cast<int64_t>(s) * a.max_blocks + (j >> a.log_b)]);
}

// t = cap tanh(x) in log2 units for x = s kx: 1 - 2 / (e^2x + 1), exact to a few 2^-24 of the cap
__device__ __forceinline__ float capped(float s, float k2, float capl) {
    const float e = ex2_approx(s * k2);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + 1.f));
    return fmaf(-2.f * capl, r, capl);
}

// That error is a part of the cap, whatever the score: up to a cap of 64 it is below 2^-14, an eighth of what rounding a
// weight to float16 is.  Above, the score counts: where |x| < cap / 2 the series of tanh about 0 (its next term is below
// 2^-23), elsewhere as above; 2^-21 of the score in all.  sl: scale in log2 units.
constexpr float kLargeCap = 64.f, kHalfLn2Sq = 0.12011325f;
// tanh y = y (1 + z (-1/3 + 2/15 z - ...)), z = y^2
__device__ constexpr float kTanh[6] = {21844.f / 6081075.f, -1382.f / 155925.f, 62.f / 2835.f, -17.f / 315.f, 2.f / 15.f, -1.f / 3.f};
__device__ __forceinline__ float capped_large(float s, float sl, float k2, float capl) {
    const float u = s * k2, z = u * u * kHalfLn2Sq, x = s * sl;                // u = 2 x / cap in log2 units; z = (x / cap)^2
    float p = kTanh[0];
    #pragma unroll
    for (int i = 1; i < 6; ++i) p = fmaf(p, z, kTanh[i]);
    return fabsf(u) < kLog2e ? fmaf(x * p, z, x) : capped(s, k2, capl);
}

// Weights are kept 2^7 above their softmax value relative to the base, which may lag the maximum by up to 2^8:
// at most 2^15 in float16, and normal ones down to 2^-21 of the largest.
constexpr float kRaise = 8.f, kLift = 7.f;

// FP8: a weight enters the products times its block's value scale v, so the base follows the maximum of t + log2 v (the
// weights' sum has the same base): what counts is a row's own largest product, whatever scales it does not see, or hardly.
// (With scales relative to the largest of a work item, a row beside a scale 2^32 times its own was 0.)  v below 2^-60 counts
// as that: values of less than 2^-51, lost in float16's rounding.  What is no scale, or so large that results overflow, is
// NaN: a row that sees it is worked out again from the definition.  (Base and sums are joined across 2^84 of scales, so that
// a weight that underflows there is below 2^-42 of the others.)
constexpr float kLeastScale = -60.f, kMostScale = 24.f;        // log2
__device__ __forceinline__ float value_log2(float v) {
    return v >= 0.f && v <= 16777216.f ? fmaxf(log2f(v), kLeastScale) : CUDART_NAN_F;
}

template <int D, kv_dtype POOL>
constexpr int kRowBytes = POOL == KV_INT4 ? D / 2 + D / 16 : POOL == KV_FP8_E4M3 ? D : 2 * D;

// Elements [part * D/8, (part + 1) * D/8) of token `off` of a (block, head) tile, as float32 (FP8: codes).
template <int D, kv_dtype POOL, bool IS_V>
__device__ __forceinline__ void load_eighth(const char* tile, int off, int part, float (&x)[D / 8]) {
    constexpr int N = D / 8;
    if constexpr (POOL == KV_INT4) {
        const char* oct = tile + (off >> 3) * Int4<D>::OCT;
        const int t = off & 7;
        const uint8_t sb = *reinterpret_cast<const uint8_t*>(
            oct + (IS_V ? int4_v_scale<D>(t, part * N) : int4_k_scale<D>(t, part * N)));
        const float s = int4_scale_value(sb);
        #pragma unroll
        for (int i = 0; i < N; i += 4) {
            const int at = IS_V ? int4_v_piece<D>(t, part * N + i) : int4_k_code<D>(t, part * N + i);
            const uint32_t w = *reinterpret_cast<const uint16_t*>(oct + at);
            #pragma unroll
            for (int k = 0; k < 4; ++k) x[i + k] = static_cast<float>(static_cast<int>(w >> (4 * k) & 15u) - 8) * s;
        }
    } else {
        const char* row = tile + (static_cast<int64_t>(off) * D + part * N) * (kRowBytes<D, POOL> / D);
        if constexpr (POOL == KV_F16) {
            #pragma unroll
            for (int i = 0; i < N; i += 8) {
                const uint4 v = *reinterpret_cast<const uint4*>(row + 2 * i);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                #pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
                    x[i + 2 * k] = f.x;
                    x[i + 2 * k + 1] = f.y;
                }
            }
        } else {
            #pragma unroll
            for (int i = 0; i < N; i += 8) {
                const uint2 v = *reinterpret_cast<const uint2*>(row + i);
                const uint32_t w[2] = {v.x, v.y};
                #pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 f = e4m3x2_to_float2(static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1))));
                    x[i + 2 * k] = f.x;
                    x[i + 2 * k + 1] = f.y;
                }
            }
        }
    }
}

// One (row, query head) by one warp, in float32 from the definition: only what the row sees is read.
// Eight lanes share a key, four keys go side by side with a softmax state each, joined at the end.
template <int D, kv_dtype POOL>
__device__ __noinline__ void attend_row(const QueryArgs& a, int s, QuerySeq seq, int i, int head) {
    constexpr int N = D / 8;
    const int lane = threadIdx.x & 31, part = lane & 7, which = lane >> 3;
    const int p = seq.ctx - seq.n + i;
    const int2 range = row_range(a, seq, i);
    float q[N], o[N];
    {
        const char* row = a.q + static_cast<int64_t>(seq.first + i) * a.q_stride + (head * D + part * N) * 2;
        #pragma unroll
        for (int e = 0; e < N; ++e) {
            q[e] = __half2float(reinterpret_cast<const __half*>(row)[e]);
            o[e] = 0.f;
        }
    }
    const float slope = a.slopes ? a.slopes[head] : 0.f;
    const int64_t tile_bytes = static_cast<int64_t>(a.B) * kRowBytes<D, POOL>;
    float m = -CUDART_INF_F, l = 0.f;
    #pragma unroll 1
    for (int j0 = range.x; j0 < range.y; j0 += 4) {
        const int j = j0 + which;
        const bool seen = j < range.y;
        float x[N], dot = 0.f;
        int blk = 0;
        int64_t tile = 0;
        if (seen) {
            blk = query_block(a, s, j);
            tile = (static_cast<int64_t>(blk) * a.H + head / a.G) * tile_bytes;
            load_eighth<D, POOL, false>(a.kpool + tile, j & (a.B - 1), part, x);
            #pragma unroll
            for (int e = 0; e < N; ++e) dot = fmaf(q[e], x[e], dot);
        }
        #pragma unroll
        for (int k = 1; k < 8; k *= 2) dot += __shfl_xor_sync(0xffffffffu, dot, k);
        if (!seen) continue;
        float t = dot * a.scale;
        if constexpr (POOL == KV_FP8_E4M3) t *= a.kscale[blk];
        if (a.cap > 0.f) t = a.cap * tanhf(t / a.cap);
        if (a.slopes) t = fmaf(-slope, static_cast<float>(abs(p - j)), t);
        t *= kLog2e;
        const float to = fmaxf(m, t), base = to == -CUDART_INF_F ? 0.f : to;
        const float keep = ex2_approx(m - base);
        float w = ex2_approx(t - base);
        m = to;
        l = fmaf(l, keep, w);
        load_eighth<D, POOL, true>(a.vpool + tile, j & (a.B - 1), part, x);
        if constexpr (POOL == KV_FP8_E4M3) w *= a.vscale[blk];
        #pragma unroll
        for (int e = 0; e < N; ++e) o[e] = fmaf(w, x[e], o[e] * keep);
    }
    #pragma unroll
    for (int k = 8; k < 32; k *= 2) {
        const float other = __shfl_xor_sync(0xffffffffu, m, k);
        const float to = fmaxf(m, other), base = to == -CUDART_INF_F ? 0.f : to;
        const float mine = ex2_approx(m - base), theirs = ex2_approx(other - base);
        l = l * mine + __shfl_xor_sync(0xffffffffu, l, k) * theirs;
        #pragma unroll
        for (int e = 0; e < N; ++e) o[e] = o[e] * mine + __shfl_xor_sync(0xffffffffu, o[e], k) * theirs;
        m = to;
    }
    if (which != 0) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    char* row = a.out + static_cast<int64_t>(seq.first + i) * a.out_stride + (head * D + part * N) * 2;
    #pragma unroll
    for (int e = 0; e < N; ++e) reinterpret_cast<__half*>(row)[e] = __float2half_rn(o[e] * inv);
}

#endif  // __CUDACC__

// Rows of a unit (sequence, K/V head) that one 16-row matrix product holds: the few-row kernel's.
constexpr int kFewRows = 16;
constexpr int kFewSeqs = 1024;         // sequences per launch of it

// The kernels' launchers.
int launch_query_prompt(const kv_pool* pool, int layer, const QueryArgs& a, bool pdl, cudaStream_t stream);
size_t few_space(const kv_pool* pool, size_t* counters);       // workspace bytes, those of its counters (at its start)
int launch_query_few(const kv_pool* pool, const QueryArgs& a, void* workspace, bool pdl, cudaStream_t stream);

}  // namespace kvp
