// Decode attention over 4-bit pools (KV_INT4): the same result, work items, split-context merge
// and launch flags as attention_kernel.cuh, with a consumer made for 4-bit tiles.
//
// Per 16 tokens and K/V head, with the tokens (and the output's elements) as the M side of
// mma.m16n8k16 and the query heads as its N side:
//   S^T  = K Q^T        A = K expanded in registers, B = the query rows
//   softmax             fp32, log2 domain, the base raised only when the weights would leave float16
//   O^T += V^T P^T      A = V^T expanded in registers, B = P^T from the S accumulators
//                       (movmatrix)
// The weights enter as two float16 terms, value and rounding error (p = hi + lo), so P V is as exact
// as with float32 weights.  Up to 4 query heads per K/V head take the even columns and the odd column
// beside each holds the errors, at no further mma; 8 query heads fill all columns and the errors are
// a second mma into the same sums (37.0 us for 32 x 4096 tokens of 64 / 8 heads; with one term, off by
// 2^-11, 33.3).  All sums are float32.
//
// Every warp works alone: it goes through its own range, copies its chunks with cp.async into two stages of
// its own in shared memory and multiplies them, with no producer warp and no barrier.  (A 16-token tile of
// one head is 1152 bytes, and every bulk copy costs the SM 80-100 cycles whatever its size; a
// 16-byte cp.async per lane moves 512 bytes of a warp's own choosing.)  The tile layout (int4.cuh)
// makes a lane's fragments of 8 tokens the 16 bytes that the same lane copied.
//
// Work: the launch's chunks of 32 tokens, over all (sequence, head) units one after the other (each
// unit counting kUnitCost chunks more), are cut into equal ranges, one per warp, neighbouring
// ranges in one CTA, so every warp ends at the same time whatever the lengths.  A range holds the
// end of one unit, whole units, and the start of another.  A CTA joins the parts of its warps in
// shared memory; what crosses CTAs goes through (m, l, o) parts in the workspace, merged by the
// CTA that finishes last, in two levels when there are more than kMergeFan.  (Items of at most P
// tokens claimed one by one, as in attention_kernel.cuh, cost 2.4 us of a warp each here, against
// 1.7 us per chunk: a claim's and the queries' round trips, the fence before the ticket.)

#include "attention_kernel.cuh"
#include "int4.cuh"
#include "pool_types.cuh"

namespace kvp {
namespace {

// Warps of a CTA, one CTA per SM: four for each scheduler.  (8 query heads hold two columns of state per
// lane and fit 128 registers with 20 bytes spilled, 8 with head size 64; 12 warps with 160: 178 us for 192
// sequences of 64 / 8 heads where 16 take 174.)
constexpr int kWarps = 16;
// Query rows of the next item staged beside the stages, copied with its first chunk.  With 8 query heads
// there is no room: the first item's rows use the LATER part's place before it is written, and the
// others', asked into L2 with the item's block ids, are read from there.
template <int G> constexpr bool kStageQ = G < 8;
constexpr int kUnitCost = 2;                       // chunks that beginning and ending a unit costs a warp
// Tokens per chunk, one softmax update: 4608 bytes of K and V whatever the head size.  (Head size 64
// with 32-token chunks pays the loop's fixed part twice per byte: 0.74 of the copy peak where 64 give 0.81.)
constexpr int chunk_tokens(int head_dim) { return head_dim == 64 ? 64 : 32; }
template <int D> constexpr int kOcts = chunk_tokens(D) / 8;

// An item: a unit's part inside a warp's range.
struct __align__(16) ItemSlot {
    int s, h, oct0, lo;                                // sequence, head, first oct, rows before the window
    int first, last, kind, pad;                        // positions of the unit's first and last chunk; its kind
};
// whole unit; a part of a unit that began in an earlier range; the start of one that goes on
enum : int { WHOLE = 0, LATER = 1, START = 2 };

// A part that a warp holds for its CTA: the unit (-1: none) and its first and last chunk.
struct __align__(16) Held { int u, first, last, pad; };

// One warp's stage: the chunk's K codes, V codes, then their scales, oct by oct.
template <int D> struct Stage {
    static constexpr int CODES = Int4<D>::CODES, SCALES = D / 2;       // bytes per oct
    static constexpr int OCTS = kOcts<D>, V = OCTS * CODES, S = 2 * V;
    static constexpr int BYTES = S + 2 * OCTS * SCALES;
    static_assert(32 % OCTS == 0, "a chunk's octs lie in one window of 32 oct ids");
};

// Dynamic shared memory, per warp: two stages (at the end the START part's rows), the next item's
// query rows (kStageQ), two item slots (this item, the next), what is held (LATER, START), their (m, l) and
// the LATER part's rows.
template <int D, int G> struct Smem {
    static constexpr int RING = 2 * Stage<D>::BYTES, QBYTES = kStageQ<G> ? G * D * 2 : 0;
    static constexpr int Q = RING, SLOTS = Q + QBYTES, HELD = SLOTS + 2 * (int)sizeof(ItemSlot);
    static constexpr int ML = HELD + 2 * (int)sizeof(Held), ROWS = (ML + 2 * G * 8 + 15) / 16 * 16;
    static constexpr int WARP = ROWS + G * D * 4;
    static constexpr int BYTES = kWarps * WARP;
    static_assert(WARP % 16 == 0 && G * D * 4 <= RING, "16-byte alignment; a part fits the stages");
};

__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// mma_16816 with a zero accumulator
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

template <int WORDS> struct Words { uint32_t w[WORDS]; };
template <int WORDS>
__device__ __forceinline__ Words<WORDS> lds_words(const char* p) {
    Words<WORDS> x;
    if constexpr (WORDS == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        x.w[0] = v.x; x.w[1] = v.y; x.w[2] = v.z; x.w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        x.w[0] = v.x; x.w[1] = v.y;
    }
    return x;
}

// what the float16 pair `rounded` of (a, b) leaves of them, as a float16 pair
__device__ __forceinline__ uint32_t rounding_errors(uint32_t rounded, float a, float b) {
    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&rounded));
    return pack_half2(a - h.x, b - h.y);
}

// byte b0 (bits 0-7) and b1 (bits 8-15) of x as the float16 pair (scale b0, scale b1)
__device__ __forceinline__ uint32_t scales_two(uint32_t x) { return __byte_perm(x, 0, 0x4140) << 7; }
// The newest token of (sequence, head): quantised by the warp (4 elements per lane) into its slot,
// before the item's loads.
template <int D>
__device__ __forceinline__ void append_row(const char* src, int in_bytes, char* oct, int token, bool is_k, int lane) {
    const bool act = lane < D / 4;
    const int e0 = act ? lane * 4 : 0;
    float x[4];
    #pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = in_bytes == 2 ? __half2float(reinterpret_cast<const __half*>(src)[e0 + i])
                             : reinterpret_cast<const float*>(src)[e0 + i];
    float amax = max_nan(max_nan(fabsf(x[0]), fabsf(x[1])), max_nan(fabsf(x[2]), fabsf(x[3])));
    amax = max_nan(amax, __shfl_xor_sync(FULL, amax, 1));
    amax = max_nan(amax, __shfl_xor_sync(FULL, amax, 2));          // the 4 lanes of a group of 16
    const uint32_t sb = int4_scale_byte(amax);
    const uint32_t piece = int4_nibbles<4>(x, amax, int4_scale_value(sb));
    if (act) {
        *reinterpret_cast<uint16_t*>(oct + (is_k ? int4_k_code<D>(token, e0) : int4_v_piece<D>(token, e0))) =
            static_cast<uint16_t>(piece);
        if ((lane & 3) == 0)
            *reinterpret_cast<uint8_t*>(oct + (is_k ? int4_k_scale<D>(token, e0) : int4_v_scale<D>(token, e0))) =
                static_cast<uint8_t>(sb);
    }
}

// Maxima (the m of parts too) are kept in raw sums: only their differences, which are exact where it matters,
// are multiplied by the scale, so no score overflows.

// What the kernel needs beside AttnArgs.  A unit that crosses CTAs b0 .. b1 has its part of CTA b in
// workspace slot b0 + b, slots 2 b0 .. b0 + b1 of its own: the next one that crosses begins in CTA b1 at
// the earliest, at slot 2 b1.  Its counters go by its first slot.
struct Int4Args {
    AttnArgs a;
    int min_range;         // chunks per range, at least
    unsigned* done;        // [slots] parts, or groups of them, finished of the unit that starts at a slot
    unsigned* group_done;  // [slots] parts finished of the group of kMergeFan that starts at a slot
};

// Lane `sub`'s elements of one row of D, in float4s LPR apart.
template <int V> struct RowAcc {
    float m, l;
    float4 o[V];
};

template <int LPR, int V>
__device__ __forceinline__ void store_out(const AttnArgs& a, int64_t row, int D, const RowAcc<V>& x, int sub) {
    const float inv = 1.f / x.l;
    const int64_t at = row * (D / 4) + sub;
    #pragma unroll
    for (int i = 0; i < V; ++i) {
        const float4 v = make_float4(x.o[i].x * inv, x.o[i].y * inv, x.o[i].z * inv, x.o[i].w * inv);
        if (a.out_f16) {                               // rounded once, from the float32 result
            const __half2 lo = __floats2half2_rn(v.x, v.y), hi = __floats2half2_rn(v.z, v.w);
            uint2 w;
            w.x = *reinterpret_cast<const unsigned*>(&lo);
            w.y = *reinterpret_cast<const unsigned*>(&hi);
            static_cast<uint2*>(a.out)[at + i * LPR] = w;
        } else {
            static_cast<float4*>(a.out)[at + i * LPR] = v;
        }
    }
}

// The parts of one unit that warps w0, w0 + 1, ... of this CTA hold (w0's of kind `kind`, then
// LATER ones), joined by one warp, all G rows at once.
template <int D, int G>
__device__ __forceinline__ void join_parts(const AttnArgs& a, char* smem, int w0, int kind, int n, int u, bool whole,
                                           int slot, float xs, int lane) {
    using Sm = Smem<D, G>;
    constexpr int LPR = 32 / G < D / 4 ? 32 / G : D / 4, V = D / 4 / LPR;
    constexpr int NM = (kWarps + LPR - 1) / LPR;    // parts' (m, l) per lane: part i * LPR + sub
    const int sub = lane % LPR, r = lane / LPR < G ? lane / LPR : G - 1;
    float2 ml[NM];
    RowAcc<V> x;
    x.m = -CUDART_INF_F;
    x.l = 0.f;
    #pragma unroll
    for (int i = 0; i < NM; ++i) {
        const int k = i * LPR + sub, kd = k == 0 ? kind : LATER;
        ml[i] = k < n ? *reinterpret_cast<const float2*>(smem + (w0 + k) * Sm::WARP + Sm::ML + ((kd - 1) * G + r) * 8)
                      : make_float2(-CUDART_INF_F, 0.f);
        x.m = fmaxf(x.m, ml[i].x);
    }
    #pragma unroll
    for (int o = LPR / 2; o; o >>= 1) x.m = fmaxf(x.m, __shfl_xor_sync(FULL, x.m, o));
    #pragma unroll
    for (int i = 0; i < NM; ++i) {
        ml[i].x = ex2_approx((ml[i].x - x.m) * xs);           // the part's weight, 0 past the end
        x.l = fmaf(ml[i].y, ml[i].x, x.l);
    }
    #pragma unroll
    for (int o = LPR / 2; o; o >>= 1) x.l += __shfl_xor_sync(FULL, x.l, o);
    #pragma unroll
    for (int i = 0; i < V; ++i) x.o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    #pragma unroll
    for (int i = 0; i < NM; ++i) {
        #pragma unroll 4
        for (int j = 0; j < LPR; ++j) {
            const int k = i * LPR + j;
            if (k >= n) break;
            const float w = __shfl_sync(FULL, ml[i].x, lane - sub + j);
            const char* base = smem + (w0 + k) * Sm::WARP + (k == 0 && kind == START ? 0 : Sm::ROWS) + r * D * 4;
            #pragma unroll
            for (int e = 0; e < V; ++e) {
                const float4 o = reinterpret_cast<const float4*>(base)[sub + e * LPR];
                x.o[e].x = fmaf(w, o.x, x.o[e].x);
                x.o[e].y = fmaf(w, o.y, x.o[e].y);
                x.o[e].z = fmaf(w, o.z, x.o[e].z);
                x.o[e].w = fmaf(w, o.w, x.o[e].w);
            }
        }
    }
    if (lane / LPR >= G) return;
    if (whole) {
        store_out<LPR, V>(a, static_cast<int64_t>(u) * G + r, D, x, sub);
    } else {
        const int64_t row = static_cast<int64_t>(slot) * G + r;
        if (sub == 0) reinterpret_cast<float2*>(a.part_ml)[row] = make_float2(x.m, x.l);
        #pragma unroll
        for (int i = 0; i < V; ++i) reinterpret_cast<float4*>(a.part_o + row * D)[sub + i * LPR] = x.o[i];
    }
}

// Row r of the `count` parts `stride` slots apart from `slot` on, by one warp, read through L2 (they
// were written by other SMs): into the output (`last`), else into the first part's slot.
template <int D, int G>
__device__ __forceinline__ void merge_row(const AttnArgs& a, int64_t slot, int count, int stride, int64_t u, int r, bool last,
                                          float xs, int lane) {
    constexpr int LPR = D / 4;
    const int sub = lane % LPR;                        // D 64: both half-warps do the same
    const int64_t row = slot * G + r, step = static_cast<int64_t>(stride) * G;
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + row;
    float4* po = reinterpret_cast<float4*>(a.part_o + row * D) + sub;
    // lane j holds part j's (m, l) of each 32, which arrive together with the first parts' rows: a unit
    // of few parts costs one round trip
    constexpr int AHEAD = 8;
    RowAcc<1> x;
    x.m = -CUDART_INF_F;
    x.l = 0.f;
    x.o[0] = make_float4(0.f, 0.f, 0.f, 0.f);
    #pragma unroll 1
    for (int k0 = 0; k0 < count; k0 += 32) {
        const int n = min(32, count - k0);
        const float2 v = lane < n ? __ldcg(ml + (k0 + lane) * step) : make_float2(-CUDART_INF_F, 0.f);
        float4 rows[AHEAD];
        auto fetch = [&](int k) {
            #pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                if (k + i < n) rows[i] = __ldcg(po + (k0 + k + i) * step * (D / 4));
        };
        fetch(0);
        const float mx = fmaxf(x.m, warp_max(v.x)), old = ex2_approx((x.m - mx) * xs);
        const float w = ex2_approx((v.x - mx) * xs);          // 0 past the end
        x.m = mx;
        x.l = fmaf(x.l, old, warp_sum(v.y * w));
        x.o[0] = make_float4(x.o[0].x * old, x.o[0].y * old, x.o[0].z * old, x.o[0].w * old);
        #pragma unroll 1
        for (int k = 0; k < n; k += AHEAD) {
            #pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                if (k + i >= n) break;
                const float f = __shfl_sync(FULL, w, k + i);
                x.o[0].x = fmaf(f, rows[i].x, x.o[0].x);
                x.o[0].y = fmaf(f, rows[i].y, x.o[0].y);
                x.o[0].z = fmaf(f, rows[i].z, x.o[0].z);
                x.o[0].w = fmaf(f, rows[i].w, x.o[0].w);
            }
            fetch(k + AHEAD);
        }
    }
    __syncwarp();                                      // every lane has read the first part
    if (lane >= LPR) return;
    if (last) {
        store_out<LPR, 1>(a, u * G + r, D, x, sub);
    } else {
        if (sub == 0) reinterpret_cast<float2*>(a.part_ml)[row] = make_float2(x.m, x.l);
        po[0] = x.o[0];
    }
}

// The CTA's parts of up to two units that cross CTAs (cross[i]: unit, first and last CTA) are in the
// workspace: count them, and merge what they complete, a warp per row.  Called by every thread.
template <int D, int G>
__device__ __forceinline__ void finish_parts(const Int4Args& x, const Held* cross, float xs, int* s_go) {
    const AttnArgs& a = x.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto parts_of = [&](int i) { return cross[i].u < 0 ? 0 : cross[i].last - cross[i].first + 1; };
    const int most = max(parts_of(0), parts_of(1));
    if (most == 0) return;
    // Level 0 joins groups of kMergeFan parts into the group's first slot (units with more parts than
    // that), level 1 the unit's parts or groups into the output.
    #pragma unroll 1
    for (int level = most > kMergeFan ? 0 : 1; level < 2; ++level) {
        auto first_of = [&](int i) -> int {                // of the parts this CTA's part is counted with
            return level == 0 ? (blockIdx.x - cross[i].first) / kMergeFan * kMergeFan : 0;
        };
        auto count_of = [&](int i) -> int {
            const int parts = parts_of(i);
            if (level == 0) return parts > kMergeFan ? min(kMergeFan, parts - first_of(i)) : 0;
            return parts > kMergeFan ? (parts + kMergeFan - 1) / kMergeFan : parts;
        };
        __syncthreads();                               // every warp's rows are written
        if (warp < 2 && lane == 0) {
            const int of = count_of(warp);
            const bool before = level == 1 && most > kMergeFan ? s_go[warp] != 0 : true;
            bool go = before;
            if (of > 0 && before) {
                const int at = 2 * cross[warp].first;
                unsigned* ctr = level == 0 ? x.group_done + at + first_of(warp) : x.done + at;
                go = atom_add_acq_rel_gpu(ctr, 1u) == static_cast<unsigned>(of - 1);
                if (go) *ctr = 0;                      // left zero for the next call
            }
            s_go[warp] = go;                           // this CTA is the last
        }
        __syncthreads();
        for (int j = warp; j < 2 * G; j += kWarps) {
            const int i = j / G, of = count_of(i);
            if (of > 0 && s_go[i])
                merge_row<D, G>(a, 2 * cross[i].first + first_of(i), of,
                                level == 1 && parts_of(i) > kMergeFan ? kMergeFan : 1, cross[i].u, j % G, level == 1, xs,
                                lane);
        }
    }
}

template <int D, int G>
__global__ void __launch_bounds__(kWarps * 32, 1) attention_int4_kernel(const __grid_constant__ Int4Args args) {
    const AttnArgs& a = args.a;
    constexpr int WORDS = Int4<D>::WORDS, OCT = Int4<D>::OCT;
    constexpr int MT = D / 16;                         // output tiles of 16 elements
    constexpr bool SPLIT = G <= 4;                     // odd columns: the weights' rounding errors
    constexpr int NQ = SPLIT ? 1 : 2;                  // query columns per lane
    constexpr int CT = chunk_tokens(D), NO = kOcts<D>, NW = kWarps, NU = CT / 16;
    using St = Stage<D>;
    using Sm = Smem<D, G>;
    extern __shared__ __align__(128) char smem[];
    __shared__ int s_ctx[kMaxBatch], s_end[kMaxBatch];
    __shared__ Held s_cross[2];                        // the CTA's units that cross CTAs, with their CTAs
    __shared__ int s_go[2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;

    const bool early = a.early_tables != 0;
    if (!early) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (tid == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    if (tid < 2) s_cross[tid].u = -1;
    // ---- chunks per (sequence, head) and their inclusive prefix over the launch's units
    auto chunks_of = [&](int ctx) {
        const int n = ctx - attend_first(ctx, a.window, 8);
        // an empty sequence: one chunk without tokens (unsigned: a context may reach 2^31 - 1)
        return n > 0 ? static_cast<int>((static_cast<unsigned>(n) + CT - 1) / CT) : 1;
    };
    for (int s = tid; s < a.batch; s += NW * 32) {
        int c = a.lens[s];
        if (c < 0 || c > a.ctx_limit) {
            if (blockIdx.x == 0) atomicOr(a.err, KV_DEVERR_CONTEXT);
            c = c < 0 ? 0 : a.ctx_limit;
        }
        s_ctx[s] = c;
    }
    __syncthreads();
    if (warp == 0) {
        int carry = 0;
        for (int base = 0; base < a.batch; base += 32) {
            const int s = base + lane;
            int v = s < a.batch ? a.H * (chunks_of(s_ctx[s]) + kUnitCost) : 0;
            #pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int n = __shfl_up_sync(FULL, v, o);
                if (lane >= o) v += n;
            }
            v += carry;
            if (s < a.batch) s_end[s] = v;
            carry = __shfl_sync(FULL, v, 31);
        }
    }
    __syncthreads();
    const int total = s_end[a.batch - 1];
    // ranges: at most one per warp and of min_range chunks at least; k warps of every CTA have one.
    // The first `rem` ranges have q + 1 chunks, the others q.
    const int grid = static_cast<int>(gridDim.x);
    const int want = max(total / args.min_range, 1);
    // (a whole number of warps for each of the SM's four schedulers: 8 sequences of 64 / 8 heads take 18.1 us
    // with 14 warps of 4 chunks, 16.7 with 12 of 4.6)
    const int k0 = min((want + grid - 1) / grid, NW), k = k0 > 4 ? k0 & ~3 : k0;
    const int ranges = min(want, k * grid);
    const int q = total / ranges, rem = total - q * ranges;
    auto range_begin = [&](int r) { return r * q + min(r, rem); };
    auto range_of = [&](int chunk) {
        const int c = chunk - rem * (q + 1);
        return (c < 0 ? chunk : c) / (c < 0 ? q + 1 : q) + (c < 0 ? 0 : rem);
    };

    char* const ring = smem + warp * Sm::WARP;
    char* const s_q = ring + (kStageQ<G> ? Sm::Q : Sm::ROWS);          // (the first item's, before its rows)
    ItemSlot* const slots = reinterpret_cast<ItemSlot*>(ring + Sm::SLOTS);
    Held* const held = reinterpret_cast<Held*>(ring + Sm::HELD);
    if (lane < 2) held[lane].u = -1;
    const int opb = a.B >> 3;                          // octs per (block, head) tile
    const int lg_opb = __ffs(opb) - 1;

    // Global ids of octs o0 + lane (of n left) of an item; lanes past the end repeat the last.
    auto load_oids = [&](int s, int h, int o0, int n) -> int {
        const int o = o0 + min(lane, n - 1);
        int id = a.tables[static_cast<int64_t>(s) * a.max_blocks + (o >> lg_opb)];
        if (id < 0 || id >= a.num_blocks) {
            atomicOr(a.err, KV_DEVERR_BLOCK_ID);
            id = 0;
        }
        return ((id * a.H + h) << lg_opb) + (o & (opb - 1));
    };
    // Copy nt tokens (octs w .. of the id window) into a stage.  Octs past nt are not copied: what
    // the stage holds there is masked.
    constexpr int PPO = St::CODES / 16, SPO = St::SCALES / 16;         // 16-byte pieces of an oct: 32, 4 or 16, 2
    const char* const kbase = a.kpool + lane % PPO * 16;
    const char* const vbase = a.vpool + lane % PPO * 16;
    const char* const sbase = (lane < NO * SPO ? a.kpool : a.vpool) + St::CODES + lane % SPO * 16;
    const uint32_t ring32 = smem_u32(ring) + lane * 16;
    auto copy = [&](int stage, int oids, int w, int nt) {
        const uint32_t dst = ring32 + stage * St::BYTES;
        #pragma unroll
        for (int j = 0; j < NO * PPO / 32; ++j) {
            const int i = j * 32 / PPO + lane / PPO;
            const int64_t at = static_cast<int64_t>(__shfl_sync(FULL, oids, w + i)) * OCT;
            if (i * 8 < nt) {
                cp_async16(dst + j * 512, kbase + at);
                cp_async16(dst + St::V + j * 512, vbase + at);
            }
        }
        const int i = lane / SPO % NO;
        const int64_t at = static_cast<int64_t>(__shfl_sync(FULL, oids, w + i)) * OCT;
        if (lane < 2 * NO * SPO && i * 8 < nt) cp_async16(dst + St::S, sbase + at);
    };

    const int rng0 = min(static_cast<int>(blockIdx.x) * k, ranges);    // the CTA's ranges: rng0 .. rng0 + k - 1
    const int rng = rng0 + (warp < k ? warp : k);
    int pos = range_begin(min(rng, ranges));           // first chunk not yet taken
    const int end = warp < k ? range_begin(min(rng + 1, ranges)) : pos;
    const float xs = a.qscale;                         // raw sum (q . k) -> log2-domain score
    // Weights are 2^(score - base), the base between 7 and 15 below the running maximum: at most 2^15
    // in float16, and normal there down to 2^-21 of the largest.
    const float lift = fminf(7.f / xs, 4e29f), slack = fminf(15.f / xs, 1e30f);
    const int col = SPLIT ? g >> 1 : g;                // query of mma column g (odd columns of SPLIT: none)
    const bool has_q = !(SPLIT && (g & 1)) && col < G;
    float ot[MT][4];
    float m[NQ], l[NQ];
    uint32_t qa[2 * WORDS][2];                         // B fragments of Q^T

    // The loop runs one chunk ahead of itself: chunk c + 1 of the item (or chunk 0 of the next) is
    // copied while chunk c is multiplied.  It starts on an item without tokens or result.
    int ntok = 0, lo = 0, cur = 1, stage = 1;          // this item's tokens, masked rows, slot; the stage in use
    int oid = 0, oid_next = 0;                         // oct ids of the item's current and next 32 octs
    bool first_item = true;
    for (bool started = false;; started = true) {
        if (started) {
            // Query fragments in the order the K words expand: k-step 2w takes the even elements (0, 4)
            // and (2, 6) of word w, which meet a sixteenth of K, k-step 2w+1 the odd ones (1, 5) and
            // (3, 7), which meet K.  Each kind has sums of its own, so the queries stay as they are.
            cp_async_wait();                           // rows in shared memory came with the item's first chunk
            __syncwarp();
            const char* rows = s_q;
            if (!kStageQ<G> && !first_item)
                rows = static_cast<const char*>(a.q) + (static_cast<int64_t>(slots[cur].s) * a.H + slots[cur].h) * G * D * 2;
            #pragma unroll
            for (int w = 0; w < WORDS; ++w) {
                uint4 x = make_uint4(0, 0, 0, 0);
                if (has_q) x = *reinterpret_cast<const uint4*>(rows + (col * D + t * (D / 4) + 8 * w) * 2);
                qa[2 * w][0] = __byte_perm(x.x, x.z, 0x5410);
                qa[2 * w][1] = __byte_perm(x.y, x.w, 0x5410);
                qa[2 * w + 1][0] = __byte_perm(x.x, x.z, 0x7632);
                qa[2 * w + 1][1] = __byte_perm(x.y, x.w, 0x7632);
            }
            first_item = false;
            __syncwarp();                              // the next item's rows may follow now
            #pragma unroll
            for (int q = 0; q < NQ; ++q) { m[q] = -CUDART_INF_F; l[q] = 0.f; }
            #pragma unroll
            for (int i = 0; i < MT; ++i) { ot[i][0] = ot[i][1] = ot[i][2] = ot[i][3] = 0.f; }
        }
        int next_tok = -1, next_oid = 0, next_oid2 = 0;
        bool prepared = false;
        #pragma unroll 1
        for (int tok = 0;; tok += CT) {
            const int nt = ntok - tok;                 // tokens from this chunk on
            if (nt <= 2 * CT && !prepared) {
                // the item's last chunk but one: find the next item, fetch its oct ids and queries
                prepared = true;
                int s = 0, h = 0, ctx = 0, cps = 0, unit = 0, c0 = 0, n = 0;
                if (pos < end) {
                    int hi_s = a.batch - 1;            // first sequence that ends after pos
                    while (s < hi_s) {
                        const int mid = (s + hi_s) >> 1;
                        if (s_end[mid] > pos) hi_s = mid; else s = mid + 1;
                    }
                    ctx = s_ctx[s];
                    cps = chunks_of(ctx);
                    const int start = s ? s_end[s - 1] : 0;
                    h = (pos - start) / (cps + kUnitCost);
                    unit = start + h * (cps + kUnitCost) + kUnitCost;  // the unit's first chunk
                    c0 = max(pos - unit, 0);
                    n = min(cps - c0, end - unit - c0);                // <= 0: the range ends before that
                    pos = n > 0 ? unit + c0 + n : end;
                }
                if (n > 0) {
                    const int tok0 = attend_first(ctx, a.window, 8) + c0 * CT;
                    next_tok = max(min(n * CT, ctx - tok0), 0);
                    if (lane == 0) {
                        ItemSlot* it = slots + (cur ^ 1);
                        *reinterpret_cast<int4*>(&it->s) =
                            make_int4(s, h, tok0 >> 3, c0 == 0 ? attend_start(ctx, a.window) - tok0 : 0);
                        *reinterpret_cast<int4*>(&it->first) =
                            make_int4(unit, unit + cps - 1, c0 > 0 ? LATER : n < cps ? START : WHOLE, 0);
                    }
                    const int no = (next_tok + 7) >> 3;
                    if (no > 0) next_oid = load_oids(s, h, tok0 >> 3, no);
                    if (no > 32) next_oid2 = load_oids(s, h, (tok0 >> 3) + 32, no - 32);
                }
                if (!started && early) {               // lengths and tables came early; nothing else does
                    asm volatile("griddepcontrol.wait;" ::: "memory");
                    if (tid == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
                }
                if (n > 0) {
                    if (a.k_new != nullptr && c0 + n == cps && ctx > 0) {
                        // fused append: the newest token goes to its slot before the item's copies (a bad
                        // block id, flagged by load_oids, and a length that was clamped take none)
                        const int last = ctx - 1, o = last >> 3;
                        const int id = a.tables[static_cast<int64_t>(s) * a.max_blocks + (o >> lg_opb)];
                        if (id >= 0 && id < a.num_blocks && a.lens[s] == ctx) {
                            const int64_t to = (((static_cast<int64_t>(id) * a.H + h) << lg_opb) + (o & (opb - 1))) * OCT;
                            const int64_t row = (static_cast<int64_t>(s) * a.H + h) * D * a.in_bytes;
                            append_row<D>(a.k_new + row, a.in_bytes, a.kpool + to, last & 7, true, lane);
                            append_row<D>(a.v_new + row, a.in_bytes, a.vpool + to, last & 7, false, lane);
                        }
                        __syncwarp();                  // the copies below read the row
                    }
                    const char* q = static_cast<const char*>(a.q) + (static_cast<int64_t>(s) * a.H + h) * G * D * 2;
                    constexpr int QB = G * D * 2;
                    if (kStageQ<G> || !started) {
                        #pragma unroll
                        for (int i = 0; i < (QB / 16 + 31) / 32; ++i)
                            if (i * 32 + lane < QB / 16) cp_async16(smem_u32(s_q) + (i * 32 + lane) * 16, q + (i * 32 + lane) * 16);
                    } else if (lane < QB / 128) {
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(q + lane * 128));
                    }
                }
            }
            cp_async_wait();
            __syncwarp();                              // every lane's copies of this chunk have landed, and
                                                       // every lane is done with the other stage
            if (nt > CT) {
                const int w = (tok / CT + 1) * NO & 31;
                if (w == 0) {                          // the next 32 octs
                    oid = oid_next;
                    const int ahead = (tok + CT) / 8 + 32, no = (ntok + 7) >> 3;
                    if (ahead < no) oid_next = load_oids(slots[cur].s, slots[cur].h, slots[cur].oct0 + ahead, no - ahead);
                }
                copy(stage ^ 1, oid, w, nt - CT);
            } else if (next_tok > 0) {
                copy(stage ^ 1, next_oid, 0, next_tok);
            }
            if (nt > 0) {
                // this lane's words and scales of the stage
                const char* const pc = ring + stage * St::BYTES + lane * (4 * WORDS);
                const char* const pk = ring + stage * St::BYTES + St::S + (D == 128 ? lane * 2 : lane);
                const char* const pv = ring + stage * St::BYTES + St::S + NO * St::SCALES + (D == 128 ? g : g >> 1) * 8 + 2 * t;
                // ---- S^T = K Q^T, 16 tokens per mma
                float x[NU][2 * NQ];                   // [16 tokens][token g, token g + 8] (x query columns)
                #pragma unroll
                for (int u = 0; u < NU; ++u) {
                    const Words<WORDS> k0 = lds_words<WORDS>(pc + 2 * u * St::CODES);
                    const Words<WORDS> k1 = lds_words<WORDS>(pc + (2 * u + 1) * St::CODES);
                    uint32_t b0, b1;                   // the lane's scales of 16 elements: two, D 64: one
                    if constexpr (D == 128) {
                        b0 = *reinterpret_cast<const uint16_t*>(pk + 2 * u * St::SCALES);
                        b1 = *reinterpret_cast<const uint16_t*>(pk + (2 * u + 1) * St::SCALES);
                    } else {
                        b0 = *reinterpret_cast<const uint8_t*>(pk + 2 * u * St::SCALES);
                        b1 = *reinterpret_cast<const uint8_t*>(pk + (2 * u + 1) * St::SCALES);
                    }
                    const Int4Scale f0 = int4_scale_pair(scales_two(b0)), f1 = int4_scale_pair(scales_two(b1));
                    float even[4], odd[4];
                    #pragma unroll
                    for (int w = 0; w < WORDS; ++w) {
                        const Int4Scale s0 = int4_scale_of(f0, w / 2), s1 = int4_scale_of(f1, w / 2);
                        uint32_t p0[4], p1[4];
                        int4_expand(k0.w[w], s0, p0);
                        int4_expand(k1.w[w], s1, p1);
                        if (w == 0) {
                            mma_first(even, p0[0], p1[0], p0[2], p1[2], qa[0][0], qa[0][1]);
                            mma_first(odd, p0[1], p1[1], p0[3], p1[3], qa[1][0], qa[1][1]);
                        } else {
                            mma_16816(even, p0[0], p1[0], p0[2], p1[2], qa[2 * w][0], qa[2 * w][1]);
                            mma_16816(odd, p0[1], p1[1], p0[3], p1[3], qa[2 * w + 1][0], qa[2 * w + 1][1]);
                        }
                    }
                    #pragma unroll
                    for (int q = 0; q < NQ; ++q) {
                        x[u][q] = fmaf(even[q], 16.f, odd[q]);
                        x[u][NQ + q] = fmaf(even[2 + q], 16.f, odd[2 + q]);
                    }
                }
                const int first = tok == 0 ? lo : 0;
                if (nt < CT || first > 0) {            // rows outside [first, nt) may hold anything:
                    #pragma unroll                     // scores of -inf, and V scales of zero
                    for (int u = 0; u < NU; ++u) {
                        const int t0 = 16 * u + g, t1 = t0 + 8;
                        #pragma unroll
                        for (int q = 0; q < NQ; ++q) {
                            if (t0 < first || t0 >= nt) x[u][q] = -CUDART_INF_F;
                            if (t1 < first || t1 >= nt) x[u][NQ + q] = -CUDART_INF_F;
                        }
                    }
                    for (int r = lane; r < CT; r += 32) {
                        if (r >= first && r < nt) continue;
                        char* z = ring + stage * St::BYTES + St::S + (NO + r / 8) * St::SCALES + r % 8;
                        #pragma unroll
                        for (int i = 0; i < D / 16; ++i) z[8 * i] = 0;         // the token's D/16 scales
                    }
                    __syncwarp();
                }
                // ---- softmax over the chunk: m is the base, in raw sums
                #pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    float mx = fmaxf(x[0][q], x[0][NQ + q]);
                    #pragma unroll
                    for (int u = 1; u < NU; ++u) mx = fmaxf(mx, fmaxf(x[u][q], x[u][NQ + q]));
                    if (__any_sync(FULL, mx - m[q] > slack)) {       // (m + slack may round up to mx)
                        #pragma unroll
                        for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, o));
                        const float m_new = fmaxf(m[q], mx - lift), corr = ex2_approx((m[q] - m_new) * xs);
                        m[q] = m_new;
                        l[q] *= corr;
                        #pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            ot[i][q] *= corr;
                            ot[i][2 + q] *= corr;
                            if (SPLIT) { ot[i][1] *= corr; ot[i][3] *= corr; }
                        }
                    }
                }
                auto weight = [&](float v, int q) { return ex2_approx((v - m[q]) * xs); };
                #pragma unroll
                for (int u = 0; u < NU; ++u) {
                    // each weight as two float16 terms, the value and its rounding error: in the odd
                    // column beside it, or (8 query heads) in fragments of their own
                    uint32_t pb0, pb1, pr0 = 0, pr1 = 0;
                    if constexpr (SPLIT) {
                        const float p0 = weight(x[u][0], 0), p1 = weight(x[u][1], 0);
                        l[0] += p0 + p1;
                        const float h0 = __half2float(__float2half_rn(p0)), h1 = __half2float(__float2half_rn(p1));
                        pb0 = movmatrix_t(pack_half2(h0, p0 - h0));
                        pb1 = movmatrix_t(pack_half2(h1, p1 - h1));
                    } else {
                        const float p00 = weight(x[u][0], 0), p01 = weight(x[u][1], NQ - 1);
                        const float p10 = weight(x[u][NQ], 0), p11 = weight(x[u][2 * NQ - 1], NQ - 1);
                        l[0] += p00 + p10;
                        l[NQ - 1] += p01 + p11;
                        pb0 = pack_half2(p00, p01);
                        pb1 = pack_half2(p10, p11);
                        pr0 = movmatrix_t(rounding_errors(pb0, p00, p01));
                        pr1 = movmatrix_t(rounding_errors(pb1, p10, p11));
                        pb0 = movmatrix_t(pb0);
                        pb1 = movmatrix_t(pb1);
                    }
                    // ---- O^T += V^T P^T
                    const Words<WORDS> v0 = lds_words<WORDS>(pc + St::V + 2 * u * St::CODES);
                    const Words<WORDS> v1 = lds_words<WORDS>(pc + St::V + (2 * u + 1) * St::CODES);
                    const uint32_t b0 = *reinterpret_cast<const uint16_t*>(pv + 2 * u * St::SCALES);
                    const uint32_t b1 = *reinterpret_cast<const uint16_t*>(pv + (2 * u + 1) * St::SCALES);
                    const Int4Scale s0 = int4_scale_pair(scales_two(b0)), s1 = int4_scale_pair(scales_two(b1));
                    #pragma unroll
                    for (int w = 0; w < WORDS; ++w) {
                        uint32_t e0[4], e1[4];
                        int4_expand(v0.w[w], s0, e0);
                        int4_expand(v1.w[w], s1, e1);
                        mma_16816(ot[2 * w], e0[0], e0[1], e1[0], e1[1], pb0, pb1);
                        mma_16816(ot[2 * w + 1], e0[2], e0[3], e1[2], e1[3], pb0, pb1);
                        if constexpr (!SPLIT) {
                            mma_16816(ot[2 * w], e0[0], e0[1], e1[0], e1[1], pr0, pr1);
                            mma_16816(ot[2 * w + 1], e0[2], e0[3], e1[2], e1[3], pr0, pr1);
                        }
                    }
                }
            }
            stage ^= 1;
            if (nt <= CT) break;
        }
        if (started) {
            const ItemSlot it = slots[cur];
            const int u = it.s * a.H + it.h;
            #pragma unroll
            for (int q = 0; q < NQ; ++q) {
                #pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[q] += __shfl_xor_sync(FULL, l[q], o);
            }
            // a LATER part is kept beside the stages; a START part ends the warp's work, so the stages
            // (nothing is being copied into them) take it
            char* const keep = it.kind == START ? ring : ring + Sm::ROWS;
            __syncwarp();                              // every lane has read the last chunk
            #pragma unroll
            for (int q = 0; q < NQ; ++q) {
                const int query = SPLIT ? t : 2 * t + q;
                if (query >= G) continue;
                const float f = it.kind == WHOLE ? (ntok > 0 ? 1.f / l[q] : 0.f) : 1.f;
                // this lane: elements g*D/8 .. of its query; tile i holds elements 2i and 2i+1,
                // the even one as a sixteenth
                float o[2 * MT];
                #pragma unroll
                for (int i = 0; i < MT; ++i) {
                    o[2 * i] = (SPLIT ? ot[i][0] + ot[i][1] : ot[i][q]) * 16.f * f;
                    o[2 * i + 1] = (SPLIT ? ot[i][2] + ot[i][3] : ot[i][2 + q]) * f;
                }
                const int64_t row = static_cast<int64_t>(u) * G + query;
                if (it.kind == WHOLE && a.out_f16) {   // rounded once, from the float32 result
                    __half2* dst = reinterpret_cast<__half2*>(static_cast<__half*>(a.out) + row * D + g * (D / 8));
                    #pragma unroll
                    for (int i = 0; i < MT; ++i) dst[i] = __floats2half2_rn(o[2 * i], o[2 * i + 1]);
                    continue;
                }
                if (it.kind != WHOLE && g == 0)
                    *reinterpret_cast<float2*>(ring + Sm::ML + ((it.kind - 1) * G + query) * 8) = make_float2(m[q], l[q]);
                float4* dst = it.kind == WHOLE
                                  ? reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * D + g * (D / 8))
                                  : reinterpret_cast<float4*>(keep + query * D * 4 + g * (D / 2));
                #pragma unroll
                for (int i = 0; i < MT / 2; ++i)
                    dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
            if (it.kind != WHOLE && lane == 0)
                *reinterpret_cast<int4*>(held + it.kind - 1) = make_int4(u, it.first, it.last, 0);
        }
        if (next_tok < 0) break;
        cur ^= 1;
        __syncwarp();                                  // lane 0 wrote the slot
        ntok = next_tok;
        lo = slots[cur].lo;
        oid = next_oid;
        oid_next = next_oid2;
    }
    // ---- join the CTA's parts: a unit's parts lie with consecutive warps, the first START (or, of a
    // unit from an earlier CTA, warp 0's LATER), the others LATER
    __syncthreads();
    auto held_by = [&](int w, int kind) { return reinterpret_cast<const Held*>(smem + w * Sm::WARP + Sm::HELD) + kind - 1; };
    const int cta_begin = range_begin(rng0), cta_end = range_begin(min(rng0 + k, ranges));
    // Lane w knows what warp w holds.  A warp joins the unit that starts with it; warp 0's LATER unit goes
    // to the first other warp without one.
    const int later = lane < NW ? held_by(lane, LATER)->u : -1, starts = lane < NW ? held_by(lane, START)->u : -1;
    const unsigned idle = ~__ballot_sync(FULL, starts >= 0) & ((1u << NW) - 2u);
    const int helper = idle ? __ffs(idle) - 1 : 0;
    #pragma unroll 1
    for (int kind = START; kind >= (warp == helper ? LATER : START); --kind) {
        const int w0 = kind == START ? warp : 0;
        const Held h = *held_by(w0, kind);
        if (h.u < 0) continue;
        const int n = __ffs(~(__ballot_sync(FULL, later == h.u) >> (w0 + 1)));         // w0's and the LATER parts after it
        const bool whole = h.first >= cta_begin && h.last < cta_end;
        // at most one unit comes from an earlier CTA, and one that starts here goes on
        int slot = 0;
        if (!whole) {
            const int cta = range_of(lane == 0 ? h.first : h.last) / k;
            if (lane == 0) { s_cross[kind - 1].u = h.u; s_cross[kind - 1].first = cta; }
            if (lane == 1) s_cross[kind - 1].last = cta;
            slot = __shfl_sync(FULL, cta, 0) + static_cast<int>(blockIdx.x);
        }
        join_parts<D, G>(a, smem, w0, kind, n, h.u, whole, slot, xs, lane);
    }
    __syncthreads();
    finish_parts<D, G>(args, s_cross, xs, s_go);
}

template <int D, int G>
int launch_d(const kv_pool* pool, const Int4Args& args, const AttnPlan& plan, cudaStream_t stream) {
    static unsigned long long attr_done = 0;           // the shared-memory opt-in is per device
    const unsigned long long bit = 1ull << (pool->device & 63);
    if (!(attr_done & bit)) {
        if (cudaFuncSetAttribute(attention_int4_kernel<D, G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Smem<D, G>::BYTES) != cudaSuccess ||
            cudaFuncSetAttribute(attention_int4_kernel<D, G>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                 cudaSharedmemCarveoutMaxShared) != cudaSuccess) {
            cudaGetLastError();
            return KV_ERR_CUDA;
        }
        attr_done |= bit;
    }
    const AttnArgs& all = args.a;
    for (int s0 = 0; s0 < all.batch; s0 += kMaxBatch) {
        // launches of one call run one after the other on the stream and share the workspace, whose
        // counters each leaves zero; under programmatic dependent launch a launch writes nothing
        // before the one ahead of it has completed
        Int4Args x = args;
        AttnArgs& sa = x.a;
        sa.batch = all.batch - s0 < kMaxBatch ? all.batch - s0 : kMaxBatch;
        const int64_t rows = static_cast<int64_t>(s0) * all.H;         // units before this launch
        sa.q = static_cast<const char*>(all.q) + rows * G * D * 2;
        sa.out = static_cast<char*>(all.out) + rows * G * D * (all.out_f16 ? 2 : 4);
        sa.tables = all.tables + static_cast<int64_t>(s0) * all.max_blocks;
        sa.lens = all.lens + s0;
        if (all.k_new) {
            sa.k_new = all.k_new + rows * D * all.in_bytes;
            sa.v_new = all.v_new + rows * D * all.in_bytes;
        }
        // no more CTAs than ranges of the longest contexts the call allows
        const int64_t chunks = static_cast<int64_t>(sa.batch) * all.H * (plan.max_parts + kUnitCost);
        int64_t grid = chunks / args.min_range;
        const int64_t fit = static_cast<int64_t>(pool->num_sms);
        if (grid > fit) grid = fit;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(grid < 1 ? 1 : grid));
        cfg.blockDim = dim3(kWarps * 32);
        cfg.dynamicSmemBytes = Smem<D, G>::BYTES;
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = (plan.flags & KV_DECODE_PDL) ? 1 : 0;
        if (cudaLaunchKernelEx(&cfg, attention_int4_kernel<D, G>, x) != cudaSuccess) {
            cudaGetLastError();
            return KV_ERR_CUDA;
        }
    }
    return KV_OK;
}

template <int D>
int launch_g(int group, const kv_pool* pool, const Int4Args& x, const AttnPlan& plan, cudaStream_t stream) {
    switch (group) {
        case 1: return launch_d<D, 1>(pool, x, plan, stream);
        case 2: return launch_d<D, 2>(pool, x, plan, stream);
        case 4: return launch_d<D, 4>(pool, x, plan, stream);
        case 8: return launch_d<D, 8>(pool, x, plan, stream);
        default: return KV_ERR_INVALID_ARG;
    }
}

constexpr size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Workspace: the units' counters, the part groups' counters, (m, l), o; two slots per CTA, whatever the
// batch.
struct Layout {
    size_t groups, ml, o, end;
    Layout(const kv_pool* pool, int group) {
        const size_t slots = 2 * static_cast<size_t>(pool->num_sms);
        groups = align256(slots * 4);
        ml = 2 * groups;
        o = ml + align256(slots * group * 2 * sizeof(float));
        end = o + slots * group * pool->desc.head_dim * sizeof(float) + 256;
    }
};

// Units of the largest launch of a call.
int64_t units_of(const kv_pool* pool, int batch) {
    return static_cast<int64_t>(batch < kMaxBatch ? batch : kMaxBatch) * pool->desc.num_heads;
}

}  // namespace

// plan->partition: least chunks of a range; plan->max_parts: chunks of the longest context.
int plan_attention_int4(const kv_pool* pool, int batch, int max_context, int partition_tokens, AttnPlan* plan,
                        int group, int window) {
    const kv_pool_desc& d = pool->desc;
    if (batch < 0 || max_context < 0 || window < 0 || batch > KV_MAX_DECODE_BATCH) return KV_ERR_INVALID_ARG;
    if (!valid_group(d, group)) return KV_ERR_INVALID_ARG;
    if (partition_tokens < 0 || partition_tokens % kPartAlign != 0 || partition_tokens > (1 << 24))
        return KV_ERR_INVALID_ARG;
    const int chunk = chunk_tokens(d.head_dim);
    // a sliding window bounds the tokens read per sequence (window + up to 7 masked rows)
    const int64_t reach = static_cast<int64_t>(window) + 32;
    const int64_t span = window > 0 && reach < max_context ? reach : max_context;
    const int64_t chunks = span > 0 ? (span + chunk - 1) / chunk : 1;
    // the kernel numbers a launch's chunks with an int
    if (units_of(pool, batch) * (chunks + kUnitCost) >= (int64_t{1} << 31)) return KV_ERR_INVALID_ARG;
    // below 128 tokens a range costs more than it spreads (8 sequences of 64 / 8 heads, one context of 131072: 64
    // tokens 17.4, 18.6 us; 128: 16.7, 17.0; 256: 19.9, 17.4, and 7B-shaped 15.7 where 128 take 14.8)
    constexpr int kMinTokens = 128;
    *plan = AttnPlan{};
    plan->partition = partition_tokens ? (partition_tokens + chunk - 1) / chunk : kMinTokens / chunk;
    plan->max_parts = static_cast<int>(chunks);
    plan->group = group;
    plan->window = window;
    plan->ws_bytes = Layout(pool, group).end;
    return KV_OK;
}

int launch_attention_int4(const kv_pool* pool, int layer, const void* q, const void* k_new, const void* v_new,
                          int in_bytes, void* out, const int32_t* block_tables, int max_blocks,
                          const int32_t* context_lens, int batch, int max_context, float scale, const AttnPlan& plan,
                          void* workspace, cudaStream_t stream) {
    const kv_pool_desc& d = pool->desc;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return KV_ERR_CUDA;
    if (dev != pool->device) return KV_ERR_INVALID_ARG;
    if (batch == 0) return KV_OK;
    char* ws = static_cast<char*>(workspace);
    const Layout lay(pool, plan.group);
    if (!(plan.flags & KV_DECODE_WORKSPACE_ZEROED) && cudaMemsetAsync(ws, 0, lay.ml, stream) != cudaSuccess)
        return KV_ERR_CUDA;
    Int4Args x{};
    AttnArgs& a = x.a;
    a.kpool = static_cast<char*>(pool->k_layers[layer]);
    a.vpool = static_cast<char*>(pool->v_layers[layer]);
    a.k_new = static_cast<const char*>(k_new);
    a.v_new = static_cast<const char*>(v_new);
    a.in_bytes = in_bytes;
    a.q = q;
    a.out = out;
    a.tables = block_tables;
    a.lens = context_lens;
    x.done = reinterpret_cast<unsigned*>(ws);
    x.group_done = reinterpret_cast<unsigned*>(ws + lay.groups);
    a.part_ml = reinterpret_cast<float*>(ws + lay.ml);
    a.part_o = reinterpret_cast<float*>(ws + lay.o);
    x.min_range = plan.partition;
    a.err = pool->d_err;
    a.batch = batch;
    a.H = d.num_heads;
    a.B = d.block_size;
    a.max_blocks = max_blocks;
    const int64_t lim_tables = static_cast<int64_t>(max_blocks) * d.block_size;
    a.ctx_limit = static_cast<int>(lim_tables < max_context ? lim_tables : max_context);
    a.num_blocks = d.num_blocks;
    a.early_tables = (plan.flags & KV_DECODE_PDL) && (plan.flags & KV_DECODE_EARLY_TABLES) ? 1 : 0;
    a.out_f16 = (plan.flags & KV_DECODE_OUT_F16) ? 1 : 0;
    // log2(e): softmax evaluated with 2^x.  Held finite: two sums that differ at all do so by 2^-41 or
    // more, which times 3e38 leaves nothing of the smaller one's weight already.
    a.qscale = fminf(scale * 1.4426950408889634f, 3e38f);
    a.window = plan.window;
    return d.head_dim == 128 ? launch_g<128>(plan.group, pool, x, plan, stream)
                             : launch_g<64>(plan.group, pool, x, plan, stream);
}

}  // namespace kvp
