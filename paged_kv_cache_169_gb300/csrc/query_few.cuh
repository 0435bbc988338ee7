// paged_query_attention for few rows: at most 16 rows (tokens times query heads) of a K/V head, so the keys and
// values are read once for little work and the memory is what counts.
//
// The rows are the 16 rows of mma.m16n8k16 (empty ones are zero).  Every (sequence, K/V head) is a unit of
// 16-token chunks; the chunks of all units, one after the other (and what beginning and joining a unit costs), are
// cut into equal ranges, one per CTA and SM, so every SM works as long whatever the lengths.  A CTA's eight warps take
// a unit's chunks in turn, each through a ring of its own filled by cp.async (tokens that no row sees are filled with
// zeros and not read); the part of a unit in a CTA is joined in shared memory, and what crosses CTAs through the
// workspace by the CTA that finishes last, in two levels where there are more than kFan parts.  A short unit is one
// warp's, with nothing to join, and the others go on.  Softmax as in the tensor-core kernel.
//
// Bound.  The keys and values of a unit, read once.  Measured (us): 32 single tokens after 4095 of 64 / 8 heads, capped,
// float16 101 (5.3 TB/s, 0.78 of the copy rate); 8 single tokens after 512 .. 2047 of 32 heads, biased 33 (3.4 TB/s); 64
// sequences of five drafted tokens after 16 .. 16384, 16 / 8 heads, FP8 90 (2.7 TB/s); the 32 single tokens over FP8 91 and
// over 4-bit pools 102: fewer bytes, but more instructions.  What they lose: 15 to 20 us of a call's and its units' beginnings
// and joints (prefix of the weights 1, first chunks 2, a unit's start 2.4, a joint 2 to 2.5 each, the last one 3 to 4), and
// with FP8 about 600 instructions per 16 tokens that two warps per scheduler issue in 39% of the cycles.  Twelve warps, 168
// registers each, took the same time.
//
// A lane's mma operands come straight from the ring as it stores them, in whatever order of elements and tokens that
// gives (lane 4 g + t; the queries are loaded, and the result stored, in the same order):
//   float16  ldmatrix; elements and tokens in order
//   FP8      keys: the lane's D/4 codes from element t D/4 on; values: byte matrices transposed by ldmatrix, tokens 4 t ..
//            4 t + 3, so column c of the n-th eight keys is token 4 (c / 2) + 2 n + c % 2
//   4-bit    keys: as FP8, a word's nibbles i and i + 4 side by side; values: elements g D/8 .. of tokens 2 t and
//            2 t + 1 side by side (the pool's own order), so column c of product n is element c D/8 + n
#pragma once

#include "query_attention.cuh"
#include "int4.cuh"

namespace kvp {

struct FewArgs {
    QueryArgs a;
    float2* part_ml;       // [2 * CTAs][16] of a part's rows: base in log2 units, sum of weights
    float* part_o;         // [2 * CTAs][16][D]
    unsigned *done, *group_done;       // [2 * CTAs] each: parts, or groups of them, finished; zero between calls
};

// Workspace of a launch with `ctas` CTAs.
struct FewSpace {
    size_t ml, o, bytes;
    FewSpace(int ctas, int d) {
        ml = (static_cast<size_t>(ctas) * 4 * sizeof(unsigned) + 255) / 256 * 256;
        o = ml + static_cast<size_t>(ctas) * 2 * kFewRows * sizeof(float2);
        bytes = o + static_cast<size_t>(ctas) * 2 * kFewRows * d * sizeof(float);
    }
};

namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kWarps = 8, kChunk = 16, kFan = 16;
constexpr int kLeastChunks = 16;       // of a CTA's range: two per warp
constexpr int kShort = 8;              // a unit of at most so many chunks is one warp's
// What a unit costs a CTA beside its chunks, in chunks: 2 us (queries, joining), where 16 tokens take 180 ns (float16).
template <kv_dtype POOL> constexpr int kUnitCost = POOL == KV_F16 ? 11 : POOL == KV_FP8_E4M3 ? 22 : 30;
constexpr int kShortCost = 2;

template <int D_, kv_dtype POOL_>
struct FewCfg {
    static constexpr int D = D_;
    static constexpr kv_dtype POOL = POOL_;
    static constexpr int ROW = kRowBytes<D, POOL>;
    static constexpr int RAW = kChunk * ROW;                   // bytes of a chunk's keys (or values) as stored
    static constexpr int META = POOL == KV_FP8_E4M3 ? 16 : 0;  // two blocks' key and value scales
    static constexpr int STAGE = 2 * RAW + META;
    static constexpr int PART = kFewRows * D * 4;              // a warp's part of a unit
    static constexpr bool OWN_PART = STAGE < PART;             // beside the ring; else where the last chunk was
    static constexpr int TABLES = 3 * kFewSeqs * 4 + kWarps * kFewRows * 8;
    static constexpr int FIT = (226 * 1024 - 1024 - TABLES) / kWarps;
    static constexpr int STAGES_FIT = (FIT - (OWN_PART ? PART : 0)) / STAGE;
    static constexpr int STAGES = STAGES_FIT > 8 ? 8 : STAGES_FIT;
    static constexpr int WARP = STAGES * STAGE + (OWN_PART ? PART : 0);
    static constexpr int ML_OFF = kWarps * WARP, SEQ_OFF = ML_OFF + kWarps * kFewRows * 8;
    static constexpr int SMEM = SEQ_OFF + 3 * kFewSeqs * 4;
    static_assert(STAGES >= 2 && STAGE % 16 == 0 && WARP % 16 == 0, "ring");
};

// 4 bytes global -> shared, or zeros (nothing is read)
__device__ __forceinline__ void cp_async4_or_zero(uint32_t dst, const void* src, bool read) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(read ? 4 : 0) : "memory");
}

// Positions [lo, hi) that some row of the sequence sees.
struct Span { int lo, hi; };
__device__ __forceinline__ Span seq_span(const QueryArgs& a, const QuerySeq& q) {
    Span r{1 << 30, 0};
    if (!a.ranges) {                                           // the first row's start, the last row's end
        const int2 first = row_range(a, q, 0), last = row_range(a, q, q.n - 1);
        if (last.x < last.y) {
            r.lo = first.x;                                    // (0 where the first rows lie before position 0)
            r.hi = last.y;
        }
        return r;
    }
    for (int i = 0; i < q.n; ++i) {
        const int2 x = row_range(a, q, i);
        if (x.x < x.y) {
            r.lo = min(r.lo, x.x);
            r.hi = max(r.hi, x.y);
        }
    }
    return r;
}

// Four elements of a row's result; whether they are finite.
template <int D>
__device__ __forceinline__ bool store_quarter(const QueryArgs& a, const QuerySeq& seq, int h, int row, int c4, float4 o, float l) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (l == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
    o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    const __half2 lo = __floats2half2_rn(o.x, o.y), hi = __floats2half2_rn(o.z, o.w);
    uint2 w;
    w.x = *reinterpret_cast<const uint32_t*>(&lo);
    w.y = *reinterpret_cast<const uint32_t*>(&hi);
    *reinterpret_cast<uint2*>(a.out + static_cast<int64_t>(seq.first + row / a.G) * a.out_stride +
                              (h * a.G + row % a.G) * (D * 2) + c4 * 8) = w;
    return fabsf(o.x) < CUDART_INF_F && fabsf(o.y) < CUDART_INF_F && fabsf(o.z) < CUDART_INF_F && fabsf(o.w) < CUDART_INF_F;
}

// Rows that came out not finite, by the whole CTA: a key or value that is not finite reaches, as 0 * NaN, rows that
// do not see it, so such a row is worked out again from the definition, which reads only what it sees.
template <int D, kv_dtype POOL>
__device__ __forceinline__ void redo_rows(const QueryArgs& a, int s, const QuerySeq& seq, int h, unsigned* s_odd) {
    const unsigned odd = *s_odd;
    __syncthreads();
    if (threadIdx.x == 0) *s_odd = 0;
    #pragma unroll 1
    for (int row = threadIdx.x >> 5; row < kFewRows; row += kWarps)
        if (odd >> row & 1) attend_row<D, POOL>(a, s, seq, row / a.G, h * a.G + row % a.G);
    __syncthreads();
}

template <int D, kv_dtype POOL>
__global__ void __launch_bounds__(kWarps * 32, 1) query_few_kernel(const __grid_constant__ FewArgs x) {
    using C = FewCfg<D, POOL>;
    extern __shared__ __align__(128) char smem[];
    __shared__ int s_part[kWarps];                             // bytes to a warp's part in shared memory, -1: none
    __shared__ int s_warp_sum[kWarps];
    __shared__ int s_go[2];
    // rows that came out not finite (two words: while a warp still looks at the first of the two units that a CTA joins
    // at the end, another marks rows of the second)
    __shared__ unsigned s_odd[2];
    const QueryArgs& a = x.a;
    int* const s_lo = reinterpret_cast<int*>(smem + C::SEQ_OFF);               // what the sequence's rows see
    int* const s_hi = s_lo + kFewSeqs;
    int* const s_end = s_hi + kFewSeqs;                                        // inclusive prefix of the units' weights
    // chunks of a unit of the sequence (lo > hi: no rows; lo == hi: rows that see nothing, one chunk)
    auto chunks_of = [&](int s) {
        return s_lo[s] > s_hi[s] ? 0 : max(1, (s_hi[s] - (s_lo[s] & -kChunk) + kChunk - 1) / kChunk);
    };
    float2* const s_ml = reinterpret_cast<float2*>(smem + C::ML_OFF);
    // what a unit costs beside its chunks; its weight in the ranges
    auto cost_of = [](int n) { return n > kShort ? kUnitCost<POOL> : kShortCost; };
    auto weight_of = [&](int n) { return n > 0 ? n + cost_of(n) : 0; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- what every sequence's rows see, and the prefix of the weights of the launch's units
    {
        const int per = (a.batch + kWarps * 32 - 1) / (kWarps * 32);
        int sum = 0;
        for (int s = tid * per; s < min(a.batch, (tid + 1) * per); ++s) {
            const QuerySeq q = query_seq(a, s, blockIdx.x == 0);
            s_lo[s] = q.n > 0 ? 0 : 1;
            s_hi[s] = 0;
            if (q.n > 0) {
                const Span sp = seq_span(a, q);
                if (sp.lo < sp.hi) {
                    s_lo[s] = sp.lo;
                    s_hi[s] = sp.hi;
                }
            }
            sum += weight_of(chunks_of(s)) * a.H;
        }
        int upto = sum;
        #pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int v = __shfl_up_sync(FULL, upto, o);
            if (lane >= o) upto += v;
        }
        if (lane == 31) s_warp_sum[warp] = upto;
        if (tid < 2) s_odd[tid] = 0;
        __syncthreads();
        int before = upto - sum;
        for (int w = 0; w < warp; ++w) before += s_warp_sum[w];
        for (int s = tid * per; s < min(a.batch, (tid + 1) * per); ++s) {
            before += weight_of(chunks_of(s)) * a.H;
            s_end[s] = before;
        }
        __syncthreads();
    }
    const int total = s_end[a.batch - 1];
    const int ctas = min(static_cast<int>(gridDim.x), (total + kLeastChunks - 1) / kLeastChunks);
    const int cta = blockIdx.x;
    if (cta >= ctas) return;
    auto range_at = [&](int b) { return static_cast<int>(static_cast<int64_t>(total) * b / ctas); };
    const int g0 = range_at(cta), g1 = range_at(cta + 1);
    // the CTA whose range holds weight k
    auto cta_of = [&](int k) {
        int b = static_cast<int>(static_cast<int64_t>(k) * ctas / total);
        while (range_at(b + 1) <= k) ++b;
        while (range_at(b) > k) --b;
        return b;
    };

    // A unit: sequence, head, its chunks, its start among the weights; the chunks [c0, c1) of it that are this CTA's.
    struct Unit { int s, h, n, at, c0, c1; };
    auto in_range = [&](Unit& u) {
        const int first = u.at + cost_of(u.n);
        u.c0 = max(0, g0 - first);
        u.c1 = min(u.n, g1 - first);
    };
    auto first_unit = [&]() {
        int lo = 0, hi = a.batch - 1;                          // the first sequence that ends after g0
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (s_end[mid] > g0) hi = mid; else lo = mid + 1;
        }
        Unit u;
        u.s = lo;
        u.n = chunks_of(lo);
        const int w = weight_of(u.n), start = s_end[lo] - w * a.H;
        u.h = (g0 - start) / w;
        u.at = start + u.h * w;
        in_range(u);
        return u;
    };
    auto next_unit = [&](Unit& u) {                            // false: no chunk of it is this CTA's
        u.at += weight_of(u.n);
        if (u.at + kShortCost >= min(g1, total)) return false;
        if (++u.h == a.H) {
            u.h = 0;
            do u.n = chunks_of(++u.s); while (u.n == 0);
        }
        in_range(u);
        return u.c0 < u.c1;
    };
    auto is_short = [&](const Unit& u) { return u.n <= kShort && u.c0 == 0 && u.c1 == u.n; };

    // ---- filling the ring
    char* const ring = smem + warp * C::WARP;
    const uint32_t ring32 = smem_u32(ring);
    int fill_slot = 0, fill_no = 0, fill_c = 0;                // the stage to fill; the unit's number in the CTA; its chunk
    bool filling = true;
    Unit fill = first_unit();
    auto first_chunk = [&](const Unit& u, int no) {            // of this warp
        return is_short(u) ? ((no & (kWarps - 1)) == warp ? 0 : u.c1) : u.c0 + ((warp + no) & (kWarps - 1));
    };
    auto to_chunk = [&]() {                                    // on to the next chunk that there is
        while (filling && fill_c >= fill.c1) {
            filling = next_unit(fill);
            ++fill_no;
            if (filling) fill_c = first_chunk(fill, fill_no);
        }
    };
    // the physical blocks of the chunk's 8-token halves, -1: not read; as the table has them, loaded a chunk ahead
    // and looked at when they are used (at once, every chunk waited 700 cycles for each)
    int ids[2];
    bool used[2] = {false, false};
    auto look_up = [&]() {
        used[0] = used[1] = false;
        if (!filling) return;
        const int lo = s_lo[fill.s], hi = s_hi[fill.s], j0 = (lo & -kChunk) + fill_c * kChunk;
        #pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int first = max(j0 + 8 * i, lo);
            used[i] = first < min(j0 + 8 * i + 8, hi);
            if (used[i]) ids[i] = a.tables[static_cast<int64_t>(fill.s) * a.max_blocks + (first >> a.log_b)];
        }
    };
    auto ask = [&]() {
        if (filling) {
            const int lo = s_lo[fill.s], hi = s_hi[fill.s], j0 = (lo & -kChunk) + fill_c * kChunk;
            const uint32_t st = ring32 + fill_slot * C::STAGE;
            #pragma unroll
            for (int i = 0; i < 2; ++i) ids[i] = used[i] ? checked_block(a, ids[i]) : -1;
            if constexpr (POOL == KV_INT4) {
                constexpr int PIECES = Int4<D>::OCT / 16;      // of an oct: 8 tokens
                #pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int64_t from = ((static_cast<int64_t>(max(ids[i], 0)) * a.H + fill.h) * (a.B >> 3) +
                                          ((j0 + 8 * i) & (a.B - 1)) / 8) * Int4<D>::OCT;
                    for (int u = lane; u < 2 * PIECES; u += 32) {
                        const bool v = u >= PIECES;
                        const int e = v ? u - PIECES : u;
                        cp_async16_or_zero(st + (v ? C::RAW : 0) + i * Int4<D>::OCT + e * 16, (v ? a.vpool : a.kpool) + from + e * 16,
                                           ids[i] >= 0);
                    }
                }
            } else {
                constexpr int PIECES = C::ROW / 16, STEP = 32 / PIECES;        // of a token; tokens per instruction
                const int e = lane % PIECES, r = lane / PIECES;
                // rows of 128 bytes or more: pieces swizzled by the row; of 64 bytes: by pairs of rows
                auto place = [&](int row) {
                    return row * C::ROW + ((C::ROW >= 128 ? e ^ (row & 7) : e ^ (row >> 1 & 3)) << 4);
                };
                auto half_at = [&](int i) {                    // this lane's first byte of the i-th 8 tokens in the pool
                    return ((static_cast<int64_t>(max(ids[i], 0)) * a.H + fill.h) * a.B + ((j0 + 8 * i) & (a.B - 1)) + (r & 7)) * C::ROW + e * 16;
                };
                if (ids[0] >= 0 && ids[1] >= 0 && j0 >= lo && j0 + kChunk <= hi) {
                    int64_t at[2] = {half_at(0), half_at(1)};
                    #pragma unroll
                    for (int r0 = 0; r0 < kChunk; r0 += STEP) {
                        // (STEP rows at a time of one half, or both halves at once: 16 rows)
                        const int64_t from = STEP == 16 ? (r < 8 ? at[0] : at[1]) : at[r0 >> 3] + (r0 & 7) * C::ROW;
                        cp_async16(st + place(r0 + r), a.kpool + from);
                        cp_async16(st + C::RAW + place(r0 + r), a.vpool + from);
                    }
                } else {
                    #pragma unroll 1
                    for (int r0 = 0; r0 < kChunk; r0 += STEP) {
                        const int row = r0 + r, j = j0 + row;
                        const int id = row < 8 ? ids[0] : ids[1];
                        const bool read = id >= 0 && j >= lo && j < hi;
                        const int64_t from = read ? ((static_cast<int64_t>(id) * a.H + fill.h) * a.B + (j & (a.B - 1))) * C::ROW + e * 16 : 0;
                        cp_async16_or_zero(st + place(row), a.kpool + from, read);
                        cp_async16_or_zero(st + C::RAW + place(row), a.vpool + from, read);
                    }
                }
                if constexpr (POOL == KV_FP8_E4M3) {
                    if (lane < 4) {                            // key scales of the halves, then value scales
                        const int id = lane & 1 ? ids[1] : ids[0];
                        cp_async4_or_zero(st + 2 * C::RAW + lane * 4, (lane < 2 ? a.kscale : a.vscale) + max(id, 0), id >= 0);
                    }
                }
            }
            fill_slot = fill_slot + 1 == C::STAGES ? 0 : fill_slot + 1;
            fill_c += is_short(fill) ? 1 : kWarps;
            to_chunk();
            look_up();
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    filling = fill.c0 < fill.c1 || next_unit(fill);
    if (filling) fill_c = first_chunk(fill, 0);
    to_chunk();
    look_up();
    #pragma unroll 1
    for (int i = 0; i < C::STAGES; ++i) ask();

    // ---- the CTA's units
    const bool bias = a.slopes != nullptr, cap = a.cap > 0.f, large_cap = a.cap > kLargeCap;
    const float qscale = a.scale * kLog2e, c = cap || bias ? 1.f : qscale;
    const float k2 = cap ? 2.f * kLog2e * (a.scale / a.cap) : 0.f, capl = a.cap * kLog2e;
    struct Cross { int s, h, first, last; };                   // a unit that crosses CTAs: its first and last CTA
    Cross cross[2] = {{-1, 0, 0, 0}, {-1, 0, 0, 0}};           // one that began before this CTA, one that goes on after
    int slot = 0;                                              // the ring's stage to read next
    Unit unit = first_unit();
    bool some = unit.c0 < unit.c1 || next_unit(unit);
    #pragma unroll 1
    for (int no = 0; some; ++no, some = next_unit(unit)) {
        const bool alone = is_short(unit);                     // one warp's
        int k = first_chunk(unit, no);
        if (alone && k >= unit.c1) continue;
        const int to = unit.c1, step = alone ? 1 : kWarps;
        const QuerySeq seq = query_seq(a, unit.s, false);
        const int lo = s_lo[unit.s], hi = s_hi[unit.s], base = lo & -kChunk;
        const int rows = seq.n * a.G;
        // the next head's queries are on their way to the L2
        if ((alone || warp == 0) && unit.h + 1 < a.H && lane < rows * (D * 2) / 128) {
            const int row = lane * 128 / (D * 2);
            const char* at = a.q + static_cast<int64_t>(seq.first + row / a.G) * a.q_stride + ((unit.h + 1) * a.G + row % a.G) * (D * 2) +
                             lane * 128 % (D * 2);
            asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
        }
        int2 sees[2];
        int pos[2];
        float slope[2], m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};
        uint32_t q[D / 16][4];
        #pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = g + 8 * r, i = row / a.G, hq = unit.h * a.G + row % a.G;
            sees[r] = make_int2(0, 0);
            pos[r] = seq.ctx - seq.n + i;
            slope[r] = 0.f;
            const bool some = row < rows && k < to;            // (a warp without a chunk needs none of it)
            if (some) {
                sees[r] = row_range(a, seq, i);
                if (bias) slope[r] = a.slopes[hq] * kLog2e;
            }
            const char* qr = a.q + static_cast<int64_t>(seq.first + (some ? i : 0)) * a.q_stride + hq * (D * 2);
            if constexpr (POOL == KV_F16) {
                #pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    q[x][r] = some ? *reinterpret_cast<const uint32_t*>(qr + x * 32 + t * 4) : 0u;
                    q[x][r + 2] = some ? *reinterpret_cast<const uint32_t*>(qr + x * 32 + 16 + t * 4) : 0u;
                }
            } else {
                #pragma unroll
                for (int x = 0; x < D / 32; ++x) {             // 8 elements, two products
                    const uint4 v = some ? *reinterpret_cast<const uint4*>(qr + t * (D / 2) + x * 16) : make_uint4(0, 0, 0, 0);
                    if constexpr (POOL == KV_FP8_E4M3) {
                        q[2 * x][r] = v.x;
                        q[2 * x][r + 2] = v.y;
                        q[2 * x + 1][r] = v.z;
                        q[2 * x + 1][r + 2] = v.w;
                    } else {                                   // elements i and i + 4
                        q[2 * x][r] = __byte_perm(v.x, v.z, 0x5410);
                        q[2 * x][r + 2] = __byte_perm(v.x, v.z, 0x7632);
                        q[2 * x + 1][r] = __byte_perm(v.y, v.w, 0x5410);
                        q[2 * x + 1][r + 2] = __byte_perm(v.y, v.w, 0x7632);
                    }
                }
            }
        }
        // between these positions every row sees everything
        const int all_from = __reduce_max_sync(FULL, max(g < rows ? sees[0].x : 0, g + 8 < rows ? sees[1].x : 0));
        const int all_to = __reduce_min_sync(FULL, min(g < rows ? sees[0].y : 1 << 30, g + 8 < rows ? sees[1].y : 1 << 30));
        float o[D / 8][4];
        #pragma unroll
        for (int n = 0; n < D / 8; ++n)
            #pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
        int held = -1;                                         // the stage of this warp's last chunk here, not yet filled again
        #pragma unroll 1
        for (; k < to; k += step) {
            asm volatile("cp.async.wait_group %0;" ::"n"(C::STAGES - 1) : "memory");
            __syncwarp();
            const char* st = ring + slot * C::STAGE;
            const int j0 = base + k * kChunk;
            const uint32_t kt = ring32 + slot * C::STAGE, vt = kt + C::RAW;
            float ks = 1.f, vs = 1.f, lv = 0.f;                // FP8: the scales of this lane's keys, log2 of the values'
            if constexpr (POOL == KV_FP8_E4M3) {
                const float4 f = *reinterpret_cast<const float4*>(st + 2 * C::RAW);
                ks = t < 2 ? f.x : f.y;
                vs = t < 2 ? f.z : f.w;
                // (for the base only, so an approximate one does; see value_log2)
                lv = fminf(fmaxf(__log2f(fabsf(vs)), kLeastScale), kMostScale);
            }
            // ---- scores: 16 rows by two times 8 keys
            float sc[2][4];
            #pragma unroll
            for (int n = 0; n < 2; ++n) {
                #pragma unroll
                for (int e = 0; e < 4; ++e) sc[n][e] = 0.f;
                if constexpr (POOL == KV_F16) {
                    const int r = n * 8 + (lane & 7);
                    #pragma unroll
                    for (int x = 0; x < D / 32; ++x) {
                        uint32_t b[4];
                        ldsm_x4(kt + r * (D * 2) + (((x * 4 + (lane >> 3)) ^ (r & 7)) << 4), b);
                        mma_16816(sc[n], q[2 * x][0], q[2 * x][1], q[2 * x][2], q[2 * x][3], b[0], b[1]);
                        mma_16816(sc[n], q[2 * x + 1][0], q[2 * x + 1][1], q[2 * x + 1][2], q[2 * x + 1][3], b[2], b[3]);
                    }
                } else {
                    uint32_t w[D / 32][2];                     // 8 codes (FP8), or two words of 8 nibbles each
                    if constexpr (POOL == KV_FP8_E4M3) {
                        const int r = 4 * (g >> 1) + 2 * n + (g & 1);
                        #pragma unroll
                        for (int x = 0; x < D / 64; ++x) {
                            const int piece = t * (D / 64) + x;
                            const uint4 v = *reinterpret_cast<const uint4*>(
                                st + r * C::ROW + ((C::ROW >= 128 ? piece ^ (r & 7) : piece ^ (r >> 1 & 3)) << 4));
                            w[2 * x][0] = v.x; w[2 * x][1] = v.y; w[2 * x + 1][0] = v.z; w[2 * x + 1][1] = v.w;
                        }
                    }
                    if constexpr (POOL == KV_FP8_E4M3) {
                        #pragma unroll
                        for (int x = 0; x < D / 32; ++x) {
                            #pragma unroll
                            for (int y = 0; y < 2; ++y)
                                mma_16816(sc[n], q[2 * x + y][0], q[2 * x + y][1], q[2 * x + y][2], q[2 * x + y][3],
                                          e4m3x2_to_half2_bits(static_cast<uint16_t>(w[x][y])),
                                          e4m3x2_to_half2_bits(static_cast<uint16_t>(w[x][y] >> 16)));
                        }
                    } else {
                        const char* oct = st + n * Int4<D>::OCT;
                        uint32_t words[D / 32];
                        if constexpr (D == 128) {
                            const uint4 v = *reinterpret_cast<const uint4*>(oct + lane * 16);
                            words[0] = v.x; words[1] = v.y; words[2] = v.z; words[3] = v.w;
                        } else {
                            const uint2 v = *reinterpret_cast<const uint2*>(oct + lane * 8);
                            words[0] = v.x; words[1] = v.y;
                        }
                        // the scales of the lane's D/64 groups of 16
                        const uint32_t sb = D == 128 ? *reinterpret_cast<const uint16_t*>(oct + Int4<D>::CODES + lane * 2)
                                                     : *reinterpret_cast<const uint8_t*>(oct + Int4<D>::CODES + lane);
                        #pragma unroll
                        for (int x = 0; x < D / 32; ++x) {
                            const uint32_t s = x < 2 ? sb & 0xFFu : sb >> 8;
                            uint32_t p[4];
                            int4_expand_full(words[x], s << 7 | s << 23, p);
                            mma_16816(sc[n], q[2 * x][0], q[2 * x][1], q[2 * x][2], q[2 * x][3], p[0], p[1]);
                            mma_16816(sc[n], q[2 * x + 1][0], q[2 * x + 1][1], q[2 * x + 1][2], q[2 * x + 1][3], p[2], p[3]);
                        }
                    }
                }
            }
            const bool masked = j0 < all_from || j0 + kChunk > all_to;
            #pragma unroll
            for (int n = 0; n < 2; ++n)
                #pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = e >> 1, j = j0 + (POOL == KV_FP8_E4M3 ? 4 * t + 2 * n : n * 8 + 2 * t) + (e & 1);
                    float v = sc[n][e];
                    if constexpr (POOL == KV_FP8_E4M3) v *= ks;
                    if (cap) v = large_cap ? capped_large(v, qscale, k2, capl) : capped(v, k2, capl);
                    if (bias) v = fmaf(-slope[r], fabsf(static_cast<float>(pos[r] - j)), cap ? v : v * qscale);
                    v *= c;
                    sc[n][e] = !masked || (j >= sees[r].x && j < sees[r].y) ? v : -CUDART_INF_F;
                }
            // ---- the base follows the maximum only when it is left behind by more than 2^8
            float top[2];
            #pragma unroll
            for (int r = 0; r < 2; ++r)
                top[r] = fmaxf(fmaxf(sc[0][2 * r], sc[0][2 * r + 1]), fmaxf(sc[1][2 * r], sc[1][2 * r + 1])) + lv;
            if (__any_sync(FULL, top[0] - m[0] > kRaise || top[1] - m[1] > kRaise)) {
                #pragma unroll
                for (int r = 0; r < 2; ++r) {
                    top[r] = fmaxf(top[r], __shfl_xor_sync(FULL, top[r], 1));
                    top[r] = fmaxf(top[r], __shfl_xor_sync(FULL, top[r], 2));
                    if (top[r] - m[r] > kRaise) {
                        const float keep = ex2_approx(m[r] - top[r]);
                        m[r] = top[r];
                        l[r] *= keep;
                        #pragma unroll
                        for (int n = 0; n < D / 8; ++n) {
                            o[n][2 * r] *= keep;
                            o[n][2 * r + 1] *= keep;
                        }
                    }
                }
            }
            // ---- weights, their sums and the values
            uint32_t w[4];
            #pragma unroll
            for (int n = 0; n < 2; ++n)
                #pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float off = kLift - (m[r] == -CUDART_INF_F ? 0.f : m[r]);
                    float y0 = ex2_approx(sc[n][2 * r] + off), y1 = ex2_approx(sc[n][2 * r + 1] + off);
                    l[r] += y0 + y1;
                    if constexpr (POOL == KV_FP8_E4M3) {
                        y0 *= vs;
                        y1 *= vs;
                    }
                    const __half2 hv = __floats2half2_rn(y0, y1);
                    w[2 * n + r] = *reinterpret_cast<const uint32_t*>(&hv);
                }
            if constexpr (POOL == KV_F16) {
                const int vr = lane & 15;
                #pragma unroll
                for (int n = 0; n < D / 16; ++n) {
                    uint32_t b[4];
                    ldsm_x4_t(vt + vr * (D * 2) + (((2 * n + (lane >> 4)) ^ (vr & 7)) << 4), b);
                    mma_16816(o[2 * n], w[0], w[1], w[2], w[3], b[0], b[1]);
                    mma_16816(o[2 * n + 1], w[0], w[1], w[2], w[3], b[2], b[3]);
                }
            } else if constexpr (POOL == KV_FP8_E4M3) {
                const int vr = lane & 15;
                #pragma unroll
                for (int n = 0; n < D / 32; ++n) {             // two matrices of 16 tokens by 16 elements
                    uint32_t b[4];
                    const int piece = 2 * n + (lane >> 4);
                    ldsm_b8_x2_t(vt + vr * C::ROW + ((C::ROW >= 128 ? piece ^ (vr & 7) : piece ^ (vr >> 1 & 3)) << 4), b);
                    #pragma unroll
                    for (int y = 0; y < 4; ++y)
                        mma_16816(o[4 * n + y], w[0], w[1], w[2], w[3], e4m3x2_to_half2_bits(static_cast<uint16_t>(b[y])),
                                  e4m3x2_to_half2_bits(static_cast<uint16_t>(b[y] >> 16)));
                }
            } else {
                uint32_t words[2][D / 32], scales[2];
                #pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const char* oct = st + C::RAW + n * Int4<D>::OCT;
                    if constexpr (D == 128) {
                        const uint4 v = *reinterpret_cast<const uint4*>(oct + lane * 16);
                        words[n][0] = v.x; words[n][1] = v.y; words[n][2] = v.z; words[n][3] = v.w;
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2*>(oct + lane * 8);
                        words[n][0] = v.x; words[n][1] = v.y;
                    }
                    // tokens 2 t and 2 t + 1 of the lane's group; 0 where no row sees them (what lies there may be anything)
                    const uint32_t sb = *reinterpret_cast<const uint16_t*>(oct + Int4<D>::CODES + (D == 128 ? g : g >> 1) * 8 + 2 * t);
                    const int j = j0 + n * 8 + 2 * t;
                    scales[n] = (j >= lo && j < hi ? (sb & 0xFFu) << 7 : 0u) | (j + 1 >= lo && j + 1 < hi ? (sb & 0xFF00u) << 15 : 0u);
                }
                #pragma unroll
                for (int x = 0; x < D / 32; ++x) {
                    uint32_t p0[4], p1[4];
                    int4_expand_full(words[0][x], scales[0], p0);
                    int4_expand_full(words[1][x], scales[1], p1);
                    #pragma unroll
                    for (int y = 0; y < 4; ++y) mma_16816(o[4 * x + y], w[0], w[1], w[2], w[3], p0[y], p1[y]);
                }
            }
            held = slot;
            slot = slot + 1 == C::STAGES ? 0 : slot + 1;
            __syncwarp();                                      // every lane has read the stage
            if (alone || k + kWarps < to) ask();
        }
        if (alone) {                                           // to the output
            unsigned odd = 0;
            #pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[r] += __shfl_xor_sync(FULL, l[r], 1);
                l[r] += __shfl_xor_sync(FULL, l[r], 2);
                const int row = g + 8 * r;
                const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
                char* out = a.out + static_cast<int64_t>(seq.first + row / a.G) * a.out_stride + (unit.h * a.G + row % a.G) * (D * 2);
                bool finite = true;
                #pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    const int n0 = n & ~1;
                    float2 f = POOL != KV_INT4 ? make_float2(o[n][2 * r], o[n][2 * r + 1])
                                               : make_float2(o[n0][2 * r + (n & 1)], o[n0 + 1][2 * r + (n & 1)]);
                    f = l[r] == 0.f ? make_float2(0.f, 0.f) : make_float2(f.x * inv, f.y * inv);
                    finite &= fabsf(f.x) < CUDART_INF_F && fabsf(f.y) < CUDART_INF_F;
                    const int at = POOL != KV_INT4 ? 8 * n + 2 * t : (2 * t + (n & 1)) * (D / 8) + n0;
                    if (row < rows) *reinterpret_cast<__half2*>(out + at * 2) = __floats2half2_rn(f.x, f.y);
                }
                const unsigned not_finite = __ballot_sync(FULL, row < rows && !finite);
                #pragma unroll
                for (int e = 0; e < 8; ++e)                    // (lanes 4 e .. 4 e + 3: row e)
                    if (not_finite >> (4 * e) & 15u) odd |= 1u << (e + 8 * r);
            }
            #pragma unroll 1
            for (__syncwarp(); odd; odd &= odd - 1) {          // as redo_rows
                const int row = __ffs(odd) - 1;
                attend_row<D, POOL>(a, unit.s, seq, row / a.G, unit.h * a.G + row % a.G);
            }
            continue;
        }
        // ---- this warp's part, where its last chunk was
        const int part_at = warp * C::WARP + (C::OWN_PART ? C::STAGES : held) * C::STAGE;
        if (held >= 0) {
            char* const part = smem + part_at;
            #pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[r] += __shfl_xor_sync(FULL, l[r], 1);
                l[r] += __shfl_xor_sync(FULL, l[r], 2);
                const int row = g + 8 * r;
                if (row >= rows) continue;
                if (t == 0) s_ml[warp * kFewRows + row] = make_float2(m[r], l[r]);
                #pragma unroll
                for (int n = 0; n < D / 8; n += 2) {
                    if constexpr (POOL != KV_INT4) {
                        #pragma unroll
                        for (int y = n; y < n + 2; ++y)
                            *reinterpret_cast<float2*>(part + row * (D * 4) + (((2 * y + (t >> 1)) ^ (row & 7)) << 4) + (t & 1) * 8) =
                                make_float2(o[y][2 * r], o[y][2 * r + 1]);
                    } else if (n % 4 == 0) {
                        #pragma unroll
                        for (int y = 0; y < 2; ++y)
                            *reinterpret_cast<float4*>(part + row * (D * 4) + ((((2 * t + y) * (D / 32) + n / 4) ^ (row & 7)) << 4)) =
                                make_float4(o[n][2 * r + y], o[n + 1][2 * r + y], o[n + 2][2 * r + y], o[n + 3][2 * r + y]);
                    }
                }
            }
        }
        if (lane == 0) s_part[warp] = held >= 0 ? part_at : -1;
        __syncthreads();
        // ---- the CTA's part of the unit: to the output, or to the workspace
        const bool whole = unit.c0 == 0 && unit.c1 == unit.n;
        const int later = unit.c0 > 0 ? 0 : 1, space = 2 * cta + later;
        if (!whole) {
            const int first = unit.at + cost_of(unit.n);
            cross[later] = Cross{unit.s, unit.h, cta_of(first), cta_of(first + unit.n - 1)};
        }
        for (int e = tid; e < rows * (D / 4); e += kWarps * 32) {
            const int row = e / (D / 4), c4 = e % (D / 4);
            float mm = -CUDART_INF_F, ll = 0.f;
            #pragma unroll
            for (int v = 0; v < kWarps; ++v)
                if (s_part[v] >= 0) mm = fmaxf(mm, s_ml[v * kFewRows + row].x);
            const float off = mm == -CUDART_INF_F ? 0.f : mm;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            #pragma unroll
            for (int v = 0; v < kWarps; ++v) {
                if (s_part[v] < 0) continue;
                const float2 ml = s_ml[v * kFewRows + row];
                const float f = ex2_approx(ml.x - off);
                const float4 p = *reinterpret_cast<const float4*>(smem + s_part[v] + row * (D * 4) + ((c4 ^ (row & 7)) << 4));
                ll = fmaf(ml.y, f, ll);
                sum.x = fmaf(p.x, f, sum.x);
                sum.y = fmaf(p.y, f, sum.y);
                sum.z = fmaf(p.z, f, sum.z);
                sum.w = fmaf(p.w, f, sum.w);
            }
            if (whole) {
                if (!store_quarter<D>(a, seq, unit.h, row, c4, sum, ll)) atomicOr(&s_odd[0], 1u << row);
            } else {
                if (c4 == 0) x.part_ml[space * kFewRows + row] = make_float2(mm, ll);
                reinterpret_cast<float4*>(x.part_o)[(space * kFewRows + row) * (D / 4) + c4] = sum;
            }
        }
        __syncthreads();
        if (whole && s_odd[0]) redo_rows<D, POOL>(a, unit.s, seq, unit.h, &s_odd[0]);
        if (held >= 0) ask();                                  // into the held stage
    }
    asm volatile("cp.async.wait_all;" ::: "memory");

    // ---- units that cross CTAs: counted, and joined by the CTA that completes them
    auto parts_of = [&](int i) { return cross[i].s < 0 ? 0 : cross[i].last - cross[i].first + 1; };
    auto space_of = [&](int i, int b) { return 2 * b + (b == cross[i].first ? 1 : 0); };
    const int most = max(parts_of(0), parts_of(1));
    if (most == 0) return;
    #pragma unroll 1
    for (int level = most > kFan ? 0 : 1; level < 2; ++level) {
        // level 0: groups of kFan parts into the group's first place; level 1: the parts, or groups, into the output
        auto first_of = [&](int i) { return level == 0 ? cross[i].first + (cta - cross[i].first) / kFan * kFan : cross[i].first; };
        auto count_of = [&](int i) {
            const int parts = parts_of(i);
            if (level == 0) return parts > kFan ? min(kFan, cross[i].last + 1 - first_of(i)) : 0;
            return parts > kFan ? (parts + kFan - 1) / kFan : parts;
        };
        __threadfence();
        __syncthreads();                                       // every row of the CTA's parts is written
        if (warp < 2 && lane == 0) {
            const int n = count_of(warp);
            bool go = n > 0 && (level == 0 || parts_of(warp) <= kFan || s_go[warp]);
            if (go) {
                unsigned* ctr = (level == 0 ? x.group_done : x.done) + space_of(warp, first_of(warp));
                go = atom_add_acq_rel_gpu(ctr, 1u) == static_cast<unsigned>(n - 1);
                if (go) *ctr = 0;                              // left zero for the next call
            }
            s_go[warp] = go;
        }
        __syncthreads();
        #pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            if (!s_go[i] || count_of(i) == 0) continue;
            const int n = count_of(i), stride = level == 1 && parts_of(i) > kFan ? kFan : 1, b0 = first_of(i);
            const QuerySeq seq = query_seq(a, cross[i].s, false);
            const int rows = seq.n * a.G;
            for (int e = tid; e < rows * (D / 4); e += kWarps * 32) {
                const int row = e / (D / 4), c4 = e % (D / 4);
                float2 ml[kFan];
                float4 p[kFan];
                float mm = -CUDART_INF_F, ll = 0.f;
                #pragma unroll
                for (int v = 0; v < kFan; ++v) {
                    ml[v] = make_float2(-CUDART_INF_F, 0.f);
                    if (v < n) {
                        const int at_row = space_of(i, b0 + v * stride) * kFewRows + row;
                        ml[v] = __ldcg(x.part_ml + at_row);
                        p[v] = __ldcg(reinterpret_cast<const float4*>(x.part_o) + at_row * (D / 4) + c4);
                    }
                }
                #pragma unroll
                for (int v = 0; v < kFan; ++v) mm = fmaxf(mm, ml[v].x);
                const float off = mm == -CUDART_INF_F ? 0.f : mm;
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
                #pragma unroll
                for (int v = 0; v < kFan; ++v) {
                    if (v >= n) break;
                    const float f = ex2_approx(ml[v].x - off);
                    ll = fmaf(ml[v].y, f, ll);
                    sum.x = fmaf(p[v].x, f, sum.x);
                    sum.y = fmaf(p[v].y, f, sum.y);
                    sum.z = fmaf(p[v].z, f, sum.z);
                    sum.w = fmaf(p[v].w, f, sum.w);
                }
                if (level == 1) {
                    if (!store_quarter<D>(a, seq, cross[i].h, row, c4, sum, ll)) atomicOr(&s_odd[i], 1u << row);
                } else {
                    // (the group's first place: each thread replaces what it alone has read, but for (m, l))
                    const int at_row = space_of(i, b0) * kFewRows + row;
                    reinterpret_cast<float4*>(x.part_o)[at_row * (D / 4) + c4] = sum;
                    s_ml[i * kFewRows + row] = make_float2(mm, ll);
                }
            }
            __syncthreads();
            if (level == 0 && tid < rows) x.part_ml[space_of(i, b0) * kFewRows + tid] = s_ml[i * kFewRows + tid];
            if (level == 1 && s_odd[i]) redo_rows<D, POOL>(a, cross[i].s, seq, cross[i].h, &s_odd[i]);
        }
    }
}

template <typename C>
int launch_few_typed(const kv_pool* pool, const FewArgs& x, int ctas, bool pdl, cudaStream_t stream) {
    static unsigned long long attr_done = 0;               // the shared-memory opt-in is a per-device attribute
    const unsigned long long bit = 1ull << (pool->device & 63);
    if (!(attr_done & bit)) {
        if (cudaFuncSetAttribute(query_few_kernel<C::D, C::POOL>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
            cudaSuccess)
            return KV_ERR_CUDA;
        attr_done |= bit;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    for (int s0 = 0; s0 < x.a.batch; s0 += kFewSeqs) {
        FewArgs y = x;                                     // (rows of q and out are found through query_start)
        y.a.batch = x.a.batch - s0 < kFewSeqs ? x.a.batch - s0 : kFewSeqs;
        y.a.query_start += s0;
        y.a.lens += s0;
        y.a.tables += static_cast<int64_t>(s0) * x.a.max_blocks;
        cfg.gridDim = dim3(static_cast<unsigned>(ctas));
        if (cudaLaunchKernelEx(&cfg, query_few_kernel<C::D, C::POOL>, y) != cudaSuccess) {
            cudaGetLastError();
            return KV_ERR_CUDA;
        }
    }
    return KV_OK;
}

template <kv_dtype POOL>
int launch_few_pool(const kv_pool* pool, const FewArgs& x, int ctas, bool pdl, cudaStream_t stream) {
    return pool->desc.head_dim == 128 ? launch_few_typed<FewCfg<128, POOL>>(pool, x, ctas, pdl, stream)
                                      : launch_few_typed<FewCfg<64, POOL>>(pool, x, ctas, pdl, stream);
}

}  // namespace
}  // namespace kvp
