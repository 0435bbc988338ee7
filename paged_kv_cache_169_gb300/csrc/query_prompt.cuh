// paged_query_attention for many rows: the tensor-core kernel.
//
// Mathematics.  Rows are (token, query head) of a K/V head.  Over key tiles of 128 a row keeps a base m, the sum l of its
// weights and O: with t_j the masked scores in log2 units, w_j = 2^(t_j - m + 7) in float16, l += w_j, O += w_j v_j, and
// where a tile's maximum leaves m behind by more than 2^8 (rare after the first tile) m goes up and l and O by the
// difference down.  The result is O / l.  (FP8: t_j + log2 of v_j's scale s_j in place of t_j, so w_j is the weight times the
// scale, O += w_j times the codes, l += w_j / s_j.)
//
// Bound.  4 D operations per visible pair on the tensor cores; the special function unit makes an exponential a pair (a
// capped score an exponential and a quarter of a reciprocal more), 512 cycles of 128 x 128 pairs where the matrix products
// take 1024 (D = 128).
//
// Shape.  A work item is two row tiles of 128 rows (a token's G heads side by side) of one K/V head; a CTA per SM takes
// items from the grid as long as there are any.  Tensor memory holds two score tiles (the float16 weights go over them)
// and two O: 512 columns at D = 128, so a row tile's products and its softmax follow one another, and the two row tiles
// take turns.  Warps 0-15 softmax, 8 to a row tile, 16 rows each; 16 matrix products; 17 keys and values (TMA for float16
// pools, bulk copies and four widening warps for the others); 18 items and queries, an item ahead.
//
// Few items over long contexts are cut into parts of the keys (QueryArgs::splits): their sums go to the workspace in
// float32 and query_join_kernel joins them, in order.
//
// Measured (us; D = 128 but for the last): 4 x 2048 tokens of 40 heads 180 (955 TFLOP/s), 2 x 8192 of them 1003 (1370);
// 2 x 4096 tokens, 64 / 8 heads, capped 676 (733 with a cap above 64); 512 rows after 16k tokens in FP8, 4 x, 64 / 8 heads
// 1247 (856; 1210 with value scales relative to the item's largest, which cost other rows their bits); packed documents with
// a bias, 4-bit, 248; ragged prompts, D = 64, prefixes seen both ways 265 (550).  What it waits for: per key tile 1660 cycles
// of softmax and 1660 of products and barrier round trips one behind the other; an item's start and end 7000 cycles.
// Before: 8 softmax warps with 64-key steps 187, 768, 1540, 313, 267; store warps for the result and 128-key
// steps 211, 797, 1690, 284, 260; both row tiles' products issued as they came (the softmaxes ran at the same time, then
// the products) 190, 806, 1664, 236, 266; scores taken 64 columns at a time (more free registers, the base's loop spilt)
// 264, 1160, 2127, 285, 275.
#pragma once

#include <type_traits>

#include "query_attention.cuh"
#include "tcgen05.cuh"
#include "widen.cuh"

namespace kvp {

struct PromptArgs {
    CUtensorMap qmap;                  // [num_tokens][heads][D / 64][64], boxes of a row tile's 64-element halves
    CUtensorMap kmap, vmap;            // float16 pools: the layer's row maps, a block of one head per copy
    QueryArgs a;
    int items;                         // bound of the work items
};

int launch_query_prompt_fp8(const kv_pool* pool, const PromptArgs& p, bool pdl, cudaStream_t stream);
int launch_query_prompt_int4(const kv_pool* pool, const PromptArgs& p, bool pdl, cudaStream_t stream);

namespace {

constexpr int kTile = 128;             // rows of a row tile and keys of a key tile
constexpr int kSoftmaxWarps = 16, kMmaWarp = 16, kLoadWarp = 17, kItemWarp = 18, kWidenWarp = 20;      // (19: none)
constexpr int kFactorTiles = 8;        // key tiles whose FP8 scales are kept (more than are in flight)

template <int D_, kv_dtype POOL_>
struct PromptCfg {
    static constexpr int D = D_;
    static constexpr kv_dtype POOL = POOL_;
    static constexpr bool WIDEN = POOL != KV_F16;              // tiles are widened to float16 on their way
    // 64-element (128-byte) columns of a tile.  A key or value tile is [16 groups of 8 rows][HALVES][8][128 bytes], a
    // query tile [HALVES][128][128 bytes], both 128-byte swizzled.
    static constexpr int HALVES = D / 64;
    static constexpr int TILE = HALVES * kTile * 128;          // bytes of 128 rows as float16
    // key and value tiles in flight as float16, and as stored
    static constexpr int SLOTS = D == 128 ? (WIDEN ? 3 : 4) : 8;
    static constexpr int RAWS = WIDEN ? (D == 128 ? 2 : 4) : 0;
    static constexpr int RAW = WIDEN ? kTile * kRowBytes<D, POOL> : 0;
    // Registers: 96 (20 warps) or 80 (24 warps) per thread at launch, shared out by fours of warps
    static constexpr int WARPS = WIDEN ? 24 : 20;
    static constexpr int REGS_SOFTMAX = WIDEN ? 96 : 104, REGS_ISSUE = WIDEN ? 48 : 64, REGS_WIDEN = 48;
    static_assert(WIDEN ? 4 * REGS_SOFTMAX + REGS_ISSUE + REGS_WIDEN <= 6 * 80 : 4 * REGS_SOFTMAX + REGS_ISSUE <= 5 * 96, "registers");
    static constexpr int Q_OFF = 0, KV_OFF = 2 * TILE, RAW_OFF = KV_OFF + SLOTS * TILE;
    static constexpr int OUT_OFF = RAW_OFF + RAWS * RAW;       // 64 elements of a softmax warp's 16 rows on their way out
    static constexpr int FACTOR_OFF = OUT_OFF + kSoftmaxWarps * 16 * 128;
    static constexpr int FACTORS = POOL == KV_FP8_E4M3 ? kFactorTiles * 3 * 16 * 4 : 0;
    static constexpr int BAR_OFF = FACTOR_OFF + FACTORS;
    static constexpr int BARS = 2 * SLOTS + 2 * RAWS + 5 * 2 + 2 * 2 + 3;
    static constexpr int MISC_OFF = (BAR_OFF + BARS * 8 + 15) / 16 * 16;
    static constexpr int SMEM = MISC_OFF + 160 + 1024;         // and up to 1024 bytes of alignment
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(BAR_OFF % 16 == 0 && RAW % 16 == 0, "alignment");
};

template <int N> __device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Maximum of three.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// capped() of four with one reciprocal: 1/a = b (cd) / (ab cd) and so on, each factor below 2^30 + 1 (tanh is 1 long
// before).  Four multiplications and the reciprocal are off by 7 2^-24 together: t within 2^-20 of the cap
// (kLargeCap at most).  The special function unit makes 5 values for four scores where it made 8 (2 x 4096 capped tokens:
// 773 -> 700 us then).
__device__ __forceinline__ void capped4(float* x, float k2, float capl) {
    float2 y[2], a[2];
    #pragma unroll
    for (int i = 0; i < 2; ++i) {
        y[i] = __fmul2_rn(make_float2(x[2 * i], x[2 * i + 1]), make_float2(k2, k2));
        a[i] = __fadd2_rn(make_float2(ex2_approx(fminf(y[i].x, 30.f)), ex2_approx(fminf(y[i].y, 30.f))), make_float2(1.f, 1.f));
    }
    const float2 ab = __fmul2_rn(a[0], a[1]);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ab.x * ab.y));
    const float2 inv = make_float2(r * ab.y, r * ab.x);
    #pragma unroll
    for (int i = 0; i < 2; ++i) {
        float2 t = __ffma2_rn(__fmul2_rn(inv, a[1 - i]), make_float2(-2.f * capl, -2.f * capl), make_float2(capl, capl));
        t = __ffma2_rn(y[i], make_float2(0.f, 0.f), t);        // (a NaN, which the minimum has left out, of its own only)
        x[2 * i] = t.x;
        x[2 * i + 1] = t.y;
    }
}

// capped_large() of two scores below half the cap.
__device__ __forceinline__ float2 tanh_series2(float2 s, float sl, float k2) {
    auto both = [](float c) { return make_float2(c, c); };
    const float2 u = __fmul2_rn(s, both(k2)), z = __fmul2_rn(__fmul2_rn(u, u), both(kHalfLn2Sq)), x = __fmul2_rn(s, both(sl));
    float2 p = both(kTanh[0]);
    #pragma unroll
    for (int i = 1; i < 6; ++i) p = __ffma2_rn(p, z, both(kTanh[i]));
    return __ffma2_rn(__fmul2_rn(x, p), z, x);
}

// A place in a ring of N: how often it went round, too.
template <int N> struct Ring {
    int slot = 0, times = 0;
    __device__ __forceinline__ void advance() {
        if (++slot == N) {
            slot = 0;
            ++times;
        }
    }
};

// Byte offset of 16 bytes (8 elements, the ch-th of a row) in a key or value tile.
template <int HALVES>
__device__ __forceinline__ uint32_t tile_at(int r, int ch) {
    return (((r >> 3) * HALVES + (ch >> 3)) << 10) + ((r & 7) << 7) + (((ch & 7) ^ (r & 7)) << 4);
}

// The warp's first lane's value.  The compiler knows the result to be the same in every lane, so branches on it
// keep a warp together and operands made of it may be uniform registers, as the matrix instructions' must be.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// A bounded wait by a whole warp: all of its lanes go on, or none.  Eight seconds: a warp that works its 16 rows out again
// (attend_row: 0.36 us a position and row) lets the rest of its CTA wait, over 170 thousand positions for one second, over
// 1.4 million for eight.  (A limit from the context's length, read from the arguments, cost FP8 chunks 3%.)
constexpr uint64_t kPromptWaitNs = 8 * kWaitLimitNs;
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int* err) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, err, kPromptWaitNs));
}

// Key tiles [a, b) of each row tile, numbered from position `base`; the work item's are those that either row tile
// needs.  With a distance bias they are taken from the last one down: it lowers the scores on the way, and the softmax's
// base, once found, stays (upwards, steep heads raise it at every tile: 313 us against 250 for packed 4-bit documents).
// Without one upwards: the rows of a causal tile then find their base in the same tile (a 2048-token prompt took 5% longer
// downwards).
template <bool DOWN>
struct KeyTiles {
    int base, end, a0, b0, a1, b1, n;
    __device__ __forceinline__ int a(int t) const { return t ? a1 : a0; }
    __device__ __forceinline__ int b(int t) const { return t ? b1 : b0; }
    __device__ __forceinline__ bool on(int t, int j) const { return j >= a(t) && j < b(t); }
    __device__ __forceinline__ bool is(int j) const { return j >= 0 && j < n; }
    __device__ __forceinline__ int from(int j) const {         // j, or the first of the item's key tiles after it
        while (is(j) && !on(0, j) && !on(1, j)) j += DOWN ? -1 : 1;
        return j;
    }
    __device__ __forceinline__ int first() const { return from(DOWN ? n - 1 : 0); }
    __device__ __forceinline__ int next(int j) const { return from(DOWN ? j - 1 : j + 1); }
    __device__ __forceinline__ int below(int j) const {        // how many of them are less than j
        return max(0, min(b0, j) - a0) + max(0, min(b1, j) - a1) - max(0, min(min(b0, b1), j) - max(a0, a1));
    }
    __device__ __forceinline__ int tiles() const { return below(n); }
    __device__ __forceinline__ int before(int j) const { return DOWN ? tiles() - below(j + 1) : below(j); }
};

// A work item: a pair of row tiles of a (sequence, K/V head).  s < 0: there are no more.
struct Item {
    int s, head, token;                // its first token
    int first, n, ctx;                 // the sequence (QuerySeq)
    int lo[2], hi[2];                  // positions that some row of a row tile sees
    int z, from, to;                   // the part of the keys, and its positions
};
struct PromptMisc {
    uint4 claim;                       // the answer to a claim of the next item
    Item item[2];
    uint32_t tmem;
};
static_assert(sizeof(PromptMisc) <= 160, "PromptCfg::SMEM");

template <bool DOWN>
__device__ __forceinline__ KeyTiles<DOWN> key_tiles(const Item& x, int block) {
    KeyTiles<DOWN> k;
    k.base = min(x.lo[0], x.lo[1]) & -block;
    k.end = max(x.hi[0], x.hi[1]);
    auto from = [&](int t) { return x.lo[t] < x.hi[t] ? (x.lo[t] - k.base) / kTile : 0; };
    auto to = [&](int t) { return x.lo[t] < x.hi[t] ? (x.hi[t] - k.base + kTile - 1) / kTile : 0; };
    k.a0 = from(0);
    k.b0 = to(0);
    k.a1 = from(1);
    k.b1 = to(1);
    k.n = max(k.b0, k.b1);
    return k;
}

// Take over a CTA of this launch that has not begun: its index arrives in 16 bytes of shared memory.  (PTX ISA:
// clusterlaunchcontrol.  The grid is all items, and the CTAs that run take the others' places one by one.)
__device__ __forceinline__ void claim_item(uint32_t answer, uint32_t bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer),
                 "r"(bar) : "memory");
}
// The claimed CTA's index, -1: there was none left.
__device__ __forceinline__ int claimed_item(const uint4& v) {
    int x;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .b64 lo, hi;\n\t.reg .pred p;\n\t"
        "mov.b64 lo, {%1, %2};\n\tmov.b64 hi, {%3, %4};\n\tmov.b128 h, {lo, hi};\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "mov.b32 %0, -1;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, h;\n\t}"
        : "=&r"(x) : "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w));
    return x;
}

// CAP: none, up to kLargeCap, above it.
enum Cap : int { NO_CAP = 0, SMALL_CAP = 1, LARGE_CAP = 2 };

template <int D, kv_dtype POOL, bool BIAS, int CAP>
__global__ void __launch_bounds__(PromptCfg<D, POOL>::WARPS * 32, 1)
query_prompt_kernel(const __grid_constant__ PromptArgs p) {
    using C = PromptCfg<D, POOL>;
    extern __shared__ char smem_raw[];
    char* const smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
    const uint32_t base32 = smem_u32(smem);
    PromptMisc* const misc = reinterpret_cast<PromptMisc*>(smem + C::MISC_OFF);
    const QueryArgs& a = p.a;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    auto bar = [&](int i) { return base32 + C::BAR_OFF + 8 * i; };
    auto full = [&](int slot) { return bar(slot); };
    auto empty = [&](int slot) { return bar(C::SLOTS + slot); };
    auto raw_full = [&](int i) { return bar(2 * C::SLOTS + i); };
    auto raw_empty = [&](int i) { return bar(2 * C::SLOTS + C::RAWS + i); };
    constexpr int B0 = 2 * C::SLOTS + 2 * C::RAWS;
    auto q_there = [&](int t) { return bar(B0 + t); };         // a row tile's queries
    auto q_free = [&](int t) { return bar(B0 + 2 + t); };      // and their place
    auto s_there = [&](int t) { return bar(B0 + 4 + t); };     // its scores of a key tile
    auto w_there = [&](int t) { return bar(B0 + 6 + t); };     // its weights
    auto o_there = [&](int t) { return bar(B0 + 8 + t); };     // its sums after a key tile
    auto item_there = [&](int i) { return bar(B0 + 10 + i); };
    auto item_free = [&](int i) { return bar(B0 + 12 + i); };
    const uint32_t edge = bar(B0 + 14), done = bar(B0 + 15), claim = bar(B0 + 16);
    // FP8, per 8 tokens of a tile: 16 times (factor of the scores, log2 of the value scale), then 16 times 1 / value scale
    float* const factors = reinterpret_cast<float*>(smem + C::FACTOR_OFF);

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::SLOTS; ++i) {
            mbar_init(full(i), C::WIDEN ? 4 : 1);
            mbar_init(empty(i), 1);
        }
        for (int i = 0; i < C::RAWS; ++i) {
            mbar_init(raw_full(i), 1);
            mbar_init(raw_empty(i), 4);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(q_there(t), 1);
            mbar_init(q_free(t), 1);
            mbar_init(s_there(t), 1);
            mbar_init(w_there(t), 8);
            mbar_init(o_there(t), 1);
            mbar_init(item_there(t), 1);
            mbar_init(item_free(t), C::WARPS - 2);
        }
        mbar_init(edge, 1);
        mbar_init(done, 1);
        mbar_init(claim, 1);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) tmem_alloc(smem_u32(&misc->tmem));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tmem = uniform(misc->tmem);
    const int per_tile = kTile / a.G, log_g = __ffs(a.G) - 1;  // tokens of a row tile
    bool fine = true;                                          // no wait of this warp has run out
    int count = 0;                                             // items so far
    Item it;
    KeyTiles<BIAS> keys;
    auto wait = [&](uint32_t b, int times) {                   // for the barrier's times-th completion (from 0)
        fine = fine && warp_wait(b, times & 1, a.err);
        return fine;
    };
    // The next item, as uniform values; false: there is none.
    auto next_item = [&]() {
        const int i = count & 1;
        if (!wait(item_there(i), count >> 1)) return false;
        const Item& x = misc->item[i];
        it.s = uniform(x.s);
        it.head = uniform(x.head);
        it.token = uniform(x.token);
        it.first = uniform(x.first);
        it.n = uniform(x.n);
        it.ctx = uniform(x.ctx);
        #pragma unroll
        for (int t = 0; t < 2; ++t) {
            it.lo[t] = uniform(x.lo[t]);
            it.hi[t] = uniform(x.hi[t]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(item_free(i));
        ++count;
        keys = key_tiles<BIAS>(it, a.B);
        return it.s >= 0;
    };

    if (warp < kSoftmaxWarps) {
        // ======== softmax, 16 rows a warp; the result out.  Four lanes share two rows, r and r + 8 of the warp's, and have
        // columns 8 g + 2 (lane & 3) and the next one of each group g of 8: rows need no other warp.
        more_registers<C::REGS_SOFTMAX>();
        const int rt = warp >> 3, rows0 = (warp & 3) * 32 + (warp & 4) * 4, quad = lane & 3;
        const uint32_t lanes = static_cast<uint32_t>(rows0) << 16;
        const uint32_t st = tmem + lanes + rt * kTile, ot = tmem + lanes + 2 * kTile + rt * D;
        char* const own = smem + C::OUT_OFF + warp * (16 * 128);
        constexpr int DIR = BIAS ? -1 : 1;                     // of the key tiles
        const float qscale = a.scale * kLog2e;
        const float k2 = CAP ? 2.f * kLog2e * (a.scale / a.cap) : 0.f, capl = a.cap * kLog2e;
        const float c = CAP || BIAS || POOL == KV_FP8_E4M3 ? 1.f : qscale;     // scores to log2 units
        int i = 0, tiles = 0;                                  // this row tile's key tiles so far; the items'
        auto row_of = [&](int r) { return rows0 + (lane >> 2) + 8 * r; };
        // An item's part of this thread, taken while the last products of the item before are made.  (The rest stays in
        // shared memory until the result is out: registers are short here.)
        struct Part {
            int steps, j0;                                     // key tiles; the first one's position
            int2 sees[2];
            float slope[2];
            int pos0;                                          // the first row's position
            int tile;                                          // FP8: the first one's number
        } next;
        auto fetch = [&]() {
            if (!wait(item_there(count & 1), count >> 1)) return false;
            const Item& x = misc->item[count & 1];
            if (uniform(x.s) < 0) return false;
            const auto k = key_tiles<BIAS>(x, a.B);
            next.steps = uniform(k.b(rt) - k.a(rt));
            const int j = BIAS ? k.b(rt) - 1 : k.a(rt);
            next.j0 = uniform(k.base + j * kTile);
            if (POOL == KV_FP8_E4M3) next.tile = tiles + uniform(k.before(j));
            #pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int token = x.token + rt * per_tile + (row_of(r) >> log_g);
                int2 sees = token < x.n ? row_range(a, QuerySeq{x.first, x.n, x.ctx}, token) : make_int2(0, 0);
                sees = make_int2(max(sees.x, x.from), min(sees.y, x.to));
                next.sees[r] = sees.x < sees.y ? sees : make_int2(0, 0);
                next.slope[r] = BIAS ? a.slopes[x.head * a.G + (row_of(r) & (a.G - 1))] * kLog2e : 0.f;
            }
            next.pos0 = x.ctx - x.n + x.token + rt * per_tile;
            return true;
        };
        bool some_item = fetch();
        #pragma unroll 1
        while (some_item) {
            const Item& x0 = misc->item[count & 1];
            const int stop = i + next.steps, pos0 = next.pos0;
            int j0 = next.j0, tile = next.tile;
            const int2 sees[2] = {next.sees[0], next.sees[1]};
            const float slope[2] = {next.slope[0], next.slope[1]};
            float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};    // the base (log2 units), this thread's sum of weights
            const int i0 = i;
            #pragma unroll 1
            for (; i < stop; ++i, j0 += DIR * kTile) {
                if (!wait(s_there(rt), i)) break;
                tc_fence_after();
                float x[64];                                   // [group of 8 columns][row][2]
                uint32_t* const xr = reinterpret_cast<uint32_t*>(x);
                const float4* scales = nullptr;                // FP8
                tmem_load_16x64(st, xr);
                if constexpr (POOL != KV_FP8_E4M3) {
                    tmem_load_16x64(st + 64, xr + 32);
                    tmem_wait_load32(xr);
                    tmem_wait_load32(xr + 32);
                } else {
                    scales = reinterpret_cast<const float4*>(factors + tile++ % kFactorTiles * 48);
                    #pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        float4 f[4];
                        #pragma unroll
                        for (int k = 0; k < 4; ++k) f[k] = scales[4 * half + k];       // (beside the scores' way here)
                        tmem_wait_load32(xr + 32 * half);
                        if (half == 0) tmem_load_16x64(st + 64, xr + 32);
                        #pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float* const y = x + 32 * half + 2 * e;
                            const float of = e & 2 ? f[e >> 2].z : f[e >> 2].x, lv = e & 2 ? f[e >> 2].w : f[e >> 2].y;
                            const float2 at = make_float2(y[0], y[1]), by = make_float2(of, of);
                            const float2 s = CAP ? __fmul2_rn(at, by) : __ffma2_rn(at, by, make_float2(lv, lv));
                            y[0] = s.x;
                            y[1] = s.y;
                        }
                    }
                }
                if (CAP) {
                    if constexpr (CAP == SMALL_CAP) {
                        #pragma unroll
                        for (int k = 0; k < 64; k += 4) capped4(x + k, k2, capl);
                    } else {
                        // scores below half the cap, as most are below a large one, need no exponential
                        float top = 0.f;
                        #pragma unroll
                        for (int k = 0; k < 64; k += 2) top = max3(fabsf(x[k]), fabsf(x[k + 1]), top);
                        if (__any_sync(0xffffffffu, top * k2 >= kLog2e)) {
                            #pragma unroll
                            for (int k = 0; k < 64; ++k) x[k] = capped_large(x[k], qscale, k2, capl);
                        } else {
                            #pragma unroll
                            for (int k = 0; k < 64; k += 2) {
                                const float2 y = tanh_series2(make_float2(x[k], x[k + 1]), qscale, k2);
                                x[k] = y.x;
                                x[k + 1] = y.y;
                            }
                        }
                    }
                    if constexpr (POOL == KV_FP8_E4M3) {
                        #pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float4 v = scales[k];
                            #pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float* const y = x + 8 * k + 2 * e;
                                const float lv = e < 2 ? v.y : v.w;
                                const float2 s = __fadd2_rn(make_float2(y[0], y[1]), make_float2(lv, lv));
                                y[0] = s.x;
                                y[1] = s.y;
                            }
                        }
                    }
                }
                if (BIAS) {
                    const float mul = CAP || POOL == KV_FP8_E4M3 ? 1.f : qscale;
                    #pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float from = static_cast<float>(pos0 + (row_of(r) >> log_g) - j0 - 2 * quad);
                        #pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            float& y = x[(k >> 1) * 4 + 2 * r + (k & 1)];
                            y = fmaf(-slope[r], fabsf(from - static_cast<float>((k >> 1) * 8 + (k & 1))), y * mul);
                        }
                    }
                }
                if (__any_sync(0xffffffffu, max(sees[0].x, sees[1].x) > j0 || min(sees[0].y, sees[1].y) < j0 + kTile)) {
                    #pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int from = sees[r].x - j0 - 2 * quad;
                        const unsigned len = sees[r].y - sees[r].x;
                        #pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (static_cast<unsigned>((k >> 1) * 8 + (k & 1) - from) >= len)
                                x[(k >> 1) * 4 + 2 * r + (k & 1)] = -CUDART_INF_F;
                    }
                }
                float top[2];
                #pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float t0 = fmaxf(x[2 * r], x[2 * r + 1]), t1 = fmaxf(x[2 * r + 4], x[2 * r + 5]);
                    #pragma unroll
                    for (int g = 2; g < 16; g += 2) {
                        t0 = max3(x[4 * g + 2 * r], x[4 * g + 2 * r + 1], t0);
                        t1 = max3(x[4 * g + 2 * r + 4], x[4 * g + 2 * r + 5], t1);
                    }
                    top[r] = fmaxf(t0, t1);
                }
                #pragma unroll
                for (int k = 1; k < 4; k *= 2) {
                    top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], k));
                    top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], k));
                }
                // The base follows the maximum only when it is left behind by more than 2^8, which is rare after the
                // first tile.  (m -inf: it is, but for a row that sees nothing yet)
                if (__any_sync(0xffffffffu, top[0] * c - m[0] > kRaise || top[1] * c - m[1] > kRaise)) {
                    float keep[2] = {1.f, 1.f};
                    #pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        if (top[r] * c - m[r] > kRaise) {
                            keep[r] = ex2_approx(m[r] - top[r] * c);
                            m[r] = top[r] * c;
                            l[r] *= keep[r];
                        }
                    }
                    if (i > i0) {
                        if (!wait(o_there(rt), i - 1)) break;
                        tc_fence_after();
                        #pragma unroll 1
                        for (int k = 0; k < D; k += 16) {
                            uint32_t o[8];
                            tmem_load_16x16(ot + k, o);
                            #pragma unroll
                            for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep[e >> 1 & 1]);
                            tmem_store_16x16(ot + k, o);
                        }
                    }
                }
                // weights, and their sums
                const float2 c2 = make_float2(c, c);
                float2 sum[2];
                float4 vf;
                uint32_t w[32];
                #pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const int r = k & 1;
                    const float off = kLift - (m[r] == -CUDART_INF_F ? 0.f : m[r]);
                    float2 y = __ffma2_rn(make_float2(x[2 * k], x[2 * k + 1]), c2, make_float2(off, off));
                    y.x = ex2_approx(y.x);
                    y.y = ex2_approx(y.y);
                    if constexpr (POOL == KV_FP8_E4M3) {       // (y: the weight times its value scale)
                        if (k % 8 == 0) vf = scales[8 + k / 8];
                        const float f = k % 8 < 2 ? vf.x : k % 8 < 4 ? vf.y : k % 8 < 6 ? vf.z : vf.w;
                        sum[r] = k < 2 ? __fmul2_rn(y, make_float2(f, f)) : __ffma2_rn(y, make_float2(f, f), sum[r]);
                    } else {
                        sum[r] = k < 2 ? y : __fadd2_rn(sum[r], y);
                    }
                    const __half2 hv = __floats2half2_rn(y.x, y.y);
                    w[k] = *reinterpret_cast<const uint32_t*>(&hv);
                }
                tmem_store_16x64(st, w);
                tmem_wait_store();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(w_there(rt));
                l[0] += sum[0].x + sum[0].y;
                l[1] += sum[1].x + sum[1].y;
            }
            if (!fine) break;
            const Item it = x0;
            if (POOL == KV_FP8_E4M3) tiles += key_tiles<BIAS>(x0, a.B).tiles();
            __syncwarp();
            if (lane == 0) mbar_arrive(item_free(count & 1));
            ++count;
            #pragma unroll
            for (int k = 1; k < 4; k *= 2) {
                l[0] += __shfl_xor_sync(0xffffffffu, l[0], k);
                l[1] += __shfl_xor_sync(0xffffffffu, l[1], k);
            }
            some_item = fetch();
            if (!fine || (i > i0 && !wait(o_there(rt), i - 1))) break;
            tc_fence_after();
            const bool any = i > i0;
            if (a.splits > 1) {                                // a part of the rows' keys: to the workspace
                auto place = [&](int r, int token) {
                    const int64_t row = it.z * a.part_rows + part_row(a.part_by_sequence, a.max_queries, it.s, it.first, token);
                    return row * (a.H * a.G) + it.head * a.G + (row_of(r) & (a.G - 1));
                };
                #pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int token = it.token + rt * per_tile + (row_of(r) >> log_g);
                    const int64_t at = place(r, token);
                    if (token < it.n && quad == 0) a.part_ml[at] = any ? make_float2(m[r], l[r]) : make_float2(-CUDART_INF_F, 0.f);
                }
                #pragma unroll 1
                for (int k = 0; any && k < D; k += 16) {
                    uint32_t o[8];
                    tmem_load_16x16(ot + k, o);
                    #pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int token = it.token + rt * per_tile + (row_of(r) >> log_g);
                        if (token >= it.n) continue;
                        const int64_t at = place(r, token);
                        #pragma unroll
                        for (int g = 0; g < 2; ++g)
                            *reinterpret_cast<float2*>(a.part_o + at * D + k + 8 * g + 2 * quad) =
                                make_float2(__uint_as_float(o[4 * g + 2 * r]), __uint_as_float(o[4 * g + 2 * r + 1]));
                    }
                }
                tc_fence_before();
                continue;
            }
            // the result, 64 elements at a time through shared memory, so that a store writes whole lines
            const float inv[2] = {l[0] == 0.f ? 0.f : 1.f / l[0], l[1] == 0.f ? 0.f : 1.f / l[1]};
            char* const to = a.out + static_cast<int64_t>(it.first + it.token + rt * per_tile) * a.out_stride +
                             it.head * a.G * (D * 2) + (lane & 7) * 16;
            const int left = it.n - it.token - rt * per_tile;  // tokens of the row tile
            float2 odd[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};    // NaN: something was not finite
            #pragma unroll 1
            for (int half = 0; half < C::HALVES; ++half) {
                uint32_t o[32];                                // (without a key tile: whatever is there, not used)
                tmem_load_16x64(ot + half * 64, o);
                tmem_wait_load32(o);
                #pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const int r = k & 1, at = (lane >> 2) + 8 * r;
                    const float2 f = __fmul2_rn(make_float2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1])),
                                                make_float2(inv[r], inv[r]));
                    odd[r] = __ffma2_rn(f, make_float2(0.f, 0.f), odd[r]);
                    const __half2 hv = __floats2half2_rn(f.x, f.y);
                    *reinterpret_cast<uint32_t*>(own + at * 128 + (((k >> 1) ^ (at & 7)) << 4) + quad * 4) =
                        any && l[r] != 0.f ? *reinterpret_cast<const uint32_t*>(&hv) : 0u;
                }
                __syncwarp();
                uint4 v[4];
                #pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = k * 4 + (lane >> 3);
                    v[k] = *reinterpret_cast<const uint4*>(own + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
                }
                #pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = rows0 + k * 4 + (lane >> 3), tok = r >> log_g;
                    if (tok < left)
                        *reinterpret_cast<uint4*>(to + tok * a.out_stride + (r & (a.G - 1)) * (D * 2) + half * 128) = v[k];
                }
                __syncwarp();
            }
            tc_fence_before();
            // A key or value that is not finite reaches, as 0 * NaN, rows that do not see it: a row that came out so
            // is worked out again from the definition, which reads only what it sees.
            #pragma unroll
            for (int r = 0; r < 2; ++r) {
                unsigned again = __ballot_sync(0xffffffffu, any && l[r] != 0.f && row_of(r) >> log_g < left &&
                                                                !(odd[r].x + odd[r].y == 0.f));
                again = (again | again >> 1 | again >> 2 | again >> 3) & 0x11111111u;          // a bit per row
                #pragma unroll 1
                while (again) {
                    const int at = rows0 + ((__ffs(again) - 1) >> 2) + 8 * r;
                    again &= again - 1;
                    attend_row<D, POOL>(a, it.s, QuerySeq{it.first, it.n, it.ctx}, it.token + rt * per_tile + (at >> log_g),
                                        it.head * a.G + (at & (a.G - 1)));
                }
            }
        }
    } else if (C::WIDEN && warp >= kWidenWarp) {
        // ======== stored tiles to float16
        if constexpr (C::WIDEN) {
            fewer_registers<C::REGS_WIDEN>();
            const int tid = static_cast<int>(threadIdx.x) - kWidenWarp * 32;
            int ring = 0;
            while (next_item()) {
                #pragma unroll 1
                for (int j = keys.first(); fine && keys.is(j); j = keys.next(j)) {
                    const int rows = min(kTile, keys.end - (keys.base + j * kTile));
                    #pragma unroll
                    for (int kv = 0; kv < 2; ++kv, ++ring) {
                        const int slot = ring % C::SLOTS, raw = ring % C::RAWS;
                        if (!wait(raw_full(raw), ring / C::RAWS) ||
                            (ring >= C::SLOTS && !wait(empty(slot), ring / C::SLOTS - 1)))
                            break;
                        const char* from = smem + C::RAW_OFF + raw * C::RAW;
                        char* to = smem + C::KV_OFF + slot * C::TILE;
                        auto place = [&](int r, int ch) { return reinterpret_cast<uint4*>(to + tile_at<C::HALVES>(r, ch)); };
                        if (kv == 0) widen_rows<D, POOL, false, kTile, 128>(from, 0, rows, tid, place);
                        else widen_rows<D, POOL, true, kTile, 128>(from, 0, rows, tid, place);
                        fence_async_shared();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(full(slot));
                            mbar_arrive(raw_empty(raw));
                        }
                    }
                }
            }
        }
    } else {
        fewer_registers<C::REGS_ISSUE>();
    }
    if (warp == kMmaWarp) {
        // ======== matrix products: the warp stays together, one lane issues.  A row tile's products of a key tile and its
        // next scores, the next item's too, go behind one another, then the other row tile's: so the two take turns, one's
        // softmax runs while the other's products do.
        constexpr uint32_t s_shape = tc_idesc(kTile, false), o_shape = tc_idesc(D, true);
        // A look at a barrier takes 200 cycles beside the products' reads of shared memory: lanes 0 to 3 look at one each.
        auto wait4 = [&](uint32_t b0, int n0, uint32_t b1, int n1, uint32_t b2, int n2, uint32_t b3, int n3) {
            const uint32_t b = lane == 1 ? b1 : lane == 2 ? b2 : lane == 3 ? b3 : b0;
            const int n = lane == 1 ? n1 : lane == 2 ? n2 : lane == 3 ? n3 : n0;
            return wait(b, n);
        };
        int i0 = 0, i1 = 0;                                    // the row tiles' key tiles so far
        int j = 0;                                             // the key tile whose scores are asked for next
        bool fresh = true;                                     // it is its item's first
        // (Four products a turn: instructions are fetched beside the softmax's, and long straight runs of them come late:
        // 672 and 178 us for the capped and the 2048-token prompts where eight take 684 and 187.)
        auto scores = [&](int t, int at, bool last) {          // S = Q K^T (one lane)
            const uint64_t q_desc = tc_desc(base32 + C::Q_OFF + t * C::TILE, 0, 1024);
            const uint64_t k_desc = tc_desc(base32 + C::KV_OFF + at * C::TILE, 0, C::HALVES * 1024);
            #pragma unroll 4
            for (int k = 0; k < D / 16; ++k)
                tc_mma_ss(tmem + t * kTile, q_desc + (((k >> 2) * (kTile * 128) + (k & 3) * 32) >> 4),
                          k_desc + (((k >> 2) * 1024 + (k & 3) * 32) >> 4), s_shape, k > 0);
            tc_commit(s_there(t));
            if (last) tc_commit(q_free(t));
        };
        auto values = [&](int t, int at, bool add) {           // O += W V (one lane)
            const uint64_t v_desc = tc_desc(base32 + C::KV_OFF + at * C::TILE, 1024, C::HALVES * 1024);
            #pragma unroll 4
            for (int k = 0; k < kTile / 16; ++k)
                tc_mma_ts(tmem + 2 * kTile + t * D, tmem + t * kTile + k * 8, v_desc + k * (C::HALVES * 2048 >> 4), o_shape,
                          add || k > 0);
            tc_commit(o_there(t));
        };
        // What the next key tile's scores of row tile t take: the tile is on; it is t's last of the item, or t has none.
        struct Next { bool on, last, none; };
        auto next_of = [&](int t, bool more) {
            const bool on = more && keys.on(t, j);
            return Next{on, on && j == (BIAS ? keys.a(t) : keys.b(t) - 1), fresh && keys.a(t) == keys.b(t)};
        };
        auto ask = [&](int t, int at, const Next& n) {         // (one lane)
            if (n.on) scores(t, at, n.last);
            else if (n.none) mbar_arrive(q_free(t));
        };
        Ring<C::SLOTS> ring;
        bool item = next_item();
        while (item && fine) {
            j = keys.first();
            fresh = true;
            const bool more0 = keys.is(j);
            if (!wait4(q_there(0), count - 1, q_there(1), count - 1, more0 ? full(ring.slot) : q_there(0),
                       more0 ? ring.times : count - 1, q_there(0), count - 1))
                break;
            const Next first0 = next_of(0, more0), first1 = next_of(1, more0);
            if (elect_one()) {
                ask(0, ring.slot, first0);
                ask(1, ring.slot, first1);
                if (more0) tc_commit(empty(ring.slot));
            }
            __syncwarp();
            if (!more0) {
                item = next_item();
                continue;
            }
            bool more = true, now0 = first0.on, now1 = first1.on, some0 = false, some1 = false;
            #pragma unroll 1
            while (more) {                                     // (a key tile's scores are issued: its values, the next one's scores)
                ring.advance();
                const int v = ring.slot, v_times = ring.times;
                ring.advance();
                const int k = ring.slot;
                j = keys.next(j);
                more = keys.is(j);
                fresh = false;
                if (!more && (item = next_item())) {           // (one without key tiles waits for these products' end)
                    j = keys.first();
                    fresh = more = keys.is(j);
                }
                if (!fine) break;
                const Next n0 = next_of(0, more), n1 = next_of(1, more);
                // its values and weights, the next tile's keys; of another item, these and its queries by themselves
                const bool with = more && !fresh;
                if (!wait4(full(v), v_times, with ? full(k) : full(v), with ? ring.times : v_times, now0 ? w_there(0) : full(v),
                           now0 ? i0 : v_times, full(v), v_times))
                    break;
                tc_fence_after();
                if (elect_one()) {
                    if (now0) values(0, v, some0);
                    if (!fresh) ask(0, k, n0);
                }
                __syncwarp();
                if (fresh && !wait4(full(k), ring.times, q_there(0), count - 1, full(k), ring.times, full(k), ring.times)) break;
                if (fresh && elect_one()) ask(0, k, n0);
                __syncwarp();
                if (now1 && !wait(w_there(1), i1)) break;
                tc_fence_after();
                if (elect_one()) {
                    if (now1) values(1, v, some1);
                    tc_commit(empty(v));
                    if (!fresh) {
                        ask(1, k, n1);
                        if (more) tc_commit(empty(k));
                    }
                }
                __syncwarp();
                if (fresh && !wait(q_there(1), count - 1)) break;
                if (fresh && elect_one()) {
                    ask(1, k, n1);
                    tc_commit(empty(k));
                }
                __syncwarp();
                i0 += now0;
                i1 += now1;
                some0 = !fresh && (some0 || now0);             // (the next one's sums are added to its item's)
                some1 = !fresh && (some1 || now1);
                now0 = n0.on;
                now1 = n1.on;
            }
        }
        if (elect_one()) tc_commit(done);                      // nothing of it is in flight at the end
        __syncwarp();
        warp_wait(done, 0, a.err);
    } else if (warp == kLoadWarp) {
        // ======== keys and values in: a lane per block; float16 straight to its place, others as stored
        constexpr int DEPTH = C::WIDEN ? C::RAWS : C::SLOTS;
        auto there = [&](int i) { return C::WIDEN ? raw_full(i) : full(i); };
        auto gone = [&](int i) { return C::WIDEN ? raw_empty(i) : empty(i); };
        const int log_b = a.log_b, blk = lane;
        const uint32_t block_bytes = C::WIDEN ? a.B * kRowBytes<D, POOL> : a.B * D * 2;
        int ring = 0, edges = 0;
        while (next_item()) {
            int j = keys.first();
            // the tile's blocks are looked up a tile ahead
            auto look_up = [&](int at) {
                const int x = keys.base + at * kTile + (blk << log_b);
                return keys.is(at) && blk << log_b < kTile && x < keys.end ? query_block(a, it.s, x) : -1;
            };
            int id = look_up(j);
            #pragma unroll 1
            while (fine && keys.is(j)) {
                const int rows = min(kTile, keys.end - (keys.base + j * kTile)), jn = keys.next(j);
                const int next_id = look_up(jn);
                const uint32_t bytes = ((rows + a.B - 1) >> log_b) * block_bytes;
                if constexpr (POOL == KV_FP8_E4M3) {
                    const int of = __shfl_sync(0xffffffffu, id, lane < 16 ? 8 * lane >> log_b : 0);
                    if (lane < 16) {                           // per 8 tokens
                        float* const f = factors + (ring >> 1) % kFactorTiles * 48;
                        const float lv = value_log2(of >= 0 ? a.vscale[of] : 0.f);
                        f[2 * lane] = of >= 0 ? a.kscale[of] * (CAP ? 1.f : a.scale * kLog2e) : 0.f;
                        f[32 + lane] = lv == lv ? exp2f(-lv) : 0.f;
                        f[2 * lane + 1] = lv;
                    }
                    __syncwarp();
                }
                #pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const int slot = ring % DEPTH;
                    if (ring >= DEPTH && !wait(gone(slot), ring / DEPTH - 1)) break;
                    // values past the end: zero, they meet weights of zero
                    const bool tail = !C::WIDEN && kv == 1 && rows < kTile;
                    const uint32_t b = tail ? edge : there(slot);
                    if (lane == 0) mbar_arrive_expect_tx(b, bytes);
                    __syncwarp();
                    if (id >= 0) {
                        if constexpr (C::WIDEN) {
                            const int64_t from = (static_cast<int64_t>(id) * a.H + it.head) * block_bytes;
                            bulk_g2s(base32 + C::RAW_OFF + slot * C::RAW + blk * block_bytes, (kv ? a.vpool : a.kpool) + from,
                                     block_bytes, b);
                        } else {
                            tma_load_4d(base32 + C::KV_OFF + slot * C::TILE + blk * block_bytes, kv ? &p.vmap : &p.kmap, 0, 0, 0,
                                        (id * a.H + it.head) << (log_b - 3), b);
                        }
                    }
                    ++ring;
                    if (tail) {
                        if (!wait(edge, edges++)) break;
                        #pragma unroll 1
                        for (int u = rows * (D / 8) + lane; u < kTile * (D / 8); u += 32)
                            *reinterpret_cast<uint4*>(smem + C::KV_OFF + slot * C::TILE +
                                                      tile_at<C::HALVES>(u / (D / 8), u % (D / 8))) = make_uint4(0, 0, 0, 0);
                        fence_async_shared();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(full(slot));
                    }
                }
                j = jn;
                id = next_id;
            }
        }
        // before the CTA ends: every copy that was asked for has landed
        for (int r = max(0, ring - DEPTH); r < ring; ++r) mbar_wait_bounded(there(r % DEPTH), r / DEPTH & 1, a.err);
    } else if (warp == kItemWarp) {
        // ======== work items: what the rows see, and their queries, an item ahead of the others
        int s32 = -32, before = 0, upto = 0, lane_items = 0, lane_upto = 0;    // the sequences walked now, one a lane
        QuerySeq lane_seq{0, 0, 0};
        int index = blockIdx.x, claims = 0, asked = 0;         // (asked: items whose queries were asked for, in part at least)
        auto ask = [&]() {
            if (lane == 0) {
                mbar_arrive_expect_tx(claim, 16);
                claim_item(smem_u32(&misc->claim), claim);
            }
            __syncwarp();
        };
        auto answer = [&]() {
            if (!wait(claim, claims++)) return -1;
            const int x = uniform(claimed_item(misc->claim));
            __syncwarp();
            fence_async_shared();                              // (the next answer may overwrite it)
            return x;
        };
        ask();
        #pragma unroll 1
        while (true) {
            // The sequences' items one after the other; of a sequence the later row tiles, which see more keys, first,
            // each for every head.  Indices only grow, so the sequences are walked 32 at a time, a lane each.
            int s = 0, head = 0, token = 0, z = 0;
            QuerySeq seq{0, 0, 0};
            while (index >= 0 && index >= upto && s32 + 32 < a.batch) {
                s32 += 32;
                before = upto;
                lane_seq = QuerySeq{0, 0, 0};
                if (s32 + lane < a.batch) lane_seq = query_seq(a, s32 + lane, true);
                lane_items = prompt_tiles(lane_seq.n, a.G) * a.H * a.splits;
                lane_upto = lane_items;
                #pragma unroll
                for (int o = 1; o < 32; o *= 2) {
                    const int v = __shfl_up_sync(0xffffffffu, lane_upto, o);
                    if (lane >= o) lane_upto += v;
                }
                upto = before + __shfl_sync(0xffffffffu, lane_upto, 31);
            }
            if (index >= upto) {                               // beyond the last item
                index = answer();
                if (index >= 0) ask();
                continue;
            }
            if (index >= 0) {
                const int of = __ffs(__ballot_sync(0xffffffffu, before + lane_upto > index)) - 1;
                s = s32 + of;
                const int nth = index - before - __shfl_sync(0xffffffffu, lane_upto - lane_items, of), at = nth / a.splits;
                const int tiles = __shfl_sync(0xffffffffu, lane_items, of) / (a.H * a.splits);
                z = nth - at * a.splits;
                head = at % a.H;
                token = (tiles - 1 - at / a.H) * 2 * per_tile;
                seq = QuerySeq{__shfl_sync(0xffffffffu, lane_seq.first, of), __shfl_sync(0xffffffffu, lane_seq.n, of),
                               __shfl_sync(0xffffffffu, lane_seq.ctx, of)};
            }
            Item x{index < 0 ? -1 : s, head, token, seq.first, seq.n, seq.ctx, {1 << 30, 1 << 30}, {0, 0}, z, 0, 1 << 30};
            if (index >= 0) {
                #pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int from = token + t * per_tile, to = min(from + per_tile, seq.n);
                    for (int k = from + lane; k < to; k += 32) {
                        const int2 r = row_range(a, seq, k);
                        if (r.x < r.y) {
                            x.lo[t] = min(x.lo[t], r.x);
                            x.hi[t] = max(x.hi[t], r.y);
                        }
                    }
                    x.lo[t] = __reduce_min_sync(0xffffffffu, x.lo[t]);
                    x.hi[t] = __reduce_max_sync(0xffffffffu, x.hi[t]);
                }
                if (a.splits > 1 && max(x.hi[0], x.hi[1]) > 0) {               // an equal part of the item's key tiles
                    const int base = min(x.lo[0], x.lo[1]) & -a.B, tiles = (max(x.hi[0], x.hi[1]) - base + kTile - 1) / kTile;
                    x.from = base + tiles * z / a.splits * kTile;
                    x.to = base + tiles * (z + 1) / a.splits * kTile;
                    #pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        x.lo[t] = max(x.lo[t], x.from);
                        x.hi[t] = min(x.hi[t], x.to);
                        if (x.lo[t] >= x.hi[t]) {
                            x.lo[t] = 1 << 30;
                            x.hi[t] = 0;
                        }
                    }
                }
            }
            const int i = count & 1;
            if (count >= 2 && !wait(item_free(i), (count >> 1) - 1)) break;
            if (lane == 0) {
                misc->item[i] = x;
                mbar_arrive(item_there(i));
            }
            __syncwarp();
            if (index < 0) break;
            // queries (rows past the sequence's are another's, or zero past the last: what comes of them is not stored)
            #pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (count >= 1 && !wait(q_free(t), count - 1)) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_there(t), C::TILE);
                    #pragma unroll
                    for (int h = 0; h < C::HALVES; ++h)
                        tma_load_4d(base32 + C::Q_OFF + t * C::TILE + h * (kTile * 128), &p.qmap, 0, h, head * a.G,
                                    seq.first + token + t * per_tile, q_there(t));
                }
                __syncwarp();
                asked = count + 1;
            }
            if (!fine) break;
            ++count;
            // (the last index is followed to the end of the sequences, so that all are looked at, and no item is left
            // where rows out of order make more of them than the grid)
            if (index >= p.items - 1) {
                ++index;
            } else {
                index = answer();
                if (index >= 0) ask();
            }
            if (!fine) break;
        }
        // what is in flight after a wait ran out (queries, a claim's answer) lands before the CTA ends
        if (!fine && lane == 0) {
            for (int t = 0; t < 2 && asked; ++t) mbar_wait_bounded(q_there(t), (asked - 1) & 1, a.err);
            mbar_wait_bounded(claim, claims & 1, a.err);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_free(tmem);
    }
}

// The parts of a row's keys, joined: a warp per (row, query head).
template <int D, kv_dtype POOL>
__global__ void __launch_bounds__(256) query_join_kernel(const __grid_constant__ QueryArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int N = D / 32;
    const int heads = a.H * a.G, lane = threadIdx.x & 31;
    const int64_t per_seq = static_cast<int64_t>(a.max_queries) * heads, all = per_seq * a.batch;
    #pragma unroll 1
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); u < all; u += static_cast<int64_t>(gridDim.x) * 8) {
        const int s = static_cast<int>(u / per_seq), r = static_cast<int>(u - s * per_seq), i = r / heads, head = r - i * heads;
        const QuerySeq seq = query_seq(a, s, false);
        if (i >= seq.n) continue;
        const int64_t row = part_row(a.part_by_sequence, a.max_queries, s, seq.first, i) * heads + head, step = a.part_rows * heads;
        const float2 mine = lane < a.splits ? __ldcg(a.part_ml + lane * step + row) : make_float2(-CUDART_INF_F, 0.f);
        float top = mine.y != 0.f ? mine.x : -CUDART_INF_F;
        #pragma unroll
        for (int k = 1; k < 32; k *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        const float factor = mine.y != 0.f ? ex2_approx(mine.x - top) : 0.f;
        float l = 0.f, o[N] = {};
        #pragma unroll 4
        for (int z = 0; z < a.splits; ++z) {                   // (in order: the same bits every time)
            const float f = __shfl_sync(0xffffffffu, factor, z), lz = __shfl_sync(0xffffffffu, mine.y, z);
            if (lz == 0.f) continue;                           // (nothing was written)
            l = fmaf(lz, f, l);
            const float* const from = a.part_o + (z * step + row) * D + lane * N;
            #pragma unroll
            for (int e = 0; e < N; e += 2) {
                const float2 v = __ldcg(reinterpret_cast<const float2*>(from + e));
                o[e] = fmaf(v.x, f, o[e]);
                o[e + 1] = fmaf(v.y, f, o[e + 1]);
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        bool finite = true;
        char* const to = a.out + static_cast<int64_t>(seq.first + i) * a.out_stride + (head * D + lane * N) * 2;
        #pragma unroll
        for (int e = 0; e < N; e += 2) {
            const float2 v = make_float2(o[e] * inv, o[e + 1] * inv);
            finite &= fabsf(v.x) < CUDART_INF_F && fabsf(v.y) < CUDART_INF_F;
            *reinterpret_cast<__half2*>(to + e * 2) = __floats2half2_rn(v.x, v.y);
        }
        // (as in the kernel: a row that came out not finite, from the definition, other lanes' stores over these)
        if (__any_sync(0xffffffffu, !finite)) {
            __syncwarp();
            attend_row<D, POOL>(a, s, seq, i, head);
        }
    }
}

template <typename C, bool BIAS, int CAP>
int launch_prompt_typed(const kv_pool* pool, const PromptArgs& p, bool pdl, cudaStream_t stream) {
    static unsigned long long attr_done = 0;               // the shared-memory opt-in is a per-device attribute
    const unsigned long long bit = 1ull << (pool->device & 63);
    if (!(attr_done & bit)) {
        if (cudaFuncSetAttribute(query_prompt_kernel<C::D, C::POOL, BIAS, CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
            cudaSuccess)
            return KV_ERR_CUDA;
        attr_done |= bit;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.items));
    cfg.blockDim = dim3(C::WARPS * 32);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, query_prompt_kernel<C::D, C::POOL, BIAS, CAP>, p) != cudaSuccess) {
        cudaGetLastError();
        return KV_ERR_CUDA;
    }
    if (p.a.splits > 1) {
        const int64_t rows = static_cast<int64_t>(p.a.batch) * p.a.max_queries * p.a.H * p.a.G, most = static_cast<int64_t>(pool->num_sms) * 8;
        cfg.gridDim = dim3(static_cast<unsigned>((rows + 7) / 8 < most ? (rows + 7) / 8 : most));
        cfg.blockDim = dim3(256);
        cfg.dynamicSmemBytes = 0;
        cfg.numAttrs = 1;                                      // (it waits for the kernel above itself)
        if (cudaLaunchKernelEx(&cfg, query_join_kernel<C::D, C::POOL>, p.a) != cudaSuccess) {
            cudaGetLastError();
            return KV_ERR_CUDA;
        }
    }
    return KV_OK;
}

template <kv_dtype POOL>
int launch_prompt_pool(const kv_pool* pool, const PromptArgs& p, bool pdl, cudaStream_t stream) {
    auto launch = [&](auto bias, auto cap) {
        return pool->desc.head_dim == 128 ? launch_prompt_typed<PromptCfg<128, POOL>, bias.value, cap.value>(pool, p, pdl, stream)
                                          : launch_prompt_typed<PromptCfg<64, POOL>, bias.value, cap.value>(pool, p, pdl, stream);
    };
    auto with_cap = [&](auto bias) {
        if (p.a.cap > kLargeCap) return launch(bias, std::integral_constant<int, LARGE_CAP>{});
        if (p.a.cap > 0.f) return launch(bias, std::integral_constant<int, SMALL_CAP>{});
        return launch(bias, std::integral_constant<int, NO_CAP>{});
    };
    return p.a.slopes ? with_cap(std::true_type{}) : with_cap(std::false_type{});
}

}  // namespace
}  // namespace kvp
