// paged_query_attention for many rows: the tensor-core kernel.
#pragma once

#include "query_attention.cuh"
#include "tcgen05.cuh"
#include "widen.cuh"

namespace kvp {

struct PromptArgs {
    CUtensorMap kmap, vmap;            // float16 pools: the layer's row maps, a block of one head per copy
    QueryArgs a;
    int tiles;                         // pairs of row tiles per (sequence, K/V head)
};

int launch_query_prompt_fp8(const kv_pool* pool, const PromptArgs& p, bool pdl, cudaStream_t stream);
int launch_query_prompt_int4(const kv_pool* pool, const PromptArgs& p, bool pdl, cudaStream_t stream);

namespace {

constexpr int kTile = 128;             // rows of a row tile and keys of a key tile
constexpr int kSoftmaxWarps = 8, kMmaWarp = 8, kLoadWarp = 9, kWidenWarp = 12;
constexpr int kFactorTiles = 8;        // key tiles whose FP8 scales are kept (more than are in flight)

template <int D_, kv_dtype POOL_>
struct PromptCfg {
    static constexpr int D = D_;
    static constexpr kv_dtype POOL = POOL_;
    static constexpr bool WIDEN = POOL != KV_F16;              // tiles are widened to float16 on their way
    static constexpr int HALVES = D / 64;                      // 64-element (128-byte) columns of a tile: a tile
    // is [16 groups of 8 rows][HALVES][8][128 bytes], 128-byte swizzled
    static constexpr int TILE = HALVES * kTile * 128;          // bytes of 128 rows as float16
    // key and value tiles in flight as float16, and as stored
    static constexpr int SLOTS = D == 128 ? (WIDEN ? 4 : 5) : 8;
    static constexpr int RAWS = WIDEN ? (D == 128 ? 2 : 4) : 0;
    static constexpr int RAW = WIDEN ? kTile * kRowBytes<D, POOL> : 0;
    // Registers: 168 (12 warps) or 128 (16 warps) per thread at launch, shared out by fours of warps
    static constexpr int WARPS = WIDEN ? 16 : 12;
    static constexpr int REGS_SOFTMAX = WIDEN ? 200 : 208, REGS_ISSUE = WIDEN ? 48 : 88, REGS_WIDEN = 64;
    static_assert(WIDEN ? 2 * REGS_SOFTMAX + REGS_ISSUE + REGS_WIDEN <= 512 : 2 * REGS_SOFTMAX + REGS_ISSUE <= 504, "registers");
    static constexpr int Q_OFF = 0, KV_OFF = 2 * TILE, RAW_OFF = KV_OFF + SLOTS * TILE;
    static constexpr int FACTOR_OFF = RAW_OFF + RAWS * RAW;
    static constexpr int FACTORS = POOL == KV_FP8_E4M3 ? kFactorTiles * 2 * 16 * 4 : 0;
    static constexpr int BAR_OFF = FACTOR_OFF + FACTORS;
    // full, empty per slot; per row tile: queries there, scores there, weights there, product there; edge; done;
    // full, empty per raw tile
    static constexpr int BARS = 2 * SLOTS + 4 * 2 + 2 + 2 * RAWS;
    static constexpr int MISC_OFF = BAR_OFF + BARS * 8;
    static constexpr int SMEM = MISC_OFF + 64 + 1024;          // and up to 1024 bytes of alignment
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(BAR_OFF % 16 == 0 && RAW % 16 == 0, "alignment");
};

template <int N> __device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Byte offset of 16 bytes (8 elements, the ch-th of a row) in a tile.
template <int HALVES>
__device__ __forceinline__ uint32_t tile_at(int r, int ch) {
    return (((r >> 3) * HALVES + (ch >> 3)) << 10) + ((r & 7) << 7) + (((ch & 7) ^ (r & 7)) << 4);
}

// The warp's first lane's value.  The compiler knows the result to be the same in every lane, so branches on it
// keep a warp together and operands made of it may be uniform registers, as the matrix instructions' must be.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// A bounded wait by a whole warp: all of its lanes go on, or none.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int* err) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, err));
}

// What the CTA's roles share: visible range, its first position, key tiles per row tile.
struct PromptMisc {
    uint32_t tmem;
    int lo[2], hi[2];
    int vmax;                          // FP8: the largest value scale, as the bits of its magnitude
};

// Key tiles [a, b) of each row tile, numbered from position `base`.
struct KeyTiles {
    int base, end, a[2], b[2], n;
    __device__ __forceinline__ bool on(int t, int j) const { return j >= a[t] && j < b[t]; }
    __device__ __forceinline__ int next(int j) const {         // the first tile from j on that a row tile needs
        while (j < n && !on(0, j) && !on(1, j)) ++j;
        return j;
    }
};
__device__ __forceinline__ KeyTiles key_tiles(const PromptMisc* m, int block) {
    KeyTiles k;
    const int lo[2] = {uniform(m->lo[0]), uniform(m->lo[1])}, hi[2] = {uniform(m->hi[0]), uniform(m->hi[1])};
    k.base = min(lo[0], lo[1]) & -block;
    k.end = max(hi[0], hi[1]);
    #pragma unroll
    for (int t = 0; t < 2; ++t) {
        const bool some = lo[t] < hi[t];
        k.a[t] = some ? (lo[t] - k.base) / kTile : 0;
        k.b[t] = some ? (hi[t] - k.base + kTile - 1) / kTile : 0;
    }
    k.n = max(k.b[0], k.b[1]);
    return k;
}

template <int D, kv_dtype POOL>
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
    auto q_there = [&](int t) { return bar(2 * C::SLOTS + t); };
    auto s_there = [&](int t) { return bar(2 * C::SLOTS + 2 + t); };
    auto w_there = [&](int t) { return bar(2 * C::SLOTS + 4 + t); };
    auto o_there = [&](int t) { return bar(2 * C::SLOTS + 6 + t); };
    const uint32_t edge = bar(2 * C::SLOTS + 8), done = bar(2 * C::SLOTS + 9);
    auto raw_full = [&](int i) { return bar(2 * C::SLOTS + 10 + i); };
    auto raw_empty = [&](int i) { return bar(2 * C::SLOTS + 10 + C::RAWS + i); };
    float* const factors = reinterpret_cast<float*>(smem + C::FACTOR_OFF);     // FP8: [tile][keys, values][block]

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // the work item: later row tiles, which see more keys, first
    const int item = blockIdx.x;
    const int tile = p.tiles - 1 - item % p.tiles, head = item / p.tiles % a.H, s = item / p.tiles / a.H;
    QuerySeq seq = query_seq(a, s, threadIdx.x == 0 && tile == 0 && head == 0);
    seq = QuerySeq{uniform(seq.first), uniform(seq.n), uniform(seq.ctx)};
    const int per_tile = kTile / a.G;                          // tokens of a row tile
    if (tile * 2 * per_tile >= seq.n) return;

    // ---- set-up: barriers, tensor memory, what the rows see
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::SLOTS; ++i) {
            mbar_init(full(i), C::WIDEN ? 4 : 1);
            mbar_init(empty(i), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(q_there(t), 4);
            mbar_init(s_there(t), 1);
            mbar_init(w_there(t), 4);
            mbar_init(o_there(t), 1);
        }
        mbar_init(edge, 1);
        mbar_init(done, 1);
        for (int i = 0; i < C::RAWS; ++i) {
            mbar_init(raw_full(i), 1);
            mbar_init(raw_empty(i), 4);
        }
        misc->vmax = 0;
        fence_mbar_init();
    }
    if (threadIdx.x < 2) {
        misc->lo[threadIdx.x] = 1 << 30;
        misc->hi[threadIdx.x] = 0;
    }
    if (warp == kMmaWarp) tmem_alloc(smem_u32(&misc->tmem));
    __syncthreads();
    const int rt = warp >> 2;                                  // softmax warps: the row tile
    const int row = (warp & 3) * 32 + lane;                    // and the thread's row of it
    const int token = (tile * 2 + rt) * per_tile + row / a.G;
    int2 sees = make_int2(0, 0);
    if (warp < kSoftmaxWarps) {
        if (token < seq.n) sees = row_range(a, seq, token);
        const bool some = sees.x < sees.y;
        const int lo = __reduce_min_sync(0xffffffffu, some ? sees.x : 1 << 30);
        const int hi = __reduce_max_sync(0xffffffffu, some ? sees.y : 0);
        if (lane == 0 && lo < hi) {
            atomicMin(&misc->lo[rt], lo);
            atomicMax(&misc->hi[rt], hi);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(misc->tmem);
    const KeyTiles keys = key_tiles(misc, a.B);
    const int first_tile = keys.next(0);

    if (warp < kSoftmaxWarps) {
        // ======== queries in, softmax, result out: a thread per row
        more_registers<C::REGS_SOFTMAX>();
        constexpr int CHUNKS = D / 8;                          // 16-byte pieces of a row
        char* const qt = smem + C::Q_OFF + rt * C::TILE;
        const int64_t q0 = static_cast<int64_t>(seq.first) * a.q_stride + static_cast<int64_t>(head) * a.G * D * 2;
        // the warp's 32 rows, neighbouring pieces side by side; every load asked for before the first is stored
        uint4 qv[CHUNKS];
        const int log_g = __ffs(a.G) - 1;
        #pragma unroll
        for (int it = 0; it < CHUNKS; ++it) {
            const int u = it * 32 + lane, r = (warp & 3) * 32 + u / CHUNKS, c = u % CHUNKS;
            const int tok = (tile * 2 + rt) * per_tile + (r >> log_g);
            qv[it] = make_uint4(0, 0, 0, 0);
            if (tok < seq.n)
                qv[it] = *reinterpret_cast<const uint4*>(a.q + q0 + tok * a.q_stride + (r & (a.G - 1)) * (D * 2) + c * 16);
        }
        #pragma unroll
        for (int it = 0; it < CHUNKS; ++it) {
            const int u = it * 32 + lane, r = (warp & 3) * 32 + u / CHUNKS, c = u % CHUNKS;
            *reinterpret_cast<uint4*>(qt + tile_at<C::HALVES>(r, c)) = qv[it];
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_there(rt));

        // FP8: value scales enter the weights relative to the largest one, which multiplies the result
        float vref = 1.f;
        if constexpr (POOL == KV_FP8_E4M3) {
            float top = 0.f;
            for (int at = keys.base + static_cast<int>(threadIdx.x) * a.B; at < keys.end; at += kSoftmaxWarps * 32 * a.B)
                top = max_nan(top, fabsf(a.vscale[query_block(a, s, at)]));
            // (bits of magnitudes, NaN among them, are ordered as integers)
            const int bits = __reduce_max_sync(0xffffffffu, __float_as_int(top) & 0x7FFFFFFF);
            if (lane == 0) atomicMax(&misc->vmax, bits);
            asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxWarps * 32) : "memory");
            vref = max_nan(__int_as_float(misc->vmax), 1.17549435e-38f);
        }
        const float inv_vref = 1.f / vref;

        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;       // the warp's 32 lanes
        const uint32_t st = tmem + lanes + rt * kTile, ot = tmem + lanes + 2 * kTile + rt * D;
        const int hq = head * a.G + row % a.G;
        const bool bias = a.slopes != nullptr, cap = a.cap > 0.f;
        const float slope = bias ? a.slopes[hq] * kLog2e : 0.f;
        const float qscale = a.scale * kLog2e;
        const float k2 = cap ? 2.f * kLog2e * (a.scale / a.cap) : 0.f, capl = a.cap * kLog2e;
        const float c = cap || bias ? 1.f : qscale;            // scores to log2 units
        const int pos = seq.ctx - seq.n + token;
        float m = -CUDART_INF_F, l = 0.f;                      // the base (log2 units) and the sum of weights
        int i = 0;                                             // this row tile's key tiles so far
        bool fine = true;
        #pragma unroll 1
        for (int j = keys.a[rt]; j < keys.b[rt]; ++j, ++i) {
            if (!warp_wait(s_there(rt), i & 1, a.err)) {
                fine = false;
                break;
            }
            tc_fence_after();
            float x[kTile];
            uint32_t* const xr = reinterpret_cast<uint32_t*>(x);
            #pragma unroll
            for (int k = 0; k < 4; ++k) tmem_load32(st + 32 * k, xr + 32 * k);
            #pragma unroll
            for (int k = 0; k < 4; ++k) tmem_wait_load32(xr + 32 * k);
            const int j0 = keys.base + j * kTile;
            const float* const scales = factors + (j % kFactorTiles) * 32;
            if constexpr (POOL == KV_FP8_E4M3) {
                #pragma unroll
                for (int k = 0; k < kTile; k += 8) {
                    const float f = scales[k >> a.log_b];
                    #pragma unroll
                    for (int e = 0; e < 8; ++e) x[k + e] *= f;
                }
            }
            if (cap) {
                #pragma unroll
                for (int k = 0; k < kTile; ++k) x[k] = capped(x[k], k2, capl);
            }
            if (bias) {
                const float from = static_cast<float>(pos - j0), mul = cap ? 1.f : qscale;
                #pragma unroll
                for (int k = 0; k < kTile; ++k) x[k] = fmaf(-slope, fabsf(from - static_cast<float>(k)), x[k] * mul);
            }
            if (__any_sync(0xffffffffu, sees.x > j0 || sees.y < j0 + kTile)) {
                const int from = sees.x - j0;
                const unsigned len = sees.y - sees.x;
                #pragma unroll
                for (int k = 0; k < kTile; ++k)
                    if (static_cast<unsigned>(k - from) >= len) x[k] = -CUDART_INF_F;
            }
            float top = fmaxf(x[0], x[1]);
            #pragma unroll
            for (int k = 2; k < kTile; k += 2) top = fmaxf(fmaxf(x[k], x[k + 1]), top);
            // the base follows the maximum only when it is left behind by more than 2^8
            top *= c;
            const bool raise = top - m > kRaise;               // (m -inf: yes, but for a row that sees nothing yet)
            float keep = 1.f;
            if (raise) {
                keep = ex2_approx(m - top);
                m = top;
                l *= keep;
            }
            if (i > 0 && __any_sync(0xffffffffu, raise)) {
                if (!warp_wait(o_there(rt), (i - 1) & 1, a.err)) {
                    fine = false;
                    break;
                }
                tc_fence_after();
                #pragma unroll 1
                for (int k = 0; k < D; k += 32) {
                    uint32_t o[32];
                    tmem_load32(ot + k, o);
                    tmem_wait_load32(o);
                    #pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                    tmem_store32(ot + k, o);
                }
            }
            const float off = kLift - (m == -CUDART_INF_F ? 0.f : m);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            const float2 c2 = make_float2(c, c), off2 = make_float2(off, off);
            #pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t w[32];
                #pragma unroll
                for (int k = 0; k < 32; ++k) {
                    float2 y = __ffma2_rn(make_float2(x[64 * h + 2 * k], x[64 * h + 2 * k + 1]), c2, off2);
                    y.x = ex2_approx(y.x);
                    y.y = ex2_approx(y.y);
                    sum[k & 1] = __fadd2_rn(sum[k & 1], y);
                    if constexpr (POOL == KV_FP8_E4M3) {
                        const float f = scales[16 + ((64 * h + 2 * k) >> a.log_b)] * inv_vref;
                        y = __fmul2_rn(y, make_float2(f, f));
                    }
                    const __half2 hv = __floats2half2_rn(y.x, y.y);
                    w[k] = *reinterpret_cast<const uint32_t*>(&hv);
                }
                tmem_store32(st + 32 * h, w);
            }
            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            tmem_wait_store();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(w_there(rt));
        }
        // ---- the result: through the queries' place in shared memory, a warp its own 32 rows
        if (fine && i > 0 && !warp_wait(o_there(rt), (i - 1) & 1, a.err)) fine = false;
        if (fine && i > 0) tc_fence_after();
        const float inv = l == 0.f ? 0.f : vref / l;
        bool odd = false;                                      // something is not finite: from the definition below
        #pragma unroll 1
        for (int k = 0; k < D; k += 32) {
            uint32_t o[32];
            if (fine && i > 0) {
                tmem_load32(ot + k, o);
                tmem_wait_load32(o);
            }
            #pragma unroll
            for (int e = 0; e < 32; e += 8) {
                uint32_t w[4];
                #pragma unroll
                for (int y = 0; y < 4; ++y) {
                    float2 f = make_float2(0.f, 0.f);
                    if (fine && i > 0 && l != 0.f)
                        f = make_float2(__uint_as_float(o[e + 2 * y]) * inv, __uint_as_float(o[e + 2 * y + 1]) * inv);
                    odd |= !(fabsf(f.x) < CUDART_INF_F) || !(fabsf(f.y) < CUDART_INF_F);
                    const __half2 hv = __floats2half2_rn(f.x, f.y);
                    w[y] = *reinterpret_cast<const uint32_t*>(&hv);
                }
                const int ch = (k + e) >> 3;
                *reinterpret_cast<uint4*>(qt + tile_at<C::HALVES>(row, ch)) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        __syncwarp();
        if (fine) {
            const int64_t o0 = static_cast<int64_t>(seq.first) * a.out_stride + static_cast<int64_t>(head) * a.G * D * 2;
            uint4 ov[CHUNKS];
            #pragma unroll
            for (int it = 0; it < CHUNKS; ++it) {
                const int u = it * 32 + lane, r = (warp & 3) * 32 + u / CHUNKS, ch = u % CHUNKS;
                ov[it] = *reinterpret_cast<const uint4*>(qt + tile_at<C::HALVES>(r, ch));
            }
            #pragma unroll
            for (int it = 0; it < CHUNKS; ++it) {
                const int u = it * 32 + lane, r = (warp & 3) * 32 + u / CHUNKS, ch = u % CHUNKS;
                const int tok = (tile * 2 + rt) * per_tile + (r >> log_g);
                if (tok < seq.n)
                    *reinterpret_cast<uint4*>(a.out + o0 + tok * a.out_stride + (r & (a.G - 1)) * (D * 2) + ch * 16) = ov[it];
            }
            // A key or value that is not finite reaches, as 0 * NaN, rows that do not see it: a row that came out
            // so is worked out again from the definition, which reads only what it sees.
            unsigned again = __ballot_sync(0xffffffffu, odd && token < seq.n);
            __syncwarp();
            #pragma unroll 1
            while (again) {
                const int r = (warp & 3) * 32 + __ffs(again) - 1;
                again &= again - 1;
                attend_row<D, POOL>(a, s, seq, (tile * 2 + rt) * per_tile + r / a.G, head * a.G + r % a.G);
            }
        }
    } else if (C::WIDEN && warp >= kWidenWarp) {
        // ======== stored tiles to float16
        if constexpr (C::WIDEN) {
            fewer_registers<C::REGS_WIDEN>();
            const int tid = static_cast<int>(threadIdx.x) - kWidenWarp * 32;
            int ring = 0;
            bool fine = true;
            #pragma unroll 1
            for (int j = first_tile; fine && j < keys.n; j = keys.next(j + 1)) {
                const int rows = min(kTile, keys.end - (keys.base + j * kTile));
                #pragma unroll
                for (int kv = 0; kv < 2; ++kv, ++ring) {
                    const int slot = ring % C::SLOTS, raw = ring % C::RAWS;
                    if (!warp_wait(raw_full(raw), ring / C::RAWS & 1, a.err) ||
                        (ring >= C::SLOTS && !warp_wait(empty(slot), (ring / C::SLOTS - 1) & 1, a.err))) {
                        fine = false;
                        break;
                    }
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
    } else {
        fewer_registers<C::REGS_ISSUE>();
    }
    if (warp == kMmaWarp) {
        // ======== matrix products: the warp stays together, one lane issues
        constexpr uint32_t s_shape = tc_idesc(kTile, false), o_shape = tc_idesc(D, true);
        int n[2] = {0, 0};                                     // products of weights issued per row tile
        int slot = 0, phase = 0;                               // the ring's next tile
        bool fine = true;
        auto wait = [&](uint32_t b, uint32_t parity) { fine = fine && warp_wait(b, parity, a.err); };
        auto tile_desc = [&](int at, uint32_t lead) { return tc_desc(base32 + C::KV_OFF + at * C::TILE, lead, C::HALVES * 1024); };
        const uint64_t q_desc = tc_desc(base32 + C::Q_OFF, 0, C::HALVES * 1024);
        auto scores = [&](int t, uint64_t k_desc, uint32_t then) {     // S = Q K^T; then: the keys' release, or 0
            if (elect_one()) {
                #pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const int at = ((k >> 2) * 1024 + (k & 3) * 32) >> 4;
                    tc_mma_ss(tmem + t * kTile, q_desc + t * (C::TILE >> 4) + at, k_desc + at, s_shape, k > 0);
                }
                tc_commit(s_there(t));
                if (then) tc_commit(then);
            }
            __syncwarp();
        };
        auto take = [&]() {                                    // the ring's next tile: waited for; its place
            const int at = slot;
            wait(full(at), phase);
            if (++slot == C::SLOTS) {
                slot = 0;
                phase ^= 1;
            }
            return at;
        };
        int j = first_tile;
        if (j < keys.n) {
            const int at = take();
            #pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (!keys.on(t, j)) continue;
                wait(q_there(t), 0);
                if (fine) scores(t, tile_desc(at, 0), t == 1 || !keys.on(1, j) ? empty(at) : 0);
            }
        }
        #pragma unroll 1
        while (fine && j < keys.n) {
            const int jn = keys.next(j + 1);
            const int v_at = take();
            int k_at = -1;
            const uint64_t v_desc = tile_desc(v_at, 1024);
            #pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (keys.on(t, j)) {
                    wait(w_there(t), n[t] & 1);
                    if (!fine) break;
                    tc_fence_after();
                    if (elect_one()) {
                        #pragma unroll
                        for (int k = 0; k < kTile / 16; ++k)   // O += W V
                            tc_mma_ts(tmem + 2 * kTile + t * D, tmem + t * kTile + k * 8, v_desc + k * (C::HALVES * 2048 >> 4),
                                      o_shape, n[t] > 0 || k > 0);
                        tc_commit(o_there(t));
                        if (t == 1 || !keys.on(1, j)) tc_commit(empty(v_at));
                    }
                    __syncwarp();
                    ++n[t];
                }
                if (jn < keys.n && keys.on(t, jn)) {
                    if (k_at < 0) k_at = take();
                    wait(q_there(t), 0);
                    if (!fine) break;
                    scores(t, tile_desc(k_at, 0), t == 1 || !keys.on(1, jn) ? empty(k_at) : 0);
                }
            }
            j = jn;
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
        int ring = 0, edges = 0;
        bool fine = true;
        #pragma unroll 1
        for (int j = first_tile; fine && j < keys.n; j = keys.next(j + 1)) {
            const int j0 = keys.base + j * kTile, rows = min(kTile, keys.end - j0);
            const bool mine = (blk << log_b) < rows;
            const int id = mine ? query_block(a, s, j0 + (blk << log_b)) : 0;
            const uint32_t block_bytes = C::WIDEN ? a.B * kRowBytes<D, POOL> : a.B * D * 2;
            const uint32_t bytes = ((rows + a.B - 1) >> log_b) * block_bytes;
            if constexpr (POOL == KV_FP8_E4M3) {
                if (blk < 16) {
                    factors[(j % kFactorTiles) * 32 + blk] = mine ? a.kscale[id] : 0.f;
                    factors[(j % kFactorTiles) * 32 + 16 + blk] = mine ? a.vscale[id] : 0.f;
                }
                __syncwarp();
            }
            #pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const int slot = ring % DEPTH;
                if (ring >= DEPTH && !warp_wait(gone(slot), (ring / DEPTH - 1) & 1, a.err)) {
                    fine = false;
                    break;
                }
                const bool tail = !C::WIDEN && kv == 1 && rows < kTile;   // values past the end: zero, they meet weights of zero
                const uint32_t b = tail ? edge : there(slot);
                if (lane == 0) mbar_arrive_expect_tx(b, bytes);
                __syncwarp();
                if (mine) {
                    if constexpr (C::WIDEN) {
                        const int64_t from = (static_cast<int64_t>(id) * a.H + head) * block_bytes;
                        bulk_g2s(base32 + C::RAW_OFF + slot * C::RAW + blk * block_bytes, (kv ? a.vpool : a.kpool) + from,
                                 block_bytes, b);
                    } else {
                        tma_load_4d(base32 + C::KV_OFF + slot * C::TILE + blk * block_bytes, kv ? &p.vmap : &p.kmap, 0, 0, 0,
                                    (id * a.H + head) << (log_b - 3), b);
                    }
                }
                if (tail) {
                    fine = warp_wait(edge, edges++ & 1, a.err);
                    #pragma unroll 1
                    for (int u = rows * (D / 8) + lane; u < kTile * (D / 8); u += 32)
                        *reinterpret_cast<uint4*>(smem + C::KV_OFF + slot * C::TILE + tile_at<C::HALVES>(u / (D / 8), u % (D / 8))) =
                            make_uint4(0, 0, 0, 0);
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full(slot));
                }
                ++ring;
            }
        }
        // before the CTA ends: every copy that was asked for has landed
        for (int r = max(0, ring - DEPTH); r < ring; ++r) mbar_wait_bounded(there(r % DEPTH), r / DEPTH & 1, a.err);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_free(tmem);
    }
}

template <typename C>
int launch_prompt_typed(const kv_pool* pool, const PromptArgs& p, bool pdl, cudaStream_t stream) {
    static unsigned long long attr_done = 0;               // the shared-memory opt-in is a per-device attribute
    const unsigned long long bit = 1ull << (pool->device & 63);
    if (!(attr_done & bit)) {
        if (cudaFuncSetAttribute(query_prompt_kernel<C::D, C::POOL>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
            cudaSuccess)
            return KV_ERR_CUDA;
        attr_done |= bit;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.a.batch * p.a.H * p.tiles));
    cfg.blockDim = dim3(C::WARPS * 32);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, query_prompt_kernel<C::D, C::POOL>, p) != cudaSuccess) {
        cudaGetLastError();
        return KV_ERR_CUDA;
    }
    return KV_OK;
}

template <kv_dtype POOL>
int launch_prompt_pool(const kv_pool* pool, const PromptArgs& p, bool pdl, cudaStream_t stream) {
    return pool->desc.head_dim == 128 ? launch_prompt_typed<PromptCfg<128, POOL>>(pool, p, pdl, stream)
                                      : launch_prompt_typed<PromptCfg<64, POOL>>(pool, p, pdl, stream);
}

}  // namespace
}  // namespace kvp
