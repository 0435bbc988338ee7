// kv_append_rope, kv_append into 4-bit pools (the kernel is in append_rope_kernel.cuh); kv_gather, the
// inverse (cached tokens back as contiguous rows); kv_rope_table.

#include "append_rope_kernel.cuh"

namespace kvp {
namespace {

RopeArgs pool_side(const kv_pool* pool, int layer) {
    const kv_pool_desc& d = pool->desc;
    RopeArgs a{};
    a.kpool = static_cast<char*>(pool->k_layers[layer]);
    a.vpool = static_cast<char*>(pool->v_layers[layer]);
    a.kscale = pool->k_scales ? pool->k_scales[layer] : nullptr;
    a.vscale = pool->v_scales ? pool->v_scales[layer] : nullptr;
    a.H = d.num_heads;
    a.B = d.block_size;
    a.num_slots = static_cast<int64_t>(d.num_blocks) * d.block_size;
    a.err = pool->d_err;
    return a;
}

}  // namespace

int launch_append_rope(const kv_pool* pool, const kv_rope_args& x, const kv_rope_axes* axes) {
    const int es = elem_bytes(x.in_dtype), qs = pool->desc.dtype == KV_F32 ? 4 : 2;
    RopeArgs a = pool_side(pool, x.layer);
    a.q = static_cast<const char*>(x.q);
    a.k = static_cast<const char*>(x.k);
    a.v = static_cast<const char*>(x.v);
    a.q_out = static_cast<char*>(x.q_out);
    a.q_stride = x.q_stride * es;
    a.k_stride = x.k_stride * es;
    a.v_stride = x.v_stride * es;
    a.qo_stride = x.q_out_stride * qs;
    a.slots = x.slot_mapping;
    a.positions = x.positions;
    a.table = x.cos_sin;
    a.table_len = x.table_len;
    a.rot = x.rot_dim;
    a.adjacent = x.adjacent_pairs ? 1 : 0;
    a.n = x.num_tokens;
    a.Hq = x.q ? x.num_q_heads : 0;
    const bool pdl = (x.flags & KV_DECODE_PDL) != 0;
    if (axes) {
        a.axes = axes->num_axes;
        a.axis_stride = axes->axis_stride;
        for (int i = 0; i < x.rot_dim / 2; ++i) a.pair_axis[i >> 4] |= static_cast<uint32_t>(axes->pair_axis[i]) << (2 * (i & 15));
        return launch_rope_axes_any(pool, x.in_dtype, a, pdl, x.stream);
    }
    return launch_rope_types<false>(pool, x.in_dtype, a, pdl, x.stream);
}

int launch_append_int4(const kv_pool* pool, int layer, const void* k, const void* v, kv_dtype in_dtype,
                       const int64_t* slot_mapping, int num_tokens, cudaStream_t stream) {
    RopeArgs a = pool_side(pool, layer);
    a.k = static_cast<const char*>(k);
    a.v = static_cast<const char*>(v);
    a.k_stride = a.v_stride = static_cast<int64_t>(pool->desc.num_heads) * pool->desc.head_dim * elem_bytes(in_dtype);
    a.slots = slot_mapping;
    a.n = num_tokens;
    return launch_rope_types<false>(pool, in_dtype, a, false, stream);
}

// ---------------------------------------------------------------- gather
namespace {

constexpr int kGatherThreads = 256, kGatherWarps = kGatherThreads / 32;

struct GatherArgs {
    const char *kpool, *vpool;
    const float *kscale, *vscale;
    const int64_t* slots;
    char *k, *v;
    int n, H, B;
    int64_t num_slots;
    int* err;
};

// The unit's 8 stored elements: their bytes in a (and b).
template <int D, kv_dtype POOL>
__device__ __forceinline__ void load_stored(const char* tile, int off, int unit, uint4& a, uint4& b) {
    if constexpr (POOL == KV_F32) {
        const uint4* p = reinterpret_cast<const uint4*>(tile + (static_cast<int64_t>(off) * D + unit * 8) * 4);
        a = __ldcs(p);
        b = __ldcs(p + 1);
    } else if constexpr (POOL == KV_F16) {
        a = __ldcs(reinterpret_cast<const uint4*>(tile + (off * D + unit * 8) * 2));
    } else {
        const uint2 x = __ldcs(reinterpret_cast<const uint2*>(tile + off * D + unit * 8));
        a.x = x.x;
        a.y = x.y;
    }
}

// grid (tokens / 2, head splits): half-warps of one token each, as append_rope_kernel
template <int D, kv_dtype POOL, typename TOut>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const __grid_constant__ GatherArgs a) {
    constexpr int UPR = D / 8, HPW = 16 / UPR, UNROLL = 4;
    constexpr int ROW = POOL == KV_FP8_E4M3 ? D : POOL == KV_F16 ? 2 * D : 4 * D;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int unit = lane & (UPR - 1), sub = (lane & 15) / UPR;
    const int64_t tok = static_cast<int64_t>(blockIdx.x) * 2 + (lane >> 4);
    const int64_t slot = tok < a.n ? a.slots[tok] : -1;
    if (slot < 0) return;                              // no shuffles below
    if (slot >= a.num_slots) {
        atomicOr(a.err, KV_DEVERR_SLOT);
        return;
    }
    const int64_t blk = slot / a.B;
    const int off = static_cast<int>(slot - blk * a.B);
    float ks = 1.f, vs = 1.f;
    if constexpr (POOL == KV_FP8_E4M3) {
        ks = a.kscale[blk];
        vs = a.vscale[blk];
    }
    const int uk = (a.H + HPW - 1) / HPW, rows = 2 * uk, step = gridDim.y * kGatherWarps;
    for (int r0 = blockIdx.y * kGatherWarps + warp; r0 < rows; r0 += step * UNROLL) {
        uint4 x[UNROLL], y[UNROLL];
        #pragma unroll
        for (int j = 0; j < UNROLL; ++j) {
            const int r = r0 + j * step;
            const bool is_v = r >= uk;
            const int h = (is_v ? r - uk : r) * HPW + sub;
            if (r >= rows || h >= a.H) continue;
            load_stored<D, POOL>((is_v ? a.vpool : a.kpool) + (blk * a.H + h) * static_cast<int64_t>(a.B) * ROW, off,
                                 unit, x[j], y[j]);
        }
        #pragma unroll
        for (int j = 0; j < UNROLL; ++j) {
            const int r = r0 + j * step;
            const bool is_v = r >= uk;
            const int h = (is_v ? r - uk : r) * HPW + sub;
            if (r >= rows || h >= a.H) continue;
            char* out = (is_v ? a.v : a.k) + ((tok * a.H + h) * D + unit * 8) * static_cast<int64_t>(sizeof(TOut));
            if constexpr (POOL == KV_F32) {
                __stcs(reinterpret_cast<uint4*>(out), x[j]);
                __stcs(reinterpret_cast<uint4*>(out) + 1, y[j]);
            } else if constexpr (POOL == KV_F16 && sizeof(TOut) == 2) {
                __stcs(reinterpret_cast<uint4*>(out), x[j]);
            } else {
                float f[8];
                if constexpr (POOL == KV_F16) {
                    Raw<__half> raw;
                    raw.a = x[j];
                    widen(raw, f);
                } else {
                    const float sc = is_v ? vs : ks;
                    const uint32_t w[2] = {x[j].x, x[j].y};
                    #pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 e = e4m3x2_to_float2(static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1))));
                        f[2 * i] = e.x * sc;
                        f[2 * i + 1] = e.y * sc;
                    }
                }
                store_eight<TOut>(out, f);
            }
        }
    }
}

// 8 float16 values to the output type
template <typename TOut>
__device__ __forceinline__ void store_halves(char* out, const uint4 v) {
    if constexpr (sizeof(TOut) == 2) {
        __stcs(reinterpret_cast<uint4*>(out), v);
    } else {
        Raw<__half> raw;
        raw.a = v;
        float f[8];
        widen(raw, f);
        store_eight<TOut>(out, f);
    }
}

// 4-bit pools: a CTA takes 8 tokens, a warp one head of them at a time.  Where the tokens are the 8 of
// one oct in order (a cached prefix), K comes as 128-byte pieces that hold whole rows, and V as the
// attention kernel reads it, 16 (D 64: 8) bytes per lane holding a chunk of two tokens; lanes of
// neighbouring chunks then swap halves so that a store fills whole 32-byte sectors.  Other tokens go
// one per half-warp.  Bound: HBM, most of it the output.
template <int D, typename TOut>
__global__ void __launch_bounds__(kGatherThreads) gather_int4_kernel(const __grid_constant__ GatherArgs a) {
    constexpr int OCT = Int4<D>::OCT, CODES = Int4<D>::CODES, WORDS = Int4<D>::WORDS, ES = sizeof(TOut);
    constexpr int UPR = D / 8;                         // units of 8 elements per row
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * 8;
    const int opb = a.B >> 3;
    int64_t slot = tok0 + (lane & 7) < a.n ? a.slots[tok0 + (lane & 7)] : -1;
    if (slot >= a.num_slots) {
        atomicOr(a.err, KV_DEVERR_SLOT);
        slot = -1;
    }
    const int64_t first = __shfl_sync(FULL, slot, 0);
    const bool whole = __all_sync(FULL, first >= 0 && (first & 7) == 0 && slot == first + (lane & 7));
    const int64_t row = static_cast<int64_t>(a.H) * D * ES;            // bytes between two tokens of the output
    if (whole) {
        const int64_t blk = first / a.B;
        const int o = static_cast<int>(first - blk * a.B) >> 3;
        #pragma unroll 2
        for (int h = blockIdx.y * kGatherWarps + warp; h < a.H; h += gridDim.y * kGatherWarps) {
            const int64_t at = ((blk * a.H + h) * opb + o) * OCT;
            const char* k = a.kpool + at;
            const char* v = a.vpool + at;
            constexpr int NK = 4 * D / 128, TPK = 8 / NK;              // 128-byte pieces of K, tokens in each
            uint32_t kw[NK], kb[NK], vw[WORDS];
            const int unit = lane % UPR, tk = lane / UPR;
            #pragma unroll
            for (int j = 0; j < NK; ++j) {
                kw[j] = __ldcs(reinterpret_cast<const uint32_t*>(k + j * 128) + lane);
                kb[j] = *reinterpret_cast<const uint8_t*>(k + CODES + (j * TPK + tk) * (D / 16) + unit / 2);
            }
            if constexpr (WORDS == 4) {
                const uint4 x = __ldcs(reinterpret_cast<const uint4*>(v) + lane);
                vw[0] = x.x; vw[1] = x.y; vw[2] = x.z; vw[3] = x.w;
            } else {
                const uint2 x = __ldcs(reinterpret_cast<const uint2*>(v) + lane);
                vw[0] = x.x; vw[1] = x.y;
            }
            const uint32_t vb = *reinterpret_cast<const uint16_t*>(v + CODES + (D == 128 ? g : g >> 1) * 8 + 2 * t);
            char* ko = a.k + tok0 * row + static_cast<int64_t>(h) * D * ES;
            char* vo = a.v + tok0 * row + static_cast<int64_t>(h) * D * ES;
            #pragma unroll
            for (int j = 0; j < NK; ++j) {
                uint32_t p[4];
                int4_expand_full(kw[j], (kb[j] << 7) * 0x00010001u, p);
                store_halves<TOut>(ko + (j * TPK + tk) * row + unit * 8 * ES,
                                   make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410),
                                              __byte_perm(p[0], p[1], 0x7632), __byte_perm(p[2], p[3], 0x7632)));
            }
            const uint32_t sc = __byte_perm(vb, 0, 0x4140) << 7;
            uint32_t e[2][2 * WORDS];                  // [token][pairs of the chunk's elements]
            #pragma unroll
            for (int w = 0; w < WORDS; ++w) {
                uint32_t p[4];
                int4_expand_full(vw[w], sc, p);
                e[0][2 * w] = __byte_perm(p[0], p[1], 0x5410);
                e[0][2 * w + 1] = __byte_perm(p[2], p[3], 0x5410);
                e[1][2 * w] = __byte_perm(p[0], p[1], 0x7632);
                e[1][2 * w + 1] = __byte_perm(p[2], p[3], 0x7632);
            }
            #pragma unroll
            for (int i = 0; i < 2; ++i) {              // token 2t + i, elements g*D/8 ..
                char* out = vo + (2 * t + i) * row;
                if constexpr (D == 64) {
                    store_halves<TOut>(out + g * 8 * ES, make_uint4(e[i][0], e[i][1], e[i][2], e[i][3]));
                } else if constexpr (ES == 4) {
                    store_halves<TOut>(out + g * 16 * ES, make_uint4(e[i][0], e[i][1], e[i][2], e[i][3]));
                    store_halves<TOut>(out + (g * 16 + 8) * ES, make_uint4(e[i][4], e[i][5], e[i][6], e[i][7]));
                } else {
                    const bool odd = g & 1;
                    uint32_t x[4], own[4];
                    #pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        x[w] = __shfl_xor_sync(FULL, odd ? e[i][w] : e[i][4 + w], 4);
                        own[w] = odd ? e[i][4 + w] : e[i][w];
                    }
                    const uint4 mine = make_uint4(own[0], own[1], own[2], own[3]), other = make_uint4(x[0], x[1], x[2], x[3]);
                    char* pair = out + (g & ~1) * 32 + (odd ? 16 : 0);
                    store_halves<TOut>(pair, odd ? other : mine);
                    store_halves<TOut>(pair + 32, odd ? mine : other);
                }
            }
        }
        return;
    }
    constexpr int HPW = 16 / UPR;                      // head rows per half-warp
    const int unit = lane & (UPR - 1), sub = (lane & 15) / UPR;
    const int uk = (a.H + HPW - 1) / HPW;
    for (int pair = 0; pair < 4; ++pair) {
        const int64_t tok = tok0 + pair * 2 + (lane >> 4);
        const int64_t s = __shfl_sync(FULL, slot, pair * 2 + (lane >> 4));
        if (s < 0) continue;                           // no shuffles below
        const int64_t blk = s / a.B;
        const int off = static_cast<int>(s - blk * a.B), token = off & 7, e0 = unit * 8;
        #pragma unroll 2
        for (int r = blockIdx.y * kGatherWarps + warp; r < 2 * uk; r += gridDim.y * kGatherWarps) {
            const bool is_v = r >= uk;
            const int h = (is_v ? r - uk : r) * HPW + sub;
            if (h >= a.H) continue;
            const char* oct = (is_v ? a.vpool : a.kpool) + ((blk * a.H + h) * opb + (off >> 3)) * OCT;
            uint32_t w, b, p[4];
            if (is_v) {
                w = *reinterpret_cast<const uint16_t*>(oct + int4_v_piece<D>(token, e0)) |
                    static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(oct + int4_v_piece<D>(token, e0 + 4))) << 16;
                b = *reinterpret_cast<const uint8_t*>(oct + int4_v_scale<D>(token, e0));
            } else {
                w = *reinterpret_cast<const uint32_t*>(oct + int4_k_code<D>(token, e0));
                b = *reinterpret_cast<const uint8_t*>(oct + int4_k_scale<D>(token, e0));
            }
            int4_expand_full(w, (b << 7) * 0x00010001u, p);
            store_halves<TOut>((is_v ? a.v : a.k) + tok * row + (static_cast<int64_t>(h) * D + e0) * ES,
                               make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410),
                                          __byte_perm(p[0], p[1], 0x7632), __byte_perm(p[2], p[3], 0x7632)));
        }
    }
}

template <typename TOut>
void gather_int4(const kv_pool* pool, const GatherArgs& a, cudaStream_t stream) {
    const int octs = a.n / 8 + (a.n % 8 != 0), most = (a.H + kGatherWarps - 1) / kGatherWarps;
    // few tokens: the heads spread over CTAs (4, 8 or 16 an SM make no difference: 3.7 us for 512 tokens of 40 heads)
    int gy = (8 * pool->num_sms - 1) / octs + 1;
    gy = gy < 1 ? 1 : gy > most ? most : gy;
    const dim3 grid(static_cast<unsigned>(octs), static_cast<unsigned>(gy));
    if (pool->desc.head_dim == 128) gather_int4_kernel<128, TOut><<<grid, kGatherThreads, 0, stream>>>(a);
    else gather_int4_kernel<64, TOut><<<grid, kGatherThreads, 0, stream>>>(a);
}

template <kv_dtype POOL, typename TOut>
void gather_typed(const kv_pool* pool, const GatherArgs& a, cudaStream_t stream) {
    const int D = pool->desc.head_dim;
    const int hpw = 16 / (D / 8), rows = 2 * ((a.H + hpw - 1) / hpw), pairs = a.n / 2 + a.n % 2;
    const int most = (rows + kGatherWarps - 1) / kGatherWarps;
    // few tokens: the heads spread over CTAs (4, 8, 16 an SM: 4.7, 5.0, 6.9 us for 512 float16 tokens of 40 heads;
    // 2.2 us for 64 and 99.8 for 16384 with each)
    int gy = (8 * pool->num_sms - 1) / pairs + 1;
    gy = gy < 1 ? 1 : gy > most ? most : gy;
    const dim3 grid(static_cast<unsigned>(pairs), static_cast<unsigned>(gy));
    if (D == 128) gather_kernel<128, POOL, TOut><<<grid, kGatherThreads, 0, stream>>>(a);
    else gather_kernel<64, POOL, TOut><<<grid, kGatherThreads, 0, stream>>>(a);
}

}  // namespace

int launch_gather(const kv_pool* pool, int layer, const int64_t* slot_mapping, int num_tokens, void* k_out,
                  void* v_out, kv_dtype out_dtype, cudaStream_t stream) {
    const RopeArgs p = pool_side(pool, layer);
    GatherArgs a{};
    a.kpool = p.kpool;
    a.vpool = p.vpool;
    a.kscale = p.kscale;
    a.vscale = p.vscale;
    a.slots = slot_mapping;
    a.k = static_cast<char*>(k_out);
    a.v = static_cast<char*>(v_out);
    a.n = num_tokens;
    a.H = p.H;
    a.B = p.B;
    a.num_slots = p.num_slots;
    a.err = p.err;
    const bool half = out_dtype == KV_F16;
    switch (pool->desc.dtype) {
        case KV_F32: gather_typed<KV_F32, float>(pool, a, stream); break;
        case KV_F16: half ? gather_typed<KV_F16, __half>(pool, a, stream) : gather_typed<KV_F16, float>(pool, a, stream); break;
        case KV_FP8_E4M3:
            half ? gather_typed<KV_FP8_E4M3, __half>(pool, a, stream) : gather_typed<KV_FP8_E4M3, float>(pool, a, stream);
            break;
        default: half ? gather_int4<__half>(pool, a, stream) : gather_int4<float>(pool, a, stream);
    }
    return cudaGetLastError() == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

// ---------------------------------------------------------------- rotation table
namespace {

// One thread per (position, frequency): the angle, its cosine and sine in 64 bits, rounded once.
// (A float32 angle of position 10^5 would be off by up to 2^-8.)
__global__ void rope_table_kernel(float* table, int64_t total, int half, double base, double position_scale) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= total) return;
    const int64_t pos = i / half;
    const int f = static_cast<int>(i - pos * half);
    const double angle = static_cast<double>(pos) * position_scale * pow(base, -static_cast<double>(f) / half);
    double sn, cs;
    sincos(angle, &sn, &cs);
    float* row = table + pos * 2 * half;
    row[f] = static_cast<float>(cs);
    row[half + f] = static_cast<float>(sn);
}

}  // namespace

int launch_rope_table(float* table, int num_positions, int rot_dim, double base, double position_scale,
                      cudaStream_t stream) {
    const int64_t total = static_cast<int64_t>(num_positions) * (rot_dim / 2);
    rope_table_kernel<<<static_cast<unsigned>((total + 255) / 256), 256, 0, stream>>>(table, total, rot_dim / 2, base,
                                                                                    position_scale);
    return cudaGetLastError() == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

}  // namespace kvp
