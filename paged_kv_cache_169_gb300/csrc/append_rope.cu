// kv_append_rope: new tokens' queries and keys rotated by their positions, keys and values written
// into their slots, in one launch; kv_append into 4-bit pools (the same kernel without rotation);
// kv_gather, its inverse (cached tokens back as contiguous rows); kv_rope_table.
//
// Rotation (rotary position embedding): with angle a = position * frequency_i, elements (x, y) of
// pair i become (x cos a - y sin a, y cos a + x sin a).  Products and sums are float32, rounded
// separately (no contraction), from a float32 table of cosines and sines; the only rounding to
// fewer bits is the store (float16; FP8 and 4-bit codes are quantised from the float32 value).
//
// Layout of the work: a half-warp holds whole head rows, 8 elements (a unit) per lane, so a unit's
// partner under either pairing and the other half of its quantisation group are a shuffle away
// and every input is read once.  The two half-warps take two consecutive tokens: where their slots
// share a 32-bit word of a 4-bit V tile (slot 2m and 2m + 1), the pair of lanes writes whole words.
// A warp walks over its head rows (queries, then keys, then values) with its token's table values in
// registers.  Rows come through shared memory by cp.async, eight ahead: kept in registers, four at a
// time, too few bytes were in flight (57.4 us for 8192 tokens of 64 + 8 heads into float16).  A CTA per
// token pair in launch order keeps the addresses in use together; equal ranges of rows per warp over the
// whole call, with no tail, took 61.6 us.
// Bound: HBM (52.4 us for the float16 prompt, 0.95 of a copy's rate).  With a 4-bit pool, the instructions
// that quantise: 4097 tokens of 40 + 40 heads take 41.8 us (0.68), without quantising 34.2, without the
// stores 39.6, without both 31.7.

#include <type_traits>

#include "int4.cuh"
#include "pool_types.cuh"

namespace kvp {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kThreads = 128, kWarpsPerCta = kThreads / 32;           // append
constexpr int kGatherThreads = 256, kGatherWarps = kGatherThreads / 32;

struct RopeArgs {
    const char *q, *k, *v;
    char* q_out;
    int64_t q_stride, k_stride, v_stride, qo_stride;   // bytes between tokens
    const int64_t* slots;
    const int32_t* positions;
    const float* table;
    int table_len, rot, adjacent;
    char *kpool, *vpool;
    const float *kscale, *vscale;
    int n, Hq, H, B;
    int64_t num_slots;
    int* err;
};

// 8 elements of type TIn as float
template <typename TIn> struct Raw;
template <> struct Raw<__half> { uint4 a; };
template <> struct Raw<float> { float4 a, b; };

__device__ __forceinline__ void widen(const Raw<__half>& r, float (&x)[8]) {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void widen(const Raw<float>& r, float (&x)[8]) {
    x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w;
    x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
}

__device__ __forceinline__ uint4 halves(const float (&x)[8]) {
    uint4 r;
    const __half2 h0 = __floats2half2_rn(x[0], x[1]), h1 = __floats2half2_rn(x[2], x[3]);
    const __half2 h2 = __floats2half2_rn(x[4], x[5]), h3 = __floats2half2_rn(x[6], x[7]);
    r.x = *reinterpret_cast<const uint32_t*>(&h0);
    r.y = *reinterpret_cast<const uint32_t*>(&h1);
    r.z = *reinterpret_cast<const uint32_t*>(&h2);
    r.w = *reinterpret_cast<const uint32_t*>(&h3);
    return r;
}

template <typename TOut>
__device__ __forceinline__ void store_eight(char* out, const float (&f)[8]) {
    if constexpr (sizeof(TOut) == 2) {
        __stcs(reinterpret_cast<uint4*>(out), halves(f));
    } else {
        __stcs(reinterpret_cast<float4*>(out), make_float4(f[0], f[1], f[2], f[3]));
        __stcs(reinterpret_cast<float4*>(out) + 1, make_float4(f[4], f[5], f[6], f[7]));
    }
}

// Stores of one unit (8 elements of a row) into a pool, at the lane's address for head 0 (`at`, and for
// 4-bit tiles `sc`, its group's scale byte); `head` is the byte offset of the row's head.
// paired: lane ^ 16 holds the same unit of the token that shares this one's words of a 4-bit V tile.
template <kv_dtype POOL, bool IS_V>
__device__ __forceinline__ void store_unit(char* at, char* sc, int64_t head, float (&x)[8], float scale, bool paired,
                                           bool odd, bool live, int lane) {
    at += head;
    if constexpr (POOL == KV_F32) {
        if (!live) return;
        reinterpret_cast<float4*>(at)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(at)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else if constexpr (POOL == KV_F16) {
        if (live) *reinterpret_cast<uint4*>(at) = halves(x);
    } else if constexpr (POOL == KV_FP8_E4M3) {
        uint2 c;
        c.x = float2_to_e4m3x2(__fdiv_rn(x[0], scale), __fdiv_rn(x[1], scale)) |
              static_cast<uint32_t>(float2_to_e4m3x2(__fdiv_rn(x[2], scale), __fdiv_rn(x[3], scale))) << 16;
        c.y = float2_to_e4m3x2(__fdiv_rn(x[4], scale), __fdiv_rn(x[5], scale)) |
              static_cast<uint32_t>(float2_to_e4m3x2(__fdiv_rn(x[6], scale), __fdiv_rn(x[7], scale))) << 16;
        if (live) *reinterpret_cast<uint2*>(at) = c;
    } else {
        float amax = max_nan(max_nan(max_nan(fabsf(x[0]), fabsf(x[1])), max_nan(fabsf(x[2]), fabsf(x[3]))),
                             max_nan(max_nan(fabsf(x[4]), fabsf(x[5])), max_nan(fabsf(x[6]), fabsf(x[7]))));
        amax = max_nan(amax, __shfl_xor_sync(FULL, amax, 1));          // the group's other unit
        const uint32_t sb = int4_scale_byte(amax);
        const uint32_t w = int4_nibbles<8>(x, amax, int4_scale_value(sb));
        if constexpr (!IS_V) {
            if (!live) return;
            *reinterpret_cast<uint32_t*>(at) = w;
        } else {
            // the unit's two pieces lie in two consecutive words, each shared with the token's neighbour:
            // paired, the even token writes the first word, the odd token the second
            const uint32_t other = __shfl_xor_sync(FULL, w, 16);
            if (!live) return;
            if (paired) {
                *reinterpret_cast<uint32_t*>(at) = odd ? __byte_perm(other, w, 0x7632) : __byte_perm(w, other, 0x5410);
            } else {
                *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(w);
                *reinterpret_cast<uint16_t*>(at + 4) = static_cast<uint16_t>(w >> 16);
            }
        }
        if ((lane & 1) == 0) *reinterpret_cast<uint8_t*>(sc + head) = sb;
    }
}

// Rows a warp has asked for ahead of the one it works on (4, 8, 16: 54.1, 52.4, 55.2 us for the float16
// prompt), 16 KB per CTA whatever the type.
template <typename TIn> constexpr int kRowsAhead = sizeof(TIn) == 2 ? 8 : 4;
// CTAs per SM: quantising takes more registers (6, 7, 8: 57.7, 59.0, 63.0 us for the 4-bit prompt).
template <kv_dtype POOL> constexpr int kCtasPerSm = POOL == KV_INT4 ? 6 : 7;

enum : int { NO_ROTATION = 0, HALF_PAIRS = 1, ADJACENT_PAIRS = 2 };

template <int D, typename TIn, kv_dtype POOL, int MODE>
__global__ void __launch_bounds__(kThreads, kCtasPerSm<POOL>) append_rope_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int UPR = D / 8, HPW = 16 / UPR;         // units per row; head rows per half-warp
    constexpr int ESZ = sizeof(TIn), QSZ = POOL == KV_F32 ? 4 : 2;
    constexpr int ROW = POOL == KV_INT4 ? D / 2 + D / 16 : POOL == KV_FP8_E4M3 ? D : POOL == KV_F16 ? 2 * D : 4 * D;
    constexpr int AHEAD = kRowsAhead<TIn>, PIECES = ESZ / 2;           // 16-byte pieces of a unit
    __shared__ uint4 s_ring[kWarpsPerCta][AHEAD][PIECES][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int unit = lane & (UPR - 1), sub = (lane & 15) / UPR;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t tok = static_cast<int64_t>(blockIdx.x) * 2 + (lane >> 4);
    // ---- The head rows: queries, keys, values, HPW rows per half-warp and step, dealt to the warps in
    // turn.  A lane copies its own 16 bytes of each row to shared memory, several rows ahead, and reads
    // them back itself, so it waits for its own copies only.  The first rows are asked for before anything
    // is known of the token (one past the end takes its neighbour's).
    const int uq = (a.Hq + HPW - 1) / HPW, uk = (a.H + HPW - 1) / HPW, rows = uq + 2 * uk;
    const int start = blockIdx.y * kWarpsPerCta + warp, step = gridDim.y * kWarpsPerCta;
    const int64_t from = tok < a.n ? tok : tok - 1;
    constexpr int STEP = HPW * D * ESZ;                // bytes between a half-warp's steps
    uint4* const ring = &s_ring[warp][0][0][lane];
    const uint32_t ring32 = smem_u32(ring);
    int ask_row = start, ask_end = 0, ask_slot = 0;    // the next row to ask for, its matrix's end, its place
    const char* ask_at = nullptr;
    auto ask = [&]() {
        if (ask_row < rows) {
            if (ask_row >= ask_end) {                  // another matrix
                const bool is_q = ask_row < uq, is_k = ask_row < uq + uk;
                const int first = is_q ? 0 : is_k ? uq : uq + uk;
                ask_end = is_q ? uq : is_k ? uq + uk : rows;
                ask_at = (is_q ? a.q : is_k ? a.k : a.v) + from * (is_q ? a.q_stride : is_k ? a.k_stride : a.v_stride) +
                         (ask_row - first) * STEP + (sub * D + unit * 8) * ESZ;
            }
            // an odd head count's last step has a row too many, which reads the last one
            const int heads = ask_end == uq ? a.Hq : a.H;
            const char* at = ask_at - (HPW > 1 && ask_row + 1 == ask_end && (heads & 1) && sub ? D * ESZ : 0);
            #pragma unroll
            for (int i = 0; i < PIECES; ++i) cp_async16(ring32 + (ask_slot * PIECES + i) * 512, at + 16 * i);
            ask_row += step;
            ask_at += step * STEP;
            ask_slot = (ask_slot + 1) % AHEAD;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    #pragma unroll
    for (int i = 0; i < AHEAD - 1; ++i) ask();
    int slot_of_row = 0;
    auto next_row = [&](float (&x)[8]) {               // the next row, and one more asked for
        asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 2) : "memory");
        Raw<TIn> raw;
        uint4* const w = reinterpret_cast<uint4*>(&raw);
        #pragma unroll
        for (int i = 0; i < PIECES; ++i) w[i] = ring[(slot_of_row * PIECES + i) * 32];
        slot_of_row = (slot_of_row + 1) % AHEAD;
        ask();
        widen(raw, x);
    };
    // ---- the token: its slot, its position, its rotation
    int64_t slot = tok < a.n ? a.slots[tok] : -1;
    int pos = 0;
    bool live = slot >= 0;
    if (live && slot >= a.num_slots) {
        atomicOr(a.err, KV_DEVERR_SLOT);
        live = false;
    }
    if (MODE != NO_ROTATION && tok < a.n) {
        pos = a.positions[tok];
        if (pos < 0 || pos >= a.table_len) {
            if (live) atomicOr(a.err, KV_DEVERR_POSITION);
            live = false;
            pos = 0;
        }
    }
    if (!__any_sync(FULL, live)) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        return;
    }
    // this unit's cosines and sines for pairs of elements (half pairs: 8 of each; adjacent pairs: 4 of
    // each, every one for both elements of its pair)
    float2 c[4], s[4];
    const bool turned = unit * 8 < a.rot;
    const int half_units = a.rot >> 4;
    const bool low = unit < half_units;                // half pairs: the first element of each pair
    if constexpr (MODE != NO_ROTATION) {
        // x cos - y sin is taken as x cos + y (-sin): the same roundings
        const float* row = a.table + static_cast<int64_t>(pos) * a.rot;
        const int i0 = !turned ? 0 : MODE == ADJACENT_PAIRS ? unit * 4 : (low ? unit : unit - half_units) * 8;
        if constexpr (MODE == ADJACENT_PAIRS) {
            const float4 cv = *reinterpret_cast<const float4*>(row + i0);
            const float4 sv = *reinterpret_cast<const float4*>(row + a.rot / 2 + i0);
            c[0] = make_float2(cv.x, cv.x); c[1] = make_float2(cv.y, cv.y);
            c[2] = make_float2(cv.z, cv.z); c[3] = make_float2(cv.w, cv.w);
            s[0] = make_float2(-sv.x, sv.x); s[1] = make_float2(-sv.y, sv.y);
            s[2] = make_float2(-sv.z, sv.z); s[3] = make_float2(-sv.w, sv.w);
        } else {
            #pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float4 cv = *reinterpret_cast<const float4*>(row + i0 + 4 * j);
                float4 sv = *reinterpret_cast<const float4*>(row + a.rot / 2 + i0 + 4 * j);
                if (low) sv = make_float4(-sv.x, -sv.y, -sv.z, -sv.w);
                c[2 * j] = make_float2(cv.x, cv.y); c[2 * j + 1] = make_float2(cv.z, cv.w);
                s[2 * j] = make_float2(sv.x, sv.y); s[2 * j + 1] = make_float2(sv.z, sv.w);
            }
        }
    }
    if (!live) slot = 0;
    const int64_t blk = slot / a.B;
    const int off = static_cast<int>(slot - blk * a.B);
    // both tokens live and in one 32-bit word of a 4-bit V tile
    const int64_t other_slot = __shfl_xor_sync(FULL, live ? slot : int64_t{-2}, 16);
    const bool paired = POOL == KV_INT4 && live && other_slot == (slot ^ 1), odd = off & 1;
    float ks = 1.f, vs = 1.f;
    if constexpr (POOL == KV_FP8_E4M3) {
        ks = a.kscale[blk];
        vs = a.vscale[blk];
    }
    // this lane's addresses in the token's block, head `sub`
    const int64_t tile = static_cast<int64_t>(a.B) * ROW, tile0 = (blk * a.H + sub) * tile;
    const int e0 = unit * 8;
    char *kat = a.kpool + tile0, *vat = a.vpool + tile0, *ksc = kat, *vsc = vat;
    if constexpr (POOL == KV_INT4) {
        const int oct = (off >> 3) * Int4<D>::OCT, token = off & 7;
        ksc += oct + int4_k_scale<D>(token, e0);
        vsc += oct + int4_v_scale<D>(token, e0);
        kat += oct + int4_k_code<D>(token, e0);
        vat += oct + (paired ? int4_v_piece<D>(token & ~1, e0 + (odd ? 4 : 0)) : int4_v_piece<D>(token, e0));
    } else {
        kat += off * ROW + e0 * (ROW / D);
        vat += off * ROW + e0 * (ROW / D);
    }
    const int partner = (lane & ~(UPR - 1)) | (turned ? (low ? unit + half_units : unit - half_units) : unit);
    auto rotate = [&](float (&x)[8]) {
        if constexpr (MODE != NO_ROTATION) {
            float y[8];                                // each element's partner
            #pragma unroll
            for (int i = 0; i < 8; ++i)
                y[i] = MODE == ADJACENT_PAIRS ? x[i ^ 1] : __shfl_sync(FULL, x[i], partner);
            if (!turned) return;
            #pragma unroll
            for (int i = 0; i < 4; ++i) {              // two elements at a time, rounded op by op
                const float2 p = __fmul2_rn(make_float2(x[2 * i], x[2 * i + 1]), c[i]);
                const float2 r = __fmul2_rn(make_float2(y[2 * i], y[2 * i + 1]), s[i]);
                x[2 * i] = __fadd_rn(p.x, r.x);        // (a sum of pairs would be contracted)
                x[2 * i + 1] = __fadd_rn(p.y, r.y);
            }
        }
    };
    // ---- queries
    // q_out may be q: a lane writes only elements that it has read (what lanes past the end ask for is not used)
    char* const qo = a.q_out + tok * a.qo_stride + (sub * D + e0) * QSZ;
    int r = start;
    #pragma unroll 1
    for (; r < uq; r += step) {
        float x[8];
        next_row(x);
        rotate(x);
        if (!live || (HPW > 1 && r * HPW + sub >= a.Hq)) continue;
        char* p = qo + r * (HPW * D * QSZ);
        if constexpr (POOL == KV_F32) {
            reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
            reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
        } else {
            *reinterpret_cast<uint4*>(p) = halves(x);
        }
    }
    // ---- keys, then values
    auto cached = [&](auto is_v, char* at, char* sc, float scale) {
        constexpr bool IS_V = decltype(is_v)::value;
        #pragma unroll 1
        for (r -= IS_V ? uk : uq; r < uk; r += step) {
            float x[8];
            next_row(x);
            if constexpr (!IS_V) rotate(x);
            const bool here = live && (HPW == 1 || r * HPW + sub < a.H);
            store_unit<POOL, IS_V>(at, sc, r * HPW * tile, x, scale, paired, odd, here, lane);
        }
    };
    cached(std::integral_constant<bool, false>{}, kat, ksc, ks);
    cached(std::integral_constant<bool, true>{}, vat, vsc, vs);
}

template <typename TIn, kv_dtype POOL>
int launch_rope_typed(const kv_pool* pool, const RopeArgs& a, bool pdl, cudaStream_t stream) {
    const int D = pool->desc.head_dim;
    const int hpw = 16 / (D / 8);
    const int uq = a.Hq ? (a.Hq + hpw - 1) / hpw : 0, rows = uq + 2 * ((a.H + hpw - 1) / hpw);
    const int pairs = a.n / 2 + a.n % 2;
    // a CTA per token pair, or with few tokens as many as are resident at once, down to one row per warp
    const int most = (rows + kWarpsPerCta - 1) / kWarpsPerCta;
    int gy = pool->num_sms * kCtasPerSm<POOL> / pairs;
    gy = gy < 1 ? 1 : gy > most ? most : gy;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(pairs), static_cast<unsigned>(gy));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    auto launch = [&](auto d) {
        constexpr int DIM = decltype(d)::value;
        if (a.rot == 0) {                              // kv_append, which rotates nothing, into 4-bit pools
            if constexpr (POOL == KV_INT4) return cudaLaunchKernelEx(&cfg, append_rope_kernel<DIM, TIn, POOL, NO_ROTATION>, a);
            return cudaErrorInvalidValue;
        }
        return a.adjacent ? cudaLaunchKernelEx(&cfg, append_rope_kernel<DIM, TIn, POOL, ADJACENT_PAIRS>, a)
                          : cudaLaunchKernelEx(&cfg, append_rope_kernel<DIM, TIn, POOL, HALF_PAIRS>, a);
    };
    const cudaError_t rc = D == 128 ? launch(std::integral_constant<int, 128>{}) : launch(std::integral_constant<int, 64>{});
    if (rc != cudaSuccess) {
        cudaGetLastError();
        return KV_ERR_CUDA;
    }
    return KV_OK;
}

int launch_rope_any(const kv_pool* pool, kv_dtype in, const RopeArgs& a, bool pdl, cudaStream_t stream) {
    switch (pool->desc.dtype) {
        case KV_F32: return launch_rope_typed<float, KV_F32>(pool, a, pdl, stream);
        case KV_F16: return launch_rope_typed<__half, KV_F16>(pool, a, pdl, stream);
        case KV_FP8_E4M3:
            return in == KV_F16 ? launch_rope_typed<__half, KV_FP8_E4M3>(pool, a, pdl, stream)
                                : launch_rope_typed<float, KV_FP8_E4M3>(pool, a, pdl, stream);
        default:
            return in == KV_F16 ? launch_rope_typed<__half, KV_INT4>(pool, a, pdl, stream)
                                : launch_rope_typed<float, KV_INT4>(pool, a, pdl, stream);
    }
}

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

int launch_append_rope(const kv_pool* pool, const kv_rope_args& x) {
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
    return launch_rope_any(pool, x.in_dtype, a, (x.flags & KV_DECODE_PDL) != 0, x.stream);
}

int launch_append_int4(const kv_pool* pool, int layer, const void* k, const void* v, kv_dtype in_dtype,
                       const int64_t* slot_mapping, int num_tokens, cudaStream_t stream) {
    RopeArgs a = pool_side(pool, layer);
    a.k = static_cast<const char*>(k);
    a.v = static_cast<const char*>(v);
    a.k_stride = a.v_stride = static_cast<int64_t>(pool->desc.num_heads) * pool->desc.head_dim * elem_bytes(in_dtype);
    a.slots = slot_mapping;
    a.n = num_tokens;
    return launch_rope_any(pool, in_dtype, a, false, stream);
}

// ---------------------------------------------------------------- gather
namespace {

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

// The 8 nibbles of a word as float16 pairs times their scales, exact: p[0] holds nibbles 0 and 4 ..
// p[3] nibbles 3 and 7 (int4.cuh's expansion without the sixteenth, one instruction more).
__device__ __forceinline__ void expand_full(uint32_t w, uint32_t scales, uint32_t (&p)[4]) {
    const __half2 s = *reinterpret_cast<const __half2*>(&scales);
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t u = w >> (i < 2 ? 0 : 8);
        if (i & 1) {
            u = int4_pair<0x00F000F0u>(u, __float2half2_rn(0.0625f), __float2half2_rn(-72.f));
        } else {
            u = int4_pair<0x000F000Fu>(u, __float2half2_rn(1.f), __float2half2_rn(-1032.f));
        }
        const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&u), s);
        p[i] = *reinterpret_cast<const uint32_t*>(&r);
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
                expand_full(kw[j], (kb[j] << 7) * 0x00010001u, p);
                store_halves<TOut>(ko + (j * TPK + tk) * row + unit * 8 * ES,
                                   make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410),
                                              __byte_perm(p[0], p[1], 0x7632), __byte_perm(p[2], p[3], 0x7632)));
            }
            const uint32_t sc = __byte_perm(vb, 0, 0x4140) << 7;
            uint32_t e[2][2 * WORDS];                  // [token][pairs of the chunk's elements]
            #pragma unroll
            for (int w = 0; w < WORDS; ++w) {
                uint32_t p[4];
                expand_full(vw[w], sc, p);
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
            expand_full(w, (b << 7) * 0x00010001u, p);
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
