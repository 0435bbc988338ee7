// Decode attention over 4-bit pools (KV_INT4): the same result, work items, split-context merge
// and launch flags as attention_kernel.cuh, with a consumer made for 4-bit tiles.
//
// Per 16 tokens and K/V head, with the tokens (and the output's elements) as the M side of
// mma.m16n8k16 and the query heads as its N side:
//   S^T  = K Q^T        A = K expanded in registers, B = the query rows (fragments kept per item)
//   softmax             fp32, log2 domain, running maximum raised only when exceeded by 8
//   O^T += V^T P^T      A = V^T expanded in registers, B = P^T from the S accumulators
//                       (movmatrix)
// Up to 4 query heads per K/V head take the even columns and the odd column beside each holds
// the float16 rounding error of its weights (p = hi + lo), so P V is as exact as with float32
// weights at no further mma; 8 query heads fill all columns and p is rounded to float16 once
// (relative 2^-11, as in the other pools' tensor-core consumer).  All sums are float32.
//
// The pool's tile layout (int4.cuh) makes a lane's fragments of 8 tokens one 16-byte load, so the
// data goes from global memory straight to registers: no shared-memory ring, barriers or copies
// (a 16-token tile of one head is 1152 bytes, and every bulk copy costs the SM 80-100 cycles
// whatever its size).  The K words of the next 32 tokens are loaded as soon as those of this
// chunk are multiplied, the V words likewise, so one of the two is always in flight.
//
// Bound: HBM reads of 9/16 byte per element of K and V; the expansion costs 9 instructions per 8
// elements and lane.

#include "attention_kernel.cuh"
#include "int4.cuh"
#include "pool_types.cuh"

namespace kvp {
namespace {

constexpr int kWarps = 8, kCtasPerSm = 2;

template <int WORDS> struct Words { uint32_t w[WORDS]; };

template <int WORDS>
__device__ __forceinline__ void load_words(const char* p, Words<WORDS>& x) {
    if constexpr (WORDS == 4)
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x.w[0]), "=r"(x.w[1]), "=r"(x.w[2]), "=r"(x.w[3]) : "l"(p) : "memory");
    else
        asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                     : "=r"(x.w[0]), "=r"(x.w[1]) : "l"(p) : "memory");
}
__device__ __forceinline__ uint32_t load_u16(const char* p) {
    unsigned short v;
    asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t load_u8(const char* p) {
    uint32_t v;
    asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// byte b0 (bits 0-7) and b1 (bits 8-15) of x as the float16 pair (scale b0, scale b1)
__device__ __forceinline__ uint32_t scales_two(uint32_t x) { return __byte_perm(x, 0, 0x4140) << 7; }
// byte `which` of x as the float16 pair (scale, scale)
__device__ __forceinline__ uint32_t scales_same(uint32_t x, int which) {
    return __byte_perm(x, 0, which ? 0x4141 : 0x4040) << 7;
}

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
    const float s = int4_scale_value(sb), inv = int4_inverse(s);
    uint32_t piece = 0;
    #pragma unroll
    for (int i = 0; i < 4; ++i) piece |= int4_nibble(x[i], s, inv, 7.f * s) << (4 * i);
    if (act) {
        *reinterpret_cast<uint16_t*>(oct + (is_k ? int4_k_code<D>(token, e0) : int4_v_piece<D>(token, e0))) =
            static_cast<uint16_t>(piece);
        if ((lane & 3) == 0)
            *reinterpret_cast<uint8_t*>(oct + (is_k ? int4_k_scale<D>(token, e0) : int4_v_scale<D>(token, e0))) =
                static_cast<uint8_t>(sb);
    }
}

template <int D, int G>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) attention_int4_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int WORDS = Int4<D>::WORDS, OCT = Int4<D>::OCT;
    constexpr int KS = D / 16, MT = D / 16;            // k-steps over the elements; output tiles
    constexpr bool SPLIT = G <= 4;                     // odd columns: the weights' rounding errors
    constexpr int NQ = SPLIT ? 1 : 2;                  // query columns per lane
    constexpr int CT = 32, NO = CT / 8;                // tokens and octs per chunk
    __shared__ int s_ctx[kMaxBatch], s_end[kMaxBatch], s_P;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;

    const bool early = a.early_tables != 0;
    if (!early) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (tid == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    // ---- the launch's work list: items per sequence, inclusive prefix (as attention_kernel.cuh)
    for (int s = tid; s < a.batch; s += kWarps * 32) {
        int c = a.lens[s];
        if (c < 0 || c > a.ctx_limit) {
            if (blockIdx.x == 0) atomicOr(a.err, KV_DEVERR_CONTEXT);
            c = c < 0 ? 0 : a.ctx_limit;
        }
        s_ctx[s] = c;
    }
    __syncthreads();
    if (warp == 0) {
        int P = a.P;
        if (a.P_alt < a.P) {                           // a finer split that still fits one round of items
            int alt = 0;
            for (int s = lane; s < a.batch; s += 32)
                alt += a.H * nparts_of(s_ctx[s] - attend_first(s_ctx[s], a.window, 8), a.P_alt);
            if (__reduce_add_sync(FULL, alt) <= static_cast<int>(gridDim.x) * kWarps) P = a.P_alt;
        }
        int carry = 0;
        for (int base = 0; base < a.batch; base += 32) {
            const int s = base + lane;
            int v = 0;
            if (s < a.batch)
                v = a.H * nparts_of(s_ctx[s] - attend_first(s_ctx[s], a.window, 8),
                                    P == a.P ? part_of(P, a, s) : P);
            #pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int n = __shfl_up_sync(FULL, v, o);
                if (lane >= o) v += n;
            }
            v += carry;
            if (s < a.batch) s_end[s] = v;
            carry = __shfl_sync(FULL, v, 31);
        }
        if (lane == 0) s_P = P;
    }
    __syncthreads();
    const int n_items = s_end[a.batch - 1];
    const int P_eff = s_P;
    // with the finer split every sequence takes it
    const int s_fine = P_eff == a.P ? a.s_fine : a.batch;
    if (early) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (tid == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }

    const int opb = a.B >> 3;                          // octs per (block, head) tile
    const int lg_opb = __ffs(opb) - 1;
    const unsigned first_claim = gridDim.x * kWarps;
    unsigned pending = 0;                              // lane 0: the claimed next item (atomic in flight)
    bool claimed = false;

    // load side: the item whose chunk is loaded next; oct ids of its current and next 32 octs
    Item L{};
    int Lc = 0, Lo0 = 0, Lno = 0;
    int oid = 0, oid_next = 0;
    const char *kp = nullptr, *vp = nullptr;           // this lane's words of oct 0 of the item's head
    auto load_oids = [&](int base) -> int {            // global index of oct base + lane of the item
        const int i = min(base + lane, Lno - 1);
        if (i < 0) return 0;
        const int o = Lo0 + i;
        int id = a.tables[static_cast<int64_t>(L.s) * a.max_blocks + (o >> lg_opb)];
        if (id < 0 || id >= a.num_blocks) {
            atomicOr(a.err, KV_DEVERR_BLOCK_ID);
            id = 0;
        }
        return (id * a.H << lg_opb) + (o & (opb - 1));
    };
    auto begin_item = [&](unsigned idx) {
        L = decode_item<CT>(static_cast<int>(idx), n_items, s_ctx, s_end, a.batch, a.H, P_eff, s_fine, a.P_fine,
                            a.window, 8);
        Lc = 0;
        if (!L.valid) return;
        Lo0 = L.tok0 >> 3;
        Lno = (L.ntok + 7) >> 3;
        const int64_t head = static_cast<int64_t>(L.h) * opb * OCT;
        kp = a.kpool + head + lane * (4 * WORDS);
        vp = a.vpool + head + lane * (4 * WORDS);
        if (a.k_new != nullptr && L.last && L.ntok > 0) {
            // fused append: the newest token goes to its slot before the item's loads
            const int tok = s_ctx[L.s] - 1, o = tok >> 3;
            int id = a.tables[static_cast<int64_t>(L.s) * a.max_blocks + (o >> lg_opb)];
            if (id < 0 || id >= a.num_blocks) id = 0;  // flagged by load_oids
            const int64_t at = (((static_cast<int64_t>(id) * a.H + L.h) << lg_opb) + (o & (opb - 1))) * OCT;
            const int64_t row = (static_cast<int64_t>(L.s) * a.H + L.h) * D * a.in_bytes;
            append_row<D>(a.k_new + row, a.in_bytes, a.kpool + at, tok & 7, true, lane);
            append_row<D>(a.v_new + row, a.in_bytes, a.vpool + at, tok & 7, false, lane);
            __syncwarp();                              // the warp's loads below see the row
        }
        oid = load_oids(0);
        if (Lno > 32) oid_next = load_oids(32);
    };

    Words<WORDS> kw[NO], vw[NO];
    uint32_t ksc[NO], vsc[NO];
    int oc[NO];                                        // oct indices of the loaded chunk
    // lane offsets of the scales from the lane's words
    const int ks_off = OCT - D / 2 - lane * (4 * WORDS) + (D == 128 ? lane * 2 : lane);
    const int vs_off = OCT - D / 2 - lane * (4 * WORDS) + (D == 128 ? g : g >> 1) * 8 + 2 * t;
    auto load_k = [&]() {
        const int w = (Lc * NO) & 31;
        if (w == 0 && Lc > 0) {                        // the next 32 octs
            oid = oid_next;
            if (Lc * NO + 32 < Lno) oid_next = load_oids(Lc * NO + 32);
        }
        #pragma unroll
        for (int j = 0; j < NO; ++j) {
            oc[j] = __shfl_sync(FULL, oid, w + j);
            const char* p = kp + static_cast<int64_t>(oc[j]) * OCT;
            load_words<WORDS>(p, kw[j]);
            ksc[j] = D == 128 ? load_u16(p + ks_off) : load_u8(p + ks_off);
        }
    };
    auto load_v = [&]() {
        #pragma unroll
        for (int j = 0; j < NO; ++j) {
            const char* p = vp + static_cast<int64_t>(oc[j]) * OCT;
            load_words<WORDS>(p, vw[j]);
            vsc[j] = load_u16(p + vs_off);
        }
    };
    // B fragments of Q^T, in the order the K words expand: k-step 2w takes elements (0, 4) and
    // (1, 5) of word w, k-step 2w+1 elements (2, 6) and (3, 7).  The pairs of the odd elements
    // meet full K values, those of the even ones a sixteenth: the odd elements' query values are
    // divided by 16 (exact unless below 2^-10, then off by at most 2^-25) and the score times 16.
    uint32_t qa[KS][2];
    auto load_q = [&]() {
        const int col = SPLIT ? g >> 1 : g;            // query of column g (odd columns: none)
        const bool real = (SPLIT ? (g & 1) == 0 : true) && col < G && L.ntok > 0;
        const __half* qrow = static_cast<const __half*>(a.q) +
                             ((static_cast<int64_t>(L.s) * a.H + L.h) * G + (real ? col : 0)) * D + t * (D / 4);
        #pragma unroll
        for (int w = 0; w < WORDS; ++w) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (real) x = *reinterpret_cast<const uint4*>(qrow + 8 * w);
            const uint32_t e04 = __byte_perm(x.x, x.z, 0x5410), e15 = __byte_perm(x.x, x.z, 0x7632);
            const uint32_t e26 = __byte_perm(x.y, x.w, 0x5410), e37 = __byte_perm(x.y, x.w, 0x7632);
            const __half2 r = __float2half2_rn(0.0625f);
            const __half2 b0 = __hmul2(*reinterpret_cast<const __half2*>(&e15), r);
            const __half2 b1 = __hmul2(*reinterpret_cast<const __half2*>(&e37), r);
            qa[2 * w][0] = e04;
            qa[2 * w][1] = *reinterpret_cast<const uint32_t*>(&b0);
            qa[2 * w + 1][0] = e26;
            qa[2 * w + 1][1] = *reinterpret_cast<const uint32_t*>(&b1);
        }
    };

    float ot[MT][4];
    float m[NQ], l[NQ];
    Ticket tk{};
    const float xs = a.qscale * 16.f;

    begin_item(warp * gridDim.x + blockIdx.x);
    if (L.valid) {
        load_q();
        if (L.ntok > 0) {
            load_k();
            load_v();
        }
    }
    while (L.valid) {
        const int c = Lc, nch = L.nchunks;
        const int nt = min(CT, L.ntok - c * CT), lo = c == 0 ? L.lo : 0;
        const int is = L.s, ih = L.h, ip = L.p;
        const bool single = L.single, last = c == nch - 1;
        if (c == 0) {
            #pragma unroll
            for (int q = 0; q < NQ; ++q) { m[q] = -CUDART_INF_F; l[q] = 0.f; }
            #pragma unroll
            for (int i = 0; i < MT; ++i) { ot[i][0] = ot[i][1] = ot[i][2] = ot[i][3] = 0.f; }
        }
        // ---- S^T = K Q^T for two steps of 16 tokens
        float x[2][2 * NQ];                            // [step][token g, token g + 8] (x query columns)
        if (nt > 0) {
            #pragma unroll
            for (int u = 0; u < 2; ++u) {
                float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
                #pragma unroll
                for (int h = 0; h < 2; ++h) {          // the lane's two scale groups (D 64: one)
                    if (D == 64 && h == 1) continue;
                    const Int4Scale s0 = int4_scale_pair(scales_same(ksc[2 * u], h));
                    const Int4Scale s1 = int4_scale_pair(scales_same(ksc[2 * u + 1], h));
                    #pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const int w = 2 * h + v;
                        uint32_t p0[4], p1[4];
                        int4_expand(kw[2 * u].w[w], s0, p0);
                        int4_expand(kw[2 * u + 1].w[w], s1, p1);
                        mma_16816(sa, p0[0], p1[0], p0[1], p1[1], qa[2 * w][0], qa[2 * w][1]);
                        mma_16816(sb, p0[2], p1[2], p0[3], p1[3], qa[2 * w + 1][0], qa[2 * w + 1][1]);
                    }
                }
                const int t0 = 16 * u + g, t1 = t0 + 8;
                const bool v0 = t0 >= lo && t0 < nt, v1 = t1 >= lo && t1 < nt;
                #pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    x[u][q] = v0 ? (sa[q] + sb[q]) * xs : -CUDART_INF_F;
                    x[u][NQ + q] = v1 ? (sa[2 + q] + sb[2 + q]) * xs : -CUDART_INF_F;
                }
            }
        }
        // ---- next chunk: claim, switch items, load K (and the next item's queries)
        if (nch - 1 - c <= 2 && !claimed) {
            if (lane == 0) pending = atomicAdd(a.counter, 1u) + first_claim;
            claimed = true;
        }
        if (last) {
            begin_item(__shfl_sync(FULL, pending, 0));
            claimed = false;
            if (L.valid) load_q();
        } else {
            ++Lc;
        }
        const bool more = L.valid && L.ntok > 0;
        if (more) {
            // the V words of this chunk are still needed: their oct indices are not
            load_k();
        }
        if (nt > 0) {
            // ---- softmax over the chunk
            #pragma unroll
            for (int q = 0; q < NQ; ++q) {
                float mx = fmaxf(fmaxf(x[0][q], x[0][NQ + q]), fmaxf(x[1][q], x[1][NQ + q]));
                if (__any_sync(FULL, mx > m[q] + 8.f)) {
                    #pragma unroll
                    for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, o));
                    const float m_new = fmaxf(m[q], mx), corr = ex2_approx(m[q] - m_new);
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
            const bool part = nt < CT || lo > 0;
            #pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint32_t pb0, pb1;
                if constexpr (SPLIT) {
                    const float p0 = ex2_approx(x[u][0] - m[0]), p1 = ex2_approx(x[u][1] - m[0]);
                    l[0] += p0 + p1;
                    const float h0 = __half2float(__float2half_rn(p0)), h1 = __half2float(__float2half_rn(p1));
                    pb0 = movmatrix_t(pack_half2(h0, p0 - h0));
                    pb1 = movmatrix_t(pack_half2(h1, p1 - h1));
                } else {
                    const float p00 = ex2_approx(x[u][0] - m[0]), p01 = ex2_approx(x[u][1] - m[NQ - 1]);
                    const float p10 = ex2_approx(x[u][NQ] - m[0]), p11 = ex2_approx(x[u][2 * NQ - 1] - m[NQ - 1]);
                    l[0] += p00 + p10;
                    l[NQ - 1] += p01 + p11;
                    pb0 = movmatrix_t(pack_half2(p00, p01));
                    pb1 = movmatrix_t(pack_half2(p10, p11));
                }
                // ---- O^T += V^T P^T; rows outside [lo, nt) may hold anything: their scales are zeroed
                uint32_t b0 = vsc[2 * u], b1 = vsc[2 * u + 1];
                if (part) {
                    const int r = 16 * u + 2 * t;
                    if (r < lo || r >= nt) b0 &= 0xFF00u;
                    if (r + 1 < lo || r + 1 >= nt) b0 &= 0x00FFu;
                    if (r + 8 < lo || r + 8 >= nt) b1 &= 0xFF00u;
                    if (r + 9 < lo || r + 9 >= nt) b1 &= 0x00FFu;
                }
                const Int4Scale s0 = int4_scale_pair(scales_two(b0)), s1 = int4_scale_pair(scales_two(b1));
                #pragma unroll
                for (int w = 0; w < WORDS; ++w) {
                    uint32_t e0[4], e1[4];
                    int4_expand(vw[2 * u].w[w], s0, e0);
                    int4_expand(vw[2 * u + 1].w[w], s1, e1);
                    mma_16816(ot[2 * w], e0[0], e0[1], e1[0], e1[1], pb0, pb1);
                    mma_16816(ot[2 * w + 1], e0[2], e0[3], e1[2], e1[3], pb0, pb1);
                }
            }
        }
        if (more) load_v();
        ticket_resolve<D, G>(a, tk, lane);             // the previous item's ticket
        if (last) {
            #pragma unroll
            for (int q = 0; q < NQ; ++q) {
                #pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[q] += __shfl_xor_sync(FULL, l[q], o);
            }
            const int64_t shk = static_cast<int64_t>(is) * a.H + ih;
            #pragma unroll
            for (int q = 0; q < NQ; ++q) {
                const int query = SPLIT ? t : 2 * t + q;
                if (query >= G) continue;
                const int64_t sq = shk * G + query;
                const float f = single ? (nt > 0 ? 1.f / l[q] : 0.f) : 1.f;
                // this lane: elements g*D/8 .. of its query; tile i holds elements 2i and 2i+1,
                // the even one as a sixteenth
                float o[2 * MT];
                #pragma unroll
                for (int i = 0; i < MT; ++i) {
                    o[2 * i] = (SPLIT ? ot[i][0] + ot[i][1] : ot[i][q]) * 16.f * f;
                    o[2 * i + 1] = (SPLIT ? ot[i][2] + ot[i][3] : ot[i][2 + q]) * f;
                }
                if (single && a.out_f16) {             // rounded once, from the float32 result
                    __half2* dst = reinterpret_cast<__half2*>(static_cast<__half*>(a.out) + sq * D + g * (D / 8));
                    #pragma unroll
                    for (int i = 0; i < MT; ++i) dst[i] = __floats2half2_rn(o[2 * i], o[2 * i + 1]);
                    continue;
                }
                float* dst;
                if (single) {
                    dst = static_cast<float*>(a.out) + sq * D;
                } else {
                    const int64_t idx = sq * a.max_parts + ip;
                    if (g == 0) {
                        a.part_ml[2 * idx] = m[q];
                        a.part_ml[2 * idx + 1] = l[q];
                    }
                    dst = a.part_o + idx * D;
                }
                float4* d4 = reinterpret_cast<float4*>(dst + g * (D / 8));
                #pragma unroll
                for (int i = 0; i < MT / 2; ++i)
                    d4[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
            if (!single) {
                const int ctx = s_ctx[is];
                const int P = is >= s_fine ? a.P_fine : P_eff;
                ticket_issue(a, tk, shk, ip, nparts_of(ctx - attend_first(ctx, a.window, 8), P), lane);
            }
        }
    }
    ticket_resolve<D, G>(a, tk, lane);
    // every claim of this CTA is made and read: the last CTA of the launch leaves the work and
    // exit counters zero for the next call on this workspace
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        if (atomicAdd(a.exit_counter, 1u) == gridDim.x - 1) {
            *reinterpret_cast<volatile unsigned*>(a.counter) = 0u;
            *reinterpret_cast<volatile unsigned*>(a.exit_counter) = 0u;
        }
    }
}

template <int D, int G>
int launch_d(const kv_pool* pool, const AttnArgs& args, const AttnPlan& plan, unsigned* counters,
             cudaStream_t stream) {
    const int total = args.batch;
    for (int s0 = 0, sub = 0; s0 < total; s0 += kMaxBatch, ++sub) {
        AttnArgs sa = args;
        sa.batch = total - s0 < kMaxBatch ? total - s0 : kMaxBatch;
        const int64_t rows = static_cast<int64_t>(s0) * args.H;     // (sequence, K/V head) rows before this launch
        sa.q = static_cast<const char*>(args.q) + rows * G * D * 2;
        sa.out = static_cast<char*>(args.out) + rows * G * D * (args.out_f16 ? 2 : 4);
        sa.tables = args.tables + static_cast<int64_t>(s0) * args.max_blocks;
        sa.lens = args.lens + s0;
        if (args.k_new) {
            sa.k_new = args.k_new + rows * D * args.in_bytes;
            sa.v_new = args.v_new + rows * D * args.in_bytes;
        }
        if (args.part_ml) {
            sa.part_ml = args.part_ml + 2 * rows * G * args.max_parts;
            sa.part_o = args.part_o + rows * G * args.max_parts * D;
            sa.arrivals = args.arrivals + rows;
            if (args.grp_arrivals) sa.grp_arrivals = args.grp_arrivals + rows * args.n_grp;
        }
        sa.s_fine = args.s_fine - s0 > 0 ? args.s_fine - s0 : 0;
        sa.s_base = s0;
        sa.counter = counters + sub;
        sa.exit_counter = counters + kMaxSub + sub;
        const int64_t upper = static_cast<int64_t>(sa.batch) * args.H * args.max_parts;
        int64_t grid = (upper + kWarps - 1) / kWarps;
        if (grid > static_cast<int64_t>(pool->num_sms) * kCtasPerSm) grid = static_cast<int64_t>(pool->num_sms) * kCtasPerSm;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(grid < 1 ? 1 : grid));
        cfg.blockDim = dim3(kWarps * 32);
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = (plan.flags & KV_DECODE_PDL) ? 1 : 0;
        if (cudaLaunchKernelEx(&cfg, attention_int4_kernel<D, G>, sa) != cudaSuccess) {
            cudaGetLastError();
            return KV_ERR_CUDA;
        }
    }
    return KV_OK;
}

template <int D>
int launch_g(int group, const kv_pool* pool, const AttnArgs& a, const AttnPlan& plan, unsigned* counters,
             cudaStream_t stream) {
    switch (group) {
        case 1: return launch_d<D, 1>(pool, a, plan, counters, stream);
        case 2: return launch_d<D, 2>(pool, a, plan, counters, stream);
        case 4: return launch_d<D, 4>(pool, a, plan, counters, stream);
        case 8: return launch_d<D, 8>(pool, a, plan, counters, stream);
        default: return KV_ERR_INVALID_ARG;
    }
}

constexpr size_t align256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

int plan_attention_int4(const kv_pool* pool, int batch, int max_context, int partition_tokens, AttnPlan* plan,
                        int group, int window) {
    const kv_pool_desc& d = pool->desc;
    if (batch < 0 || max_context < 0 || window < 0 || batch > kMaxBatch * kMaxSub) return KV_ERR_INVALID_ARG;
    if (!valid_group(d, group)) return KV_ERR_INVALID_ARG;
    // a sliding window bounds the tokens read per sequence (window + up to 7 masked rows)
    const int span = (window > 0 && window + 32 < max_context) ? window + 32 : max_context;
    constexpr int kPartMin = 256, kPartMax = 1024, kPartAlt = 192;
    const int nc = kWarps * kCtasPerSm;
    int P;
    if (partition_tokens > 0) {
        if (partition_tokens % kPartAlign != 0 || partition_tokens > (1 << 24)) return KV_ERR_INVALID_ARG;
        P = partition_tokens;
    } else if (partition_tokens == 0) {
        const int64_t units = static_cast<int64_t>(batch > 0 ? batch : 1) * d.num_heads;
        const int64_t warps = static_cast<int64_t>(pool->num_sms) * nc;
        int64_t parts = group == 1 ? (8 * warps + units - 1) / units : warps / units;
        if (parts < 1) parts = 1;
        int64_t p = (static_cast<int64_t>(span) + parts - 1) / parts;
        p = (p + kPartAlign - 1) / kPartAlign * kPartAlign;
        P = static_cast<int>(p < kPartMin ? kPartMin : p > kPartMax ? kPartMax : p);
    } else {
        return KV_ERR_INVALID_ARG;
    }
    plan->partition = P;
    plan->fine_partition = P;
    plan->fine_from = batch;
    plan->alt_partition = partition_tokens == 0 && group == 1 && P == kPartMin ? kPartAlt : P;
    const int pmin = plan->alt_partition;
    plan->max_parts = span <= pmin ? 1 : (span + pmin - 1) / pmin;
    const int64_t launch_items =
        static_cast<int64_t>(batch < kMaxBatch ? batch : kMaxBatch) * d.num_heads * plan->max_parts;
    if (launch_items > (int64_t{1} << 30)) return KV_ERR_INVALID_ARG;
    plan->consumers = nc;
    plan->group = group;
    plan->window = window;
    plan->flags = 0;
    plan->pairs = false;
    size_t ws = kCounterBytes;                          // work and exit counters
    if (plan->max_parts > 1) {
        const size_t n = static_cast<size_t>(batch) * d.num_heads * group * plan->max_parts;
        ws += plan->arrivals_bytes(batch, d.num_heads);
        ws += align256(n * 2 * sizeof(float));
        ws += align256(n * d.head_dim * sizeof(float));
    }
    plan->ws_bytes = ws;
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
    unsigned* counters = reinterpret_cast<unsigned*>(ws);
    const size_t arrivals_bytes = plan.arrivals_bytes(batch, d.num_heads);
    if (!(plan.flags & KV_DECODE_WORKSPACE_ZEROED) &&
        cudaMemsetAsync(counters, 0, kCounterBytes + arrivals_bytes, stream) != cudaSuccess)
        return KV_ERR_CUDA;
    AttnArgs a{};
    a.kpool = static_cast<char*>(pool->k_layers[layer]);
    a.vpool = static_cast<char*>(pool->v_layers[layer]);
    a.k_new = static_cast<const char*>(k_new);
    a.v_new = static_cast<const char*>(v_new);
    a.in_bytes = in_bytes;
    a.q = q;
    a.out = out;
    a.tables = block_tables;
    a.lens = context_lens;
    if (plan.max_parts > 1) {                           // the workspace of launch_attention_append
        const size_t n = static_cast<size_t>(batch) * d.num_heads * plan.group * plan.max_parts;
        a.arrivals = reinterpret_cast<unsigned*>(ws + kCounterBytes);
        a.grp_arrivals =
            reinterpret_cast<unsigned*>(ws + kCounterBytes + align256(static_cast<size_t>(batch) * d.num_heads * 4));
        a.n_grp = merge_groups(plan.max_parts);
        a.part_ml = reinterpret_cast<float*>(ws + kCounterBytes + arrivals_bytes);
        a.part_o = reinterpret_cast<float*>(ws + kCounterBytes + arrivals_bytes + align256(n * 2 * sizeof(float)));
    }
    a.err = pool->d_err;
    a.batch = batch;
    a.H = d.num_heads;
    a.B = d.block_size;
    a.max_blocks = max_blocks;
    const int64_t lim_tables = static_cast<int64_t>(max_blocks) * d.block_size;
    a.ctx_limit = static_cast<int>(lim_tables < max_context ? lim_tables : max_context);
    a.P = plan.partition;
    a.P_fine = plan.fine_partition;
    a.P_alt = plan.alt_partition;
    a.s_fine = plan.fine_from;
    a.max_parts = plan.max_parts;
    a.num_blocks = d.num_blocks;
    a.early_tables = (plan.flags & KV_DECODE_PDL) && (plan.flags & KV_DECODE_EARLY_TABLES) ? 1 : 0;
    a.out_f16 = (plan.flags & KV_DECODE_OUT_F16) ? 1 : 0;
    a.qscale = scale * 1.4426950408889634f;             // log2(e): softmax evaluated with 2^x
    a.window = plan.window;
    a.fused = k_new != nullptr ? 1 : 0;
    return d.head_dim == 128 ? launch_g<128>(plan.group, pool, a, plan, counters, stream)
                             : launch_g<64>(plan.group, pool, a, plan, counters, stream);
}

}  // namespace kvp
