// Stored rows of FP8 and 4-bit pools, brought into shared memory as they are, widened to float16 there.
#pragma once

#include "int4.cuh"

#ifdef __CUDACC__
namespace kvp {

// ROWS tokens of one head (whole octs of a 4-bit tile) at `raw`, by THREADS threads (this one: tid), 8 elements at a
// time to *place(row, element / 8).  Every conversion is exact.  Values outside [from, to) become zero (what lies
// there may be anything, and it meets weights of zero); keys there are whatever they are.
template <int D, kv_dtype POOL, bool IS_V, int ROWS, int THREADS, typename Place>
__device__ __forceinline__ void widen_rows(const char* raw, int from, int to, int tid, Place place) {
    const uint4 none = make_uint4(0, 0, 0, 0);
    auto live = [&](int r) { return !IS_V || (r >= from && r < to); };
    if constexpr (POOL == KV_FP8_E4M3) {
        constexpr int PER = D / 16;                            // 16-code pieces of a row
        #pragma unroll 4
        for (int u = tid; u < ROWS * PER; u += THREADS) {
            const int r = u / PER, ch = u % PER * 2;
            const uint4 v = *reinterpret_cast<const uint4*>(raw + u * 16);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t h[8];
            #pragma unroll
            for (int k = 0; k < 8; ++k) h[k] = e4m3x2_to_half2_bits(static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1))));
            *place(r, ch) = live(r) ? make_uint4(h[0], h[1], h[2], h[3]) : none;
            *place(r, ch + 1) = live(r) ? make_uint4(h[4], h[5], h[6], h[7]) : none;
        }
    } else if constexpr (!IS_V) {
        #pragma unroll 4
        for (int u = tid; u < ROWS * (D / 8); u += THREADS) {
            const int r = u / (D / 8), ch = u % (D / 8);
            const char* oct = raw + (r >> 3) * Int4<D>::OCT;
            const uint32_t w = *reinterpret_cast<const uint32_t*>(oct + int4_k_code<D>(r & 7, ch * 8));
            const uint32_t sc = *reinterpret_cast<const uint8_t*>(oct + int4_k_scale<D>(r & 7, ch * 8));
            uint32_t x[4];
            int4_expand_full(w, (sc << 7) | (sc << 23), x);
            *place(r, ch) = make_uint4(__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410),
                                       __byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x7632));
        }
    } else {
        #pragma unroll 2
        for (int u = tid; u < ROWS / 2 * (D / 8); u += THREADS) {      // 8 elements of two tokens
            const int r = u / (D / 8) * 2, ch = u % (D / 8);
            const char* oct = raw + (r >> 3) * Int4<D>::OCT;
            const uint2 w = *reinterpret_cast<const uint2*>(oct + int4_v_piece<D>(r & 7, ch * 8));
            const uint32_t sc = *reinterpret_cast<const uint16_t*>(oct + int4_v_scale<D>(r & 7, ch * 8));
            const uint32_t scales = (sc & 0xFFu) << 7 | (sc & 0xFF00u) << 15;
            uint32_t x[4], y[4];
            int4_expand_full(w.x, scales, x);
            int4_expand_full(w.y, scales, y);
            *place(r, ch) = live(r) ? make_uint4(__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410),
                                                 __byte_perm(y[0], y[1], 0x5410), __byte_perm(y[2], y[3], 0x5410)) : none;
            *place(r + 1, ch) = live(r + 1) ? make_uint4(__byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x7632),
                                                         __byte_perm(y[0], y[1], 0x7632), __byte_perm(y[2], y[3], 0x7632))
                                            : none;
        }
    }
}

}  // namespace kvp
#endif  // __CUDACC__
