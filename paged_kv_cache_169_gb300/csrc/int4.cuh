// 4-bit pools (KV_INT4): layout of a (block, head) tile, quantisation and exact expansion.
//
// A tile is block_size / 8 octs (8 consecutive tokens each); an oct is 4*D bytes of codes and
// then one scale byte per token and 16 elements:
//   K codes   [token][D/2 bytes], element 2i in the low nibble of byte i
//   K scales  [token][D/16]
//   V codes   16-bit pieces of 4 elements of one token, element i of a piece at bits 4i:
//             [chunk of D/8 elements][token / 2][D/32 pieces of the chunk][token % 2]
//   V scales  [D/16][token]
// so that in the attention kernel lane (g, t) = (lane / 4, lane % 4) of a warp reads its tensor-
// core fragments of 8 tokens as one contiguous load at lane * D/8: of K, token g's elements
// [t*D/4, (t+1)*D/4); of V, elements [g*D/8, (g+1)*D/8) of tokens 2t and 2t+1, the two tokens'
// elements side by side as the halves of a 32-bit word.
//
// value = code * scale, code = nibble - 8 in -7 .. 7.  The scale byte is an unsigned float of 5
// exponent and 3 mantissa bits with float16's exponent bias: (byte << 7) is the scale as float16.
// A scale has 4 significant bits and a code 3, so code * scale is exact in float16; scales stop
// at 896, which keeps every step of the expansion below in float16's range (|value| <= 6272).
#pragma once

#include "kvp_internal.cuh"

namespace kvp {

template <int D> struct Int4 {
    static constexpr int OCT = 4 * D + D / 2;          // bytes of 8 tokens of one head
    static constexpr int CODES = 4 * D;                // the scales follow the codes
    static constexpr int WORDS = D / 32;               // 32-bit words per lane and oct
};

#ifdef __CUDACC__

constexpr float kInt4MaxScale = 896.f;
constexpr float kInt4MinNormal = 6.103515625e-05f;     // 2^-14: below it the scales are multiples of 2^-17
constexpr uint32_t kInt4NanScale = 0xFFu;              // 0x7F80 as float16: NaN

// max that returns NaN when either operand is NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// x / y by a reciprocal of y good to an ulp or two: q = x * inv is off by a few roundings, the
// residual x - q*y is exact in one fma, and adding residual * inv gives the exact quotient wherever
// that is a float, so a quotient halfway between two codes or scales (common for float16 inputs)
// stays there.  Residual correction by fma: P. Markstein, "Computation of elementary functions on
// the IBM RISC System/6000 processor", 1990.
__device__ __forceinline__ float int4_quotient(float x, float y, float inv) {
    const float q = x * inv;
    return fmaf(fmaf(-q, y, x), inv, q);
}

// Scale byte of a group whose largest magnitude is amax: min(amax / 7, 896) rounded to nearest
// even on the byte's grid.  A NaN in the group makes the whole group NaN.
__device__ __forceinline__ uint32_t int4_scale_byte(float amax) {
    const float s = int4_quotient(fminf(amax, 7.f * kInt4MaxScale), 7.f, 1.f / 7.f);
    const uint32_t b = __float_as_uint(s);
    const uint32_t normal = ((b + 0x7FFFFu + ((b >> 20) & 1u)) >> 20) - ((127u - 15u) << 3);
    // below 2^-14, multiples of 2^-17: 1.5 * 2^23 + s * 2^17 rounds to one in its low bits
    const uint32_t small = __float_as_uint(fmaf(s, 131072.f, 12582912.f)) & 15u;
    return !(amax == amax) ? kInt4NanScale : s < kInt4MinNormal ? small : normal;
}

__device__ __forceinline__ float int4_scale_value(uint32_t byte) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 7)));
}

__device__ __forceinline__ float int4_inverse(float s) {         // 0 for a scale of 0: code 0
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(s));
    return s > 0.f ? r : 0.f;
}

// N nibbles (code + 8, in the low 4 N bits, the first lowest) of x / s rounded to nearest even, within
// -7 .. 7.  With a scale of 4 significant bits a quotient is at most 7 (1 + 2^-4), which rounds to 7;
// only a group (amax: its largest magnitude) beyond the largest scale, or below the normal ones, where
// the scale may be rounded down by more, needs the clamp.
template <int N>
__device__ __forceinline__ uint32_t int4_nibbles(float (&x)[N], float amax, float s) {
    const float inv = int4_inverse(s);
    if (!(amax >= 7.f * kInt4MinNormal && amax <= 7.f * kInt4MaxScale)) {
        if (!(amax == amax)) s = 0.f;                  // a NaN in the group: every code 0
        #pragma unroll
        for (int i = 0; i < N; ++i) x[i] = fminf(fmaxf(x[i], -7.f * s), 7.f * s);
    }
    // 1.5 * 2^23 + 8 + q rounds q to an integer (the offset is even) in its low bits; what the constant's
    // high bits add up to, modulo 2^32, is taken off once
    constexpr uint32_t kMagic = 0x4B400000u;
    uint32_t w = 0, high = 0;
    const float2 inv2 = make_float2(inv, inv), neg_s = make_float2(-s, -s), offset = make_float2(12582920.f, 12582920.f);
    #pragma unroll
    for (int i = 0; i < N; i += 2) {                   // int4_quotient of two elements at a time
        const float2 v = make_float2(x[i], x[i + 1]), q = __fmul2_rn(v, inv2);
        const float2 r = __fadd2_rn(__ffma2_rn(__ffma2_rn(q, neg_s, v), inv2, q), offset);
        w += (__float_as_uint(r.x) << (4 * i)) + (__float_as_uint(r.y) << (4 * i + 4));
        high += (kMagic << (4 * i)) + (kMagic << (4 * i + 4));
    }
    w -= high;
    return w;
}

// Expansion of the 8 nibbles of a word to four float16 pairs, exact: a nibble under the mantissa
// of 1024.0 is 1024 + u (low nibble) or 1024 + 16 u, and one fma with a16 = scale / 16 and
// c0 = -1032 a16 or c1 = -1152 a16 gives code * scale / 16 or code * scale (every product and
// sum has at most 11 significant bits: 1032 = 129 * 8 times a 4-bit scale is at most 129 * 15 < 2^11).
// p[0] holds nibbles 0 and 4, p[1] nibbles 1 and 5, p[2] nibbles 2 and 6, p[3] nibbles 3 and 7;
// p[0] and p[2] are a sixteenth of their values, which the callers make up for.
struct Int4Scale { __half2 a16, c0, c1; };

__device__ __forceinline__ Int4Scale int4_scale_pair(uint32_t half2_bits) {   // the scales as two float16
    Int4Scale r;
    r.a16 = __hmul2(*reinterpret_cast<const __half2*>(&half2_bits), __float2half2_rn(0.0625f));
    r.c0 = __hmul2(r.a16, __float2half2_rn(-1032.f));
    r.c1 = __hmul2(r.a16, __float2half2_rn(-1152.f));
    return r;
}
// one of the two scales for both halves
__device__ __forceinline__ Int4Scale int4_scale_of(const Int4Scale& s, int which) {
    Int4Scale r;
    r.a16 = which ? __high2half2(s.a16) : __low2half2(s.a16);
    r.c0 = which ? __high2half2(s.c0) : __low2half2(s.c0);
    r.c1 = which ? __high2half2(s.c1) : __low2half2(s.c1);
    return r;
}

// (w & MASK) | 0x64006400 (1024.0 twice) in one instruction, then the fma
template <uint32_t MASK>
__device__ __forceinline__ uint32_t int4_pair(uint32_t w, const __half2 a, const __half2 c) {
    uint32_t u;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(u) : "r"(w), "n"(MASK), "r"(0x64006400u));
    const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&u), a, c);
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ void int4_expand(uint32_t w, const Int4Scale& s, uint32_t (&p)[4]) {
    p[0] = int4_pair<0x000F000Fu>(w, s.a16, s.c0);
    p[1] = int4_pair<0x00F000F0u>(w, s.a16, s.c1);
    w >>= 8;
    p[2] = int4_pair<0x000F000Fu>(w, s.a16, s.c0);
    p[3] = int4_pair<0x00F000F0u>(w, s.a16, s.c1);
}

// The 8 nibbles of a word as float16 pairs times their scales, exact: p[0] holds nibbles 0 and 4 ..
// p[3] nibbles 3 and 7 (int4_expand without the sixteenth, one instruction more).
__device__ __forceinline__ void int4_expand_full(uint32_t w, uint32_t scales, uint32_t (&p)[4]) {
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

// Byte offsets inside an oct.
template <int D> __device__ __forceinline__ int int4_k_code(int token, int element) {      // of a byte of 2
    return token * (D / 2) + element / 2;
}
template <int D> __device__ __forceinline__ int int4_k_scale(int token, int element) {
    return Int4<D>::CODES + token * (D / 16) + element / 16;
}
template <int D> __device__ __forceinline__ int int4_v_piece(int token, int element) {     // of a piece of 4
    const int chunk = element / (D / 8), w = element % (D / 8) / 4;
    return (((chunk * 4 + token / 2) * (D / 32) + w) * 2 + (token & 1)) * 2;
}
template <int D> __device__ __forceinline__ int int4_v_scale(int token, int element) {
    return Int4<D>::CODES + (element / 16) * 8 + token;
}

#endif  // __CUDACC__

}  // namespace kvp
