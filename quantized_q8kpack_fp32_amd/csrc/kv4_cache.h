// The paged 4-bit key/value cache: its record layout, its quantiser and the
// widening of its codes.
#pragma once
#include "kv_cache.h"

namespace q8k {

// A head's D values are cut into groups of 32.  A value is (code * factor) *
// scale: code in [-7, 7], held as code + 8 in four bits; factor the group's, an
// 8-bit float of four exponent and four mantissa bits, those of the fp16 whose
// bits are factor << 6 (0 to 1, steps of 2^-18 below 2^-14); scale the row's, fp32.
// code * factor has at most eight significant bits: fp16 holds it exactly, and so the
// matrix instructions take it.
//
// A page's record for one head is 68 D + 512 bytes, a multiple of 64:
//   key codes      [D/32] blocks of 1 KB   pieces of 16 values of 16 tokens, below
//   value codes    [D/32][16][64 places]   values 32 e + c (low half) and 32 e + 16 + c of the token
//                                          at place kv4_place(t)
//   key factors    [16][2][D/16]           of token 16 q + c and group 2 s + y at [c][y][q D/64 + s]
//   value factors  [D/32][64 places]
//   key scales     fp32 [64 tokens]
//   value scales   fp32 [64 tokens]
// Every byte is one token's, so an append touches no other token's.
//
// Keys: lane (c = lane % 16, g = lane / 16) of the product's A operand wants of
// token 16 q + c the values 64 s + 16 g .. + 15 (kv_cache.h): eight bytes, piece
// q D/64 + s.  Two pieces lie side by side, so that a lane loads 16 bytes and a wave 1
// KB of consecutive ones: piece p of lane (c, g) is at (p/2) 1024 + 64 c + 16 g + 8 (p%2).
// It is two words of eight values; value j of a word is at the bits from
// 4 (j/2 + 4 (j%2)) + 2 on, round the word's end: so masks bring pairs (j, j + 1) under
// the halves' exponents, for every other pair after one rotation.
// Values: of a word of four places j = 0, 2, 1, 3 of a group of four tokens, masks bring
// the pairs (0, 1) and (2, 3) of both values in the same way.
__host__ __device__ constexpr int kv4_record(int D) { return 68 * D + 8 * KV_PAGE; }
__host__ __device__ constexpr int kv4_place(int t) {
    return ((t >> 2) & 3) << 4 | (t >> 5) << 3 | ((t >> 4) & 1) << 2 | (t & 1) << 1 | ((t >> 1) & 1);
}
constexpr int KV4_V(int D) { return 32 * D; }
constexpr int KV4_KF(int D) { return 64 * D; }
constexpr int KV4_VF(int D) { return 66 * D; }
constexpr int KV4_S(int D) { return 68 * D; }

__host__ __device__ constexpr int kv_record_of(int bits, int D) { return bits == 8 ? kv_record(D) : kv4_record(D); }

// Where the eight key values 8 i .. 8 i + 7 of a token lie (a word).
template <int D>
__device__ __forceinline__ int kv4_key_word(int token, int i) {
    const int s = i >> 3, g = (i >> 1) & 3, p = (token >> 4) * (D / 64) + s;
    return (p >> 1) * 1024 + (token & 15) * 64 + g * 16 + (p & 1) * 8 + (i & 1) * 4;
}
// The factor of group y of a token's key.
template <int D>
__device__ __forceinline__ int kv4_key_factor(int token, int y) {
    return KV4_KF(D) + ((token & 15) * 2 + (y & 1)) * (D / 16) + (token >> 4) * (D / 64) + (y >> 1);
}

// ---- quantiser.  Every step is one rounding in fp32, so that codes come out the same
// wherever they are computed that way.
// The least factor that is not below r in [0, 1] (0 for NaN): above 2^-14 the top bits of
// r, rounded up; below, r in steps of 2^-18.
__device__ __forceinline__ uint32_t kv4_factor(float r) {
    r = fmaxf(r, 0.0f);
    const uint32_t small = (uint32_t)(int)ceilf(r * 262144.0f);
    return r < 6.103515625e-05f ? small : ((__builtin_bit_cast(uint32_t, r) + 0x7ffffu) >> 19) - (112u << 4);
}
__device__ __forceinline__ float kv4_factor_value(uint32_t f) { return half_bits_to_float(f << 6); }
// 1 / step of a group, or 0 where all codes are 0 (nothing but zeros, or too small beside
// the row's largest for any factor; an infinity among the row's values).
__device__ __forceinline__ float kv4_inverse(uint32_t f, float scale) {
#pragma clang fp contract(off)
    // (a step, not a quotient, is chosen: a division is too much for the compiler to take both ways)
    return 1.0f / (f == 0 || !(scale < INFINITY) ? INFINITY : kv4_factor_value(f) * scale);
}
// code + 8 of eight finite values (a and b: 0-3 and 4-7), value i's at bit S_i: kv_codes4's
// rule with 7 in the place of 127.  1.5 * 2^23 + 8 rounds a product to a whole number,
// half to even, and leaves code + 8 in the low bits of the sum, above constant ones, which
// come off all at once.
constexpr float KV4_ROUND = 12582920.0f;
template <int S0, int S1, int S2, int S3, int S4, int S5, int S6, int S7>
__device__ __forceinline__ uint64_t kv4_codes8(float4 a, float4 b, float inverse) {
#pragma clang fp contract(off)
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    constexpr int at[8] = {S0, S1, S2, S3, S4, S5, S6, S7};
    constexpr uint32_t top = 0x4b400000u;
    uint32_t w[2] = {0, 0}, off[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        w[at[i] / 32] += __builtin_bit_cast(uint32_t, v[i] * inverse + KV4_ROUND) << (at[i] % 32);
        off[at[i] / 32] += top << (at[i] % 32);
    }
    w[0] -= off[0];
    w[1] -= off[1];
    if (!(inverse < INFINITY)) {
        w[0] = w[1] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) w[at[i] / 32] |= (v[i] > 0.0f ? 15u : v[i] < 0.0f ? 1u : 8u) << (at[i] % 32);
    }
    return (uint64_t)w[1] << 32 | w[0];
}
// The word of eight values of a key.
__device__ __forceinline__ uint32_t kv4_key_codes(float4 x, float4 y, float inverse) {
    const uint32_t w = (uint32_t)kv4_codes8<0, 16, 4, 20, 8, 24, 12, 28>(x, y, inverse);
    return w << 2 | w >> 30;
}
// The codes (as numbers) of a key's word.
__device__ __forceinline__ void kv4_key_values(uint32_t word, float4& x, float4& y) {
    const uint32_t w = word >> 2 | word << 30;
    const auto c = [w](int at) { return (float)((int)(w >> at & 15u) - 8); };
    x = make_float4(c(0), c(16), c(4), c(20));
    y = make_float4(c(8), c(24), c(12), c(28));
}

// N consecutive words of a record.
template <int N>
__device__ __forceinline__ void load_words(rsrc_t rec, int off, uint32_t (&w)[N]) {
    static_assert(N == 1 || N == 2 || N == 4, "words of one load");
    if constexpr (N == 1) {
        w[0] = load4(rec, off);
    } else if constexpr (N == 2) {
        const uint2 v = load8(rec, off);
        w[0] = v.x, w[1] = v.y;
    } else {
        const uint4 v = load16(rec, off);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
}

// ---- widening.  Four bits at the bits from 2 (or 6) on of a half whose exponent is
// 256's (or 16's) read 256 + u (16 + u), u = code + 8; times the factor, less 264 (24)
// times the factor, is code * factor, rounded once and nowhere: 264 = 33 * 8 and a
// factor has five bits.
typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
struct Factors {  // of the two values of a pair, and what comes off
    h2_t f, low, high;
};
__device__ __forceinline__ Factors kv4_factors(uint32_t two) {
    Factors r;
    r.f = __builtin_bit_cast(h2_t, two);
    r.low = r.f * (_Float16)-264.0f;
    r.high = r.f * (_Float16)-24.0f;
    return r;
}
// The masks and exponents from registers: a mask and an exponent then take one
// instruction, with literals two (no instruction takes two of them).
struct Widen {
    uint32_t low_mask = 0x003c003cu, low = 0x5c005c00u, high_mask = 0x03c003c0u, high = 0x4c004c00u;
    __device__ __forceinline__ Widen() {
        asm("" : "+s"(low_mask), "+s"(high_mask));
        asm("" : "+v"(low), "+v"(high));
    }
};
__device__ __forceinline__ uint32_t kv4_low(const Widen& m, uint32_t w, const Factors& f) {
    const h2_t a = __builtin_bit_cast(h2_t, (w & m.low_mask) | m.low);
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(a, f.f, f.low));
}
__device__ __forceinline__ uint32_t kv4_high(const Widen& m, uint32_t w, const Factors& f) {
    const h2_t a = __builtin_bit_cast(h2_t, (w & m.high_mask) | m.high);
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(a, f.f, f.high));
}
// A key's word: eight values of one group.  `factor`: the factor's byte.
__device__ __forceinline__ Factors kv4_key_factors(uint32_t factor) { return kv4_factors(factor * 0x00400040u); }
__device__ __forceinline__ h8_t kv4_widen_keys(const Widen& m, uint32_t w, const Factors& f) {
    const uint32_t r = __builtin_amdgcn_alignbit(w, w, 8);
    return __builtin_bit_cast(h8_t, make_uint4(kv4_low(m, w, f), kv4_high(m, w, f), kv4_low(m, r, f), kv4_high(m, r, f)));
}
// A word of the values' factors (four tokens): those of its pairs (0, 1) and (2, 3).
struct FactorPairs {
    Factors first, second;
};
__device__ __forceinline__ FactorPairs kv4_value_factors(uint32_t f) {
    return {kv4_factors((f << 6) & 0x3fc03fc0u), kv4_factors((f >> 2) & 0x3fc03fc0u)};
}
// Two words of values (eight tokens) and their factors: the operands of values c and
// 16 + c of a group.
__device__ __forceinline__ void kv4_widen_values(const Widen& m, uint32_t w0, uint32_t w1, const FactorPairs& f0,
                                                 const FactorPairs& f1, h8_t& a, h8_t& b) {
    uint32_t x[4], y[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t w = i ? w1 : w0;
        const Factors &p = i ? f1.first : f0.first, &q = i ? f1.second : f0.second;
        x[2 * i] = kv4_low(m, w << 2, p);
        y[2 * i] = kv4_high(m, w << 2, p);
        x[2 * i + 1] = kv4_low(m, w >> 6, q);
        y[2 * i + 1] = kv4_high(m, w >> 6, q);
    }
    a = __builtin_bit_cast(h8_t, make_uint4(x[0], x[1], x[2], x[3]));
    b = __builtin_bit_cast(h8_t, make_uint4(y[0], y[1], y[2], y[3]));
}

}  // namespace q8k
