// What the attention kernels share: the operands' arithmetic and the ranges
// of a sequence's rows.
#pragma once
#include "kv_cache.h"
#include "q8k_launch.h"

namespace q8k {

typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
typedef float f4_t __attribute__((ext_vector_type(4)));

constexpr float LN2 = 0.6931471805599453f;
constexpr float LOG2E = 1.4426950408889634f;

// Eight int8 codes as eight fp16 values, exactly: a code's byte with its sign
// bit flipped is code + 128, which under the exponent byte 0x64 reads
// 1024 + code + 128; subtracting 1152 leaves the code.  Five instructions for
// four codes.
__device__ __forceinline__ uint32_t f16_sub1152(uint32_t w) {
    const h2_t off = {(_Float16)1152.0f, (_Float16)1152.0f};
    const h2_t r = __builtin_bit_cast(h2_t, w) - off;
    return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ h8_t codes_f16(uint32_t lo, uint32_t hi) {
    const uint32_t a = lo ^ 0x80808080u, b = hi ^ 0x80808080u;
    uint4 w;
    w.x = f16_sub1152(__builtin_amdgcn_perm(0x64646464u, a, 0x04010400u));
    w.y = f16_sub1152(__builtin_amdgcn_perm(0x64646464u, a, 0x04030402u));
    w.z = f16_sub1152(__builtin_amdgcn_perm(0x64646464u, b, 0x04010400u));
    w.w = f16_sub1152(__builtin_amdgcn_perm(0x64646464u, b, 0x04030402u));
    return __builtin_bit_cast(h8_t, w);
}

// Two fp32 values as one or two fp16 pieces each.  One piece, rounded to
// nearest, is off by at most 2^-11 of the value; of two, the first is truncated
// (off by 2^-10) and the second is what it left, rounded: 2^-21.  Two keep fp32
// results within fp32's own error (and fp16 ones, whose own rounding is one
// piece's).  One holds a bf16 query that is not turned exactly, and
// probabilities finer than a bf16 result by three bits (lse, which is fp32 for
// every type, is summed before they are rounded).
// (The first of two comes from an instruction that the compiler takes as it
// is: a plain conversion it may do twice, once from the rounded value and once
// fused with the product that made it, and the pieces then do not fit.)
template <int NP>
__device__ __forceinline__ void f16_pieces(float x, float y, uint32_t (&w)[2]) {
    if constexpr (NP == 2) {
        const auto h = __builtin_amdgcn_cvt_pkrtz(x, y);
        const h2_t l = {(_Float16)(x - (float)h[0]), (_Float16)(y - (float)h[1])};
        w[0] = __builtin_bit_cast(uint32_t, h);
        w[1] = __builtin_bit_cast(uint32_t, l);
    } else {
        const h2_t h = {(_Float16)x, (_Float16)y};
        w[0] = __builtin_bit_cast(uint32_t, h);
        w[1] = 0;
    }
}

// Across the four 16-lane groups of a wave (lane % 16 stays).
__device__ __forceinline__ float groups_max(float v) {
    const uint32_t x = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    const uint32_t r0 = r[0], r1 = r[1];
    const float m = fmaxf(__builtin_bit_cast(float, r0), __builtin_bit_cast(float, r1));
    const uint32_t y = __builtin_bit_cast(uint32_t, m);
    const auto t = __builtin_amdgcn_permlane16_swap(y, y, false, false);
    const uint32_t t0 = t[0], t1 = t[1];
    return fmaxf(__builtin_bit_cast(float, t0), __builtin_bit_cast(float, t1));
}
__device__ __forceinline__ float groups_sum(float v) {
    const uint32_t x = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    const uint32_t r0 = r[0], r1 = r[1];
    const float m = __builtin_bit_cast(float, r0) + __builtin_bit_cast(float, r1);
    const uint32_t y = __builtin_bit_cast(uint32_t, m);
    const auto t = __builtin_amdgcn_permlane16_swap(y, y, false, false);
    const uint32_t t0 = t[0], t1 = t[1];
    return __builtin_bit_cast(float, t0) + __builtin_bit_cast(float, t1);
}

// A power of two as a float, |e| <= 126.
__device__ __forceinline__ float pow2f(int e) { return __builtin_bit_cast(float, (uint32_t)(127 + e) << 23); }

// The exponent e with 2^e <= v < 2^(e+1) of a positive value, kept to
// [-100, 120] (zero, subnormal, infinite and NaN values included).
__device__ __forceinline__ int exponent_of(float v) {
    const int e = (int)((__builtin_bit_cast(uint32_t, v) >> 23) & 255u) - 127;
    return e < -100 ? -100 : e > 120 ? 120 : e;
}

// A sequence's new tokens and length, with what the device-side values say
// cut to what the call's sizes allow, so that no access leaves its buffer.
struct Sequence {
    int q0, n, nq, len;  // n new tokens from row q0 on, the first nq of them served
};
__device__ __forceinline__ Sequence sequence_of(const Attend& a, int64_t b) {
    Sequence s;
    int64_t q0 = a.cu_q[b], q1 = a.cu_q[b + 1];
    q0 = q0 < 0 ? 0 : q0 > a.Tq ? a.Tq : q0;
    q1 = q1 < q0 ? q0 : q1 > a.Tq ? a.Tq : q1;
    s.q0 = (int)q0;
    s.n = (int)(q1 - q0);
    s.nq = (int)(s.n > a.max_q ? a.max_q : s.n);
    const int64_t len = a.kv_len[b];
    s.len = (int)(len < 0 ? 0 : len > a.max_len ? a.max_len : len);
    return s;
}
// Tokens [first, last] that new token i of the sequence sees (none if last < first).
struct Span {
    int first, last;
};
__device__ __forceinline__ Span span_of(const Attend& a, const Sequence& s, int i) {
    Span p;
    p.last = s.len - s.n + i;
    const int64_t f = (int64_t)p.last - a.window + 1;
    p.first = a.window > 0 && f > 0 ? (int)f : 0;
    return p;
}

// One item (eight values) of query row `row`, turned.  The scale's sign goes
// with the query (and a scale of zero makes it zero), its magnitude comes in
// behind the products: score_unit.  A row whose position lies outside the
// table is NaN.
template <int D>
__device__ __forceinline__ void load_q_item(const Attend& a, const Sequence& s, int h, int row, int item, float* dst) {
    const int tok = row / a.group, t = s.q0 + tok;
    const int64_t base = (int64_t)t * a.q_stride + (int64_t)(h * a.group + row % a.group) * D;
    int oa, ob;
    kv_item(a.rope, item, oa, ob);
    float4 x = load4f(a.q, base + oa, a.dtype), y = load4f(a.q, base + ob, a.dtype);
    float f = a.scale > 0.0f ? 1.0f : a.scale < 0.0f ? -1.0f : 0.0f;
    if (a.rope.table) {
        const int p = a.pos[t];
        if (p >= 0 && p < a.rope.len)
            kv_turn(a.rope, a.rope.table + (int64_t)p * a.rope.dim, item, x, y);
        else
            f = __builtin_nanf("");
    }
    *reinterpret_cast<float4*>(dst + oa) = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
    *reinterpret_cast<float4*>(dst + ob) = make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
}

// What a product of codes with a query that was multiplied by 2^e counts in
// the exponent of 2: never zero, so that -inf stays -inf.
__device__ __forceinline__ float score_unit(const Attend& a, int e) {
    const float s = fabsf(a.scale);
    return fmaxf((s > 0.0f ? s * LOG2E : 1.0f) * pow2f(-e), 1.17549435e-38f);
}

__device__ __forceinline__ int64_t q_row_of(const Attend& a, const Sequence& s, int h, int row) {
    return (int64_t)(s.q0 + row / a.group) * a.q_heads + h * a.group + row % a.group;
}

}  // namespace q8k
