// The paged 8-bit key/value cache: its record layout, the activation types
// its operators take and the position rotation they share.
#pragma once
#include "q8k_device.h"

namespace q8k {

// Activation types (the values of Q8K_F32, Q8K_F16, Q8K_BF16).
constexpr int DT_F32 = 0, DT_F16 = 1, DT_BF16 = 2;

constexpr float LN2 = 0.6931471805599453f;
constexpr float LOG2E = 1.4426950408889634f;

// A page holds 64 tokens.  For each page and key/value head the cache holds
// one record of 128 D + 512 bytes, contiguous and a multiple of 64 bytes:
//   keys    int8 [D/64][64 tokens][64]  planes of 64 of the head's D values
//   values  int8 [D][64 places]         token t of the page at place kv_place(t)
//   kscale  fp32 [64 tokens]            a key is its code times its scale
//   vscale  fp32 [64 tokens]
// Record (page, head) starts at byte (page * heads + head) * kv_record(D).
constexpr int KV_PAGE = 64;
__host__ __device__ constexpr int kv_record(int D) { return 2 * KV_PAGE * D + 8 * KV_PAGE; }

// The layout is the one in which the attention's matrix instructions take the
// codes, so that they go from memory into the operands without a transpose:
// - a 16x16x32 f16 MFMA whose A operand is 16 tokens' keys wants of lane
//   (row = lane % 16, g = lane / 16) eight values a step; sixteen bytes of one
//   plane at 16 g are two steps, and the 64 lanes' loads are 1 KB of
//   consecutive bytes;
// - it leaves the scores of tokens 4 g + i (i < 4) of its 16 in lane group g.
//   In the next product, values^T x probabilities^T, a lane of group g holds
//   the probabilities of 32 tokens as k = 8 g + j.  With k standing for token
//   32 u + 16 (j / 4) + 4 g + j % 4 these are the scores the lane already has,
//   and the values' A operand is eight consecutive places of a row whose
//   places are ordered by (g, u, j).
__host__ __device__ constexpr int kv_place(int t) {
    return ((t >> 2) & 3) << 4 | (t >> 5) << 3 | ((t >> 4) & 1) << 2 | (t & 3);
}

// Position rotation: rows of `dim` fp32, the cosines of dim/2 angles and then
// their sines.  The first `dim` values of a head turn in pairs; dim is a
// multiple of 8, so that a lane's eight values are four whole pairs.
struct RopeView {
    const float* table;  // nullptr: no rotation
    int len;             // positions in the table
    int dim;
    int adjacent;        // pairs (2i, 2i+1); else (i, i + dim/2)
};

// A head's D values are cut into D/8 items of two groups of four, a at oa and
// b at ob, such that an item's pairs lie inside it: (a[i], b[i]) for pairs
// half a rotation apart, neighbours for adjacent pairs and where nothing turns.
__device__ __forceinline__ void kv_item(const RopeView& r, int item, int& oa, int& ob) {
    const bool half = r.table && !r.adjacent && 8 * item < r.dim;
    oa = half ? 4 * item : 8 * item;
    ob = half ? r.dim / 2 + 4 * item : 8 * item + 4;
}

// Four values as they lie in memory, and what they stand for: apart, so that
// many loads set out before the first is waited for.
__device__ __forceinline__ uint4 load4raw(const void* p, int64_t i, bool f32) {
    if (f32) return *reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
    return make_uint4(w.x, w.y, 0, 0);
}
__device__ __forceinline__ float4 raw4f(uint4 w, int dt) {
    if (dt == DT_F32) return __builtin_bit_cast(float4, w);
    if (dt == DT_BF16)
        return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                           __uint_as_float(w.y & 0xffff0000u));
    return make_float4(half_bits_to_float(w.x & 0xffffu), half_bits_to_float(w.x >> 16),
                       half_bits_to_float(w.y & 0xffffu), half_bits_to_float(w.y >> 16));
}
__device__ __forceinline__ float4 load4f(const void* p, int64_t i, int dt) {
    return raw4f(load4raw(p, i, dt == DT_F32), dt);
}

// One rounding to the type, to nearest even.
__device__ __forceinline__ uint32_t to_bf16(float v) {
    const __bf16 h = (__bf16)v;
    return __builtin_bit_cast(uint16_t, h);
}
__device__ __forceinline__ uint32_t to_f16(float v) {
    const _Float16 h = (_Float16)v;
    return __builtin_bit_cast(uint16_t, h);
}
__device__ __forceinline__ void store4f(void* p, int64_t i, int dt, float4 v) {
    if (dt == DT_F32) {
        *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = v;
        return;
    }
    uint2 w;
    if (dt == DT_BF16) {
        w.x = to_bf16(v.x) | to_bf16(v.y) << 16;
        w.y = to_bf16(v.z) | to_bf16(v.w) << 16;
    } else {
        w.x = to_f16(v.x) | to_f16(v.y) << 16;
        w.y = to_f16(v.z) | to_f16(v.w) << 16;
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = w;
}

// The rotation of one item by its cosines and sines.  Each product and each sum is
// rounded by itself (no fused multiply-add): these values decide integer
// codes, and so they come out the same wherever they are computed that way.
__device__ __forceinline__ void kv_turn(const RopeView& r, float4 c, float4 s, float4& a, float4& b) {
#pragma clang fp contract(off)
    const float4 x = a, y = b;
    if (r.adjacent) {
        a.x = x.x * c.x - x.y * s.x;
        a.y = x.x * s.x + x.y * c.x;
        a.z = x.z * c.y - x.w * s.y;
        a.w = x.z * s.y + x.w * c.y;
        b.x = y.x * c.z - y.y * s.z;
        b.y = y.x * s.z + y.y * c.z;
        b.z = y.z * c.w - y.w * s.w;
        b.w = y.z * s.w + y.w * c.w;
    } else {
        a.x = x.x * c.x - y.x * s.x;
        a.y = x.y * c.y - y.y * s.y;
        a.z = x.z * c.z - y.z * s.z;
        a.w = x.w * c.w - y.w * s.w;
        b.x = x.x * s.x + y.x * c.x;
        b.y = x.y * s.y + y.y * c.y;
        b.z = x.z * s.z + y.z * c.z;
        b.w = x.w * s.w + y.w * c.w;
    }
}

__device__ __forceinline__ float max4(float4 v) {
    return fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
}

// Maximum over aligned groups of N lanes (8, 16 or 32), in every lane of the group,
// of magnitudes: NaN are passed over, and nothing but NaN counts as 0 (q8_K's rule).
template <int N>
__device__ __forceinline__ float group_max(float v) {
    static_assert(N == 8 || N == 16 || N == 32, "lanes of a head's row");
    v = fmaxf(v, dpp_f(v, 0));
    v = fmaxf(v, dpp_f(v, 1));
    const int x = __builtin_bit_cast(int, v);
    v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, x, 0x141, 0xF, 0xF, false)));  // row_half_mirror
    if (N >= 16) v = fmaxf(v, dpp_f(v, 3));  // row_ror:8
    if (N == 32) v = fmaxf(v, __shfl_xor(v, 16, WAVE));
    return fmaxf(v, 0.0f);
}

// Codes of four values: q8_K's rule with the row's scale (q8k_quant.h),
// round-half-even(x * (127/amax)) clamped to [-127, 127].  Adding 1.5 * 2^23
// rounds a product to a whole number, half to even, and leaves it in the low
// bits of the sum.  A finite 127/amax needs no clamp; where it overflows (amax
// zero or nearly), nonzero values saturate and zeros stay zero.  A NaN's code is 0
// (the maximum takes the place of its sum: whatever bits it came with), and so are
// all codes beside an infinity (127/amax is 0, and 0 times inf NaN).
__device__ __forceinline__ uint32_t kv_codes4(float4 v, float iscale) {
#pragma clang fp contract(off)
    const float x[4] = {v.x, v.y, v.z, v.w};
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = __builtin_bit_cast(uint32_t, fmaxf(x[e] * iscale + 12582912.0f, 0.0f));
    if (!(iscale < INFINITY))
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = x[e] > 0.0f ? 127u : x[e] < 0.0f ? 129u : 0u;
    const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x0c0c0400u), b = __builtin_amdgcn_perm(w[3], w[2], 0x0c0c0400u);
    return a | b << 16;
}

}  // namespace q8k
