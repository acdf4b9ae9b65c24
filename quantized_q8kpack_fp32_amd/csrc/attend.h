// What the attention kernels share: the operands' arithmetic and the ranges
// of a sequence's rows.
#pragma once
#include "kv_cache.h"
#include "q8k_launch.h"

namespace q8k {

typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
typedef float f4_t __attribute__((ext_vector_type(4)));

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

// Maximum over the wave, in every lane, without LDS.
__device__ __forceinline__ float wave_max_dpp(float v) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v = fmaxf(v, dpp_f(v, k));
    return groups_max(v);
}

// A power of two as a float, |e| <= 126.
__device__ __forceinline__ float pow2f(int e) { return __builtin_bit_cast(float, (uint32_t)(127 + e) << 23); }

// The exponent e with 2^e <= v < 2^(e+1) of a positive value, kept to
// [-100, 120] (zero, subnormal, infinite and NaN values included).
__device__ __forceinline__ int exponent_of(float v) {
    const int e = (int)((__builtin_bit_cast(uint32_t, v) >> 23) & 255u) - 127;
    return e < -100 ? -100 : e > 120 ? 120 : e;
}

// A value that is the same in every lane, as a scalar.
__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ float uni_f(float v) { return __builtin_bit_cast(float, uni(__builtin_bit_cast(int, v))); }

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

// ---- the work items
// A sequence's rows of one key head make tiles of a.tile_rows rows.  A tile's
// pages are cut into chunks of c pages from the tile's first page on; an item
// is one tile and one chunk.  c goes by the lengths on the device, not by the
// limits the host knows (a captured step may have been captured for lengths
// far above today's): what makes about a.target items a head, of equal size
// whatever mix of lengths there is, and then for each sequence what cuts its
// pages evenly.  Items are numbered sequence by
// sequence; every workgroup finds its own by adding up the sequences before it,
// 64 at a time.  target == 0: one item a tile (there are enough of them).
struct Item {
    int64_t b, first;  // sequence; its first item's number
    int c, splits;     // pages a chunk; chunks a tile
    int tile, split;
    Sequence seq;
};
// A sequence's chunks: as many as come nearest to c pages each.
__device__ __forceinline__ int splits_of(int pages, int c) { return max(1, (pages + c / 2) / c); }
__device__ __forceinline__ int chunk_pages(int pages, int splits) { return splits == 1 ? 1 << 30 : (pages + splits - 1) / splits; }
struct Load {
    Sequence seq;
    int tiles, pages;  // tiles, and pages a tile reads at most
};
__device__ __forceinline__ Load load_of(const Attend& a, int64_t b) {
    Load l;
    l.seq = sequence_of(a, b);
    l.tiles = (l.seq.nq * a.group + a.tile_rows - 1) / a.tile_rows;
    const int first = span_of(a, l.seq, 0).first / KV_PAGE;
    const int last = span_of(a, l.seq, l.seq.nq - 1).last;
    l.pages = last < 0 ? 0 : last / KV_PAGE + 1 - first;
    if (a.window > 0 && l.tiles > 1) {
        // a tile's rows see the window and its own tokens, from anywhere in a page
        const int64_t t = (a.window + a.tile_rows / a.group + 2 + KV_PAGE - 2) / KV_PAGE + 1;
        if (t < l.pages) l.pages = (int)t;
    }
    return l;
}
// Sum of the lanes up to this one, without LDS: rows of 16 lanes, then the
// last lane of each row to the rows behind it.
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);  // row_shr:2
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);  // row_shr:4
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);  // row_shr:8
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31
    return v;
}
__device__ __forceinline__ int wave_total(int v) { return __builtin_amdgcn_readlane(wave_scan(v), 63); }
// The sequence of this lane among 64 from b0 on.
__device__ __forceinline__ Load lane_load(const Attend& a, int64_t b0) {
    const int64_t b = b0 + (threadIdx.x & 63);
    return b < a.B ? load_of(a, b) : Load{Sequence{0, 0, 0, 0}, 0, 0};
}
__device__ __forceinline__ Sequence sequence_of_lane(const Sequence& s, int lane) {
    return Sequence{__builtin_amdgcn_readlane(s.q0, lane), __builtin_amdgcn_readlane(s.n, lane),
                    __builtin_amdgcn_readlane(s.nq, lane), __builtin_amdgcn_readlane(s.len, lane)};
}

// Pages a chunk (called by whole waves; l0: lane_load(a, 0)).
__device__ __forceinline__ int chunk_of(const Attend& a, const Load& l0) {
    int64_t total = 0;
    for (int64_t b0 = 0; b0 < a.B; b0 += 64) {
        const Load l = b0 == 0 ? l0 : lane_load(a, b0);
        const int64_t n = (int64_t)l.tiles * l.pages;  // summed in two parts of 32 bits
        total += ((int64_t)wave_total((int)(n >> 20)) << 20) + wave_total((int)(n & 0xfffff));
    }
    const int64_t c = (total + a.target - 1) / a.target;
    return (int)(c < a.least ? a.least : c);
}
// Item `w` of a head; false: there is none of that number.
__device__ __forceinline__ bool item_of(const Attend& a, int64_t w, Item& it) {
    const int lane = threadIdx.x & 63;
    if (a.target == 0) {
        // whole tiles: of the longest sequence first (where the plan says so), and of
        // its last tokens, which see the most
        const int64_t b = w / a.tiles_max;
        it = Item{b, 0, 1 << 30, 1, a.tiles_max - 1 - (int)(w % a.tiles_max), 0, {}};
        if (b >= a.B) return false;
        if (a.order) {
            const Load l = lane_load(a, 0);
            int rank = 0;
            for (int j = 0; j < (int)a.B; ++j) {
                const int other = __builtin_amdgcn_readlane(l.pages, j);
                rank += other > l.pages || (other == l.pages && j < lane) ? 1 : 0;
            }
            const int at = __builtin_ctzll(__ballot(lane < (int)a.B && rank == (int)b));
            it.b = at;
            it.seq = sequence_of_lane(l.seq, at);
        } else {
            it.seq = sequence_of_lane(sequence_of(a, b), 0);
        }
        return true;
    }
    Load l = lane_load(a, 0);
    const int c = chunk_of(a, l);
    int64_t before = 0;
    for (int64_t b0 = 0; b0 < a.B; b0 += 64) {
        if (b0 > 0) l = lane_load(a, b0);
        const int splits = splits_of(l.pages, c), n = l.tiles * splits, upto = wave_scan(n);
        const uint64_t hit = __ballot(w < before + upto);
        if (hit) {
            const int at = __builtin_ctzll(hit);
            const int rest = (int)(w - before) - __builtin_amdgcn_readlane(upto - n, at);
            it.b = b0 + at;
            it.first = w - rest;
            it.splits = __builtin_amdgcn_readlane(splits, at);
            it.c = chunk_pages(__builtin_amdgcn_readlane(l.pages, at), it.splits);
            it.tile = rest / it.splits;
            it.split = rest % it.splits;
            it.seq = sequence_of_lane(l.seq, at);
            return true;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}
// First item and chunking of sequence b.
__device__ __forceinline__ Item items_of(const Attend& a, int64_t b) {
    Load l = lane_load(a, 0);
    Item it{b, 0, 0, 1, 0, 0, {}};
    const int c = chunk_of(a, l);
    for (int64_t b0 = 0; b0 <= b; b0 += 64) {
        if (b0 > 0) l = lane_load(a, b0);
        const int splits = splits_of(l.pages, c), n = l.tiles * splits, upto = wave_scan(n);
        if (b < b0 + 64) {
            const int at = uni((int)(b - b0));
            it.first += __builtin_amdgcn_readlane(upto - n, at);
            it.splits = __builtin_amdgcn_readlane(splits, at);
            it.c = chunk_pages(__builtin_amdgcn_readlane(l.pages, at), it.splits);
            it.seq = sequence_of_lane(l.seq, at);
        } else {
            it.first += __builtin_amdgcn_readlane(upto, 63);
        }
    }
    return it;
}

// A tile's rows and pages.
struct Tile {
    int row0, rows;    // its first row; rows of the sequence and head
    int tok0, head0;   // the first row's token and query head (of the key head's)
    Span lo, hi;       // of its first and last row
    int p0, p1;        // its pages
};
// Row r of a tile: its token and query head.  The division by the group is of a
// number below 2^13 (at most 4095 + 127): half added, the product with the
// rounded reciprocal is off by less than the half is from the next whole number.
struct TileRow {
    int tok, head;
};
__device__ __forceinline__ TileRow row_of_tile(const Attend& a, const Tile& t, int r) {
    const int x = t.head0 + r, q = (int)(((float)x + 0.5f) * a.inv_group);
    return TileRow{t.tok0 + q, x - q * a.group};
}
// An item's tile, its numbers as scalars (as its sequence's are): the page
// loop's addresses and branches then cost no vector instructions.
__device__ __forceinline__ Tile item_tile(const Attend& a, const Sequence& s, int tile) {
    Tile t;
    t.rows = uni(s.nq * a.group);
    t.row0 = uni(tile * a.tile_rows);
    t.tok0 = uni(t.row0 / a.group);
    t.head0 = uni(t.row0 - t.tok0 * a.group);
    const int last = min(t.rows, t.row0 + a.tile_rows) - 1;
    const Span lo = span_of(a, s, t.tok0), hi = span_of(a, s, row_of_tile(a, t, max(last - t.row0, 0)).tok);
    t.lo = Span{uni(lo.first), uni(lo.last)};
    t.hi = Span{uni(hi.first), uni(hi.last)};
    t.p0 = t.lo.first / KV_PAGE;
    t.p1 = t.hi.last >= 0 ? t.hi.last / KV_PAGE + 1 : 0;
    return t;
}

// ---- queries
// One item (eight values) of a query row on its way from memory.  The scale's
// sign goes with the query (and a scale of zero makes it zero), its magnitude
// comes in behind the products: score_unit.  A row whose position lies outside
// the table is NaN.
struct QueryItem {
    uint4 x, y;  // as they lie in memory
    float4 c, s;
    int oa, ob, p;
};
template <int D>
__device__ __forceinline__ void fetch_q(const Attend& a, const Sequence& s, int h, TileRow r, int item, QueryItem& q) {
    const int64_t t = s.q0 + r.tok;
    const int64_t base = t * a.q_stride + (int64_t)(h * a.group + r.head) * D;
    kv_item(a.rope, item, q.oa, q.ob);
    q.p = a.rope.table ? a.pos[t] : 0;
    q.x = load4raw(a.q, base + q.oa, a.dtype == DT_F32);
    q.y = load4raw(a.q, base + q.ob, a.dtype == DT_F32);
}
__device__ __forceinline__ void fetch_turn(const Attend& a, int item, QueryItem& q) {
    if (a.rope.table && 8 * item < a.rope.dim && q.p >= 0 && q.p < a.rope.len) {
        const float* row = a.rope.table + (int64_t)q.p * a.rope.dim + 4 * item;
        q.c = *reinterpret_cast<const float4*>(row);
        q.s = *reinterpret_cast<const float4*>(row + a.rope.dim / 2);
    }
}
__device__ __forceinline__ void put_q(const Attend& a, int item, const QueryItem& q, float* dst) {
    float4 x = raw4f(q.x, a.dtype), y = raw4f(q.y, a.dtype);
    float f = a.scale > 0.0f ? 1.0f : a.scale < 0.0f ? -1.0f : 0.0f;
    if (a.rope.table) {
        if (q.p >= 0 && q.p < a.rope.len) {
            if (8 * item < a.rope.dim) kv_turn(a.rope, q.c, q.s, x, y);
        } else {
            f = __builtin_nanf("");
        }
    }
    *reinterpret_cast<float4*>(dst + q.oa) = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
    *reinterpret_cast<float4*>(dst + q.ob) = make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
}

// What a product of codes with a query that was multiplied by 2^e counts in
// the exponent of 2: never zero, so that -inf stays -inf.
__device__ __forceinline__ float score_unit(const Attend& a, int e) {
    const float s = fabsf(a.scale);
    return fmaxf((s > 0.0f ? s * LOG2E : 1.0f) * pow2f(-e), 1.17549435e-38f);
}

// A running maximum m so far from zero that its steps are a half and more: the
// fused t unit - m, exact before its one rounding, would then be off zero at the
// maximum itself by as much, and its power of two by that factor.  Such a row's
// products are rounded first, as the maximum was, and their distances from it
// taken for the scores, in the same unit.
__device__ __forceinline__ bool is_far(float m) { return fabsf(m) >= 8388608.0f && m > -INFINITY; }
__device__ __forceinline__ float far_score(float t, float unit, float inv_unit, float m) {
#pragma clang fp contract(off)
    return (t * unit - m) * inv_unit;
}

// The operand of a query row from LDS, in pieces times 2^(12 - e), e the
// exponent of the row's largest magnitude; returns the row's score_unit.  Step
// 2 s + t of lane group g holds values 64 s + 16 g + 8 t + j.
template <int D, int NQ>
__device__ __forceinline__ float query_operand(const Attend& a, const float* row, int g, h8_t (&qf)[NQ][D / 32]) {
    float amax = 0.0f;
#pragma unroll
    for (int s = 0; s < D / 64; ++s)
#pragma unroll
        for (int c = 0; c < 4; ++c) amax = fmaxf(amax, max4(*reinterpret_cast<const float4*>(row + 64 * s + 16 * g + 4 * c)));
    amax = groups_max(amax);
    const int qe = 12 - exponent_of(amax);
    const float up = pow2f(qe);
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
        uint32_t w[4][2];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float2 v = *reinterpret_cast<const float2*>(row + 64 * (s / 2) + 16 * g + 8 * (s & 1) + 2 * c);
            f16_pieces<NQ>(v.x * up, v.y * up, w[c]);
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n)
            qf[n][s] = __builtin_bit_cast(h8_t, make_uint4(w[0][n], w[1][n], w[2][n], w[3][n]));
    }
    return score_unit(a, qe);
}

// A row's place in the results.
__device__ __forceinline__ int64_t q_row_of(const Attend& a, const Sequence& s, int h, TileRow r) {
    return (int64_t)(s.q0 + r.tok) * a.q_heads + h * a.group + r.head;
}

}  // namespace q8k
