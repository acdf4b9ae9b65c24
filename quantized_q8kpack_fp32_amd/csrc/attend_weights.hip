// What each cached token gets of the new tokens' attention, per key head:
//   w_j = keep old_j + sum over rows r that see j of e^(s_rj - lse_r),  s_rj = scale <q_r, key_j>,
// rows being the key head's query heads times the new tokens, lse their log sums
// as attention left them.  With lse known no row needs its other tokens, so the
// sum over rows stays where the tokens are: a wave holds the keys of one page, widened
// once, and adds up its 64 tokens while the rows go by.  No atomics: one order always.
//
// Few rows are bound by the keys' bytes: 16 sequences of up to 8191 tokens, 32 heads of
// 128 over 8, 8 bits, 20 us, 4.4 TB/s, 4 bits 17.5 us.  Many are bound by matrix instructions
// and the exponentials, which hardly overlap: 2 x 1000 tokens over 8001, 32 heads over 4, 4
// bits, bf16 and turned, 225 us, 205 of them the products: 600 TFLOP/s of the formula's, 1200
// with the queries' two pieces.  A window takes no page's reading off: its unseen tokens are
// masked (a window of 1000 over 2 x 65537, 4 bits, 22 us, as without one).
#include <type_traits>

#include "attend.h"

namespace q8k {

namespace {

constexpr int WAVES = 4, ROWS = 16;
// A share of the rows has so many tiles at least.  It is right where the workgroups without
// shares fill the device (the last 64 tokens of 4 x up to 16001, 32 heads over 8, 632
// workgroups: 43 us, by 8 52, by 4 47).  Where they are fewer it leaves compute units idle,
// and smaller shares, which are not made, would be faster (64 tokens of one sequence over
// 1000, 16 workgroups: 32 us, by 8 25, by 4 20, by 2 18; over 4000, 64: 29, 24, 20, 22; of
// heads of 64 23, 20, 17, 17, of 256 32, 26, 25, 28; over 16001, 256: 31, 29, 32, 43; 300
// over 500 with one key head 38, 29, 27, 32, with eight 40, 30, 26, 29).
constexpr int LEAST_TILES = 16;

// A page's keys of one head: on their way, and as the product's operand.
template <int D, int BITS>
struct PageKeys {
    uint4 raw[BITS == 8 ? D / 16 : D / 32];
    uint32_t fac[D / 64];
    float scale;  // of token `lane`
    __device__ __forceinline__ void fetch(rsrc_t rec, int lane) {
        const int col = lane & 15, g = lane >> 4, off = col * 64 + g * 16;
#pragma unroll
        for (int i = 0; i < (BITS == 8 ? D / 16 : D / 32); ++i) raw[i] = load16_nt(rec, off + i * 1024);
        if constexpr (BITS == 4) load_words<D / 64>(rec, KV4_KF(D) + (col * 2 + (g >> 1)) * (D / 16), fac);
        scale = __builtin_bit_cast(float, load4(rec, kv_record_of(BITS, D) - 8 * KV_PAGE + 4 * lane));
    }
    // of 16 tokens 16 q and on, steps 2 s and 2 s + 1
    __device__ __forceinline__ void widen(const Widen& masks, int q, int s, h8_t& a, h8_t& b) const {
        if constexpr (BITS == 8) {
            const uint4 c = raw[4 * s + q];
            a = codes_f16(c.x, c.y);
            b = codes_f16(c.z, c.w);
        } else {
            const int p = q * (D / 64) + s;
            const uint4 c = raw[p >> 1];
            const Factors f = kv4_key_factors(fac[p >> 2] >> (8 * (p & 3)) & 255u);
            a = kv4_widen_keys(masks, p & 1 ? c.z : c.x, f);
            b = kv4_widen_keys(masks, p & 1 ? c.w : c.y, f);
        }
    }
};

// A row: the unit of its products, log2 of its sum (inf where it sees nothing), and
// the tokens that it sees.
struct RowInfo {
    float unit, lse;
    int first, last;
};

// Row `col` of a tile.
__device__ __forceinline__ RowInfo info_of(const AttendWeights& w, const Sequence& seq, const Tile& tile, int h, int col) {
    RowInfo o{1.0f, INFINITY, 0, -1};
    if (tile.row0 + col < tile.rows) {
        const TileRow tr = row_of_tile(w.a, tile, col);
        const Span sp = span_of(w.a, seq, tr.tok);
        const float lse = w.lse[q_row_of(w.a, seq, h, tr)];
        // (a row of -inf sees nothing: what it would meet may be NaN)
        if (lse != -INFINITY) o = RowInfo{1.0f, lse * LOG2E, sp.first, sp.last};
    }
    return o;
}

// Sixteen rows of a head as the product's operand, by way of LDS, and their RowInfo.
template <int D, int NQ>
__device__ __forceinline__ RowInfo stage_rows(const AttendWeights& w, const Sequence& seq, int h, int t, int lane,
                                              float (*q_s)[D + 4], h8_t (&qf)[NQ][D / 32]) {
    const Attend& a = w.a;
    const int col = lane & 15, g = lane >> 4, rows = seq.nq * a.group;
    const Tile tile = item_tile(a, seq, t);
    QueryItem qi[D / 32];
#pragma unroll
    for (int n = 0; n < D / 32; ++n) {
        const int i = lane + 64 * n;
        fetch_q<D>(a, seq, h, row_of_tile(a, tile, min(i / (D / 8), rows - 1 - tile.row0)), i % (D / 8), qi[n]);
    }
    RowInfo o = info_of(w, seq, tile, h, col);
#pragma unroll
    for (int n = 0; n < D / 32; ++n) fetch_turn(a, (lane + 64 * n) % (D / 8), qi[n]);
#pragma unroll
    for (int n = 0; n < D / 32; ++n) {
        const int i = lane + 64 * n;
        put_q(a, i % (D / 8), qi[n], q_s[i / (D / 8)]);
    }
    __builtin_amdgcn_wave_barrier();
    o.unit = query_operand<D, NQ>(a, q_s[col], g, qf);
    __builtin_amdgcn_wave_barrier();
    return o;
}

// What 16 rows add to a page's tokens: lane (col, g) holds row col's part of tokens
// 16 q + 4 g + e.
__device__ __forceinline__ void add_row(const f4_t (&s4)[4], const float* scales, const RowInfo& row, int j0, int g,
                                        float (&sum)[4][4]) {
    float t[4][4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const f4_t ks = *reinterpret_cast<const f4_t*>(scales + 16 * q + 4 * g);
#pragma unroll
        for (int e = 0; e < 4; ++e) t[q][e] = __builtin_fmaf(s4[q][e] * ks[e], row.unit, -row.lse);
    }
    if (__any(row.first > j0 || row.last < j0 + KV_PAGE - 1)) {
        // pages that some row sees only in part (what lies in unseen places may be anything)
        const uint32_t from = j0 + 4 * g - row.first, most = row.last - row.first;
        const bool none = row.last < row.first;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) t[q][e] = !none && from + (16 * q + e) <= most ? t[q][e] : -INFINITY;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[q][e] += __builtin_amdgcn_exp2f(t[q][e]);
}
// Over the sixteen lanes of a row, halving what a lane holds at each step: lane (col, g)
// is left with token 16 q + 4 g + e, q = 2 (col / 4 % 2) + col / 8, e = col % 4.
__device__ __forceinline__ float rows_sum(const float (&sum)[4][4], int col) {
    const auto swap = [](float v, auto ctrl) {
        return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctrl)::value, 0xF, 0xF, false));
    };
    const bool b2 = col & 4, b3 = col & 8, b1 = col & 2, b0 = col & 1;
    float x[2][4], y[4], z[2];
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            x[q][e] = (b2 ? sum[q + 2][e] : sum[q][e]) +
                      swap(b2 ? sum[q][e] : sum[q + 2][e], std::integral_constant<int, 0x141>{});  // row_half_mirror
#pragma unroll
    for (int e = 0; e < 4; ++e)
        y[e] = (b3 ? x[1][e] : x[0][e]) + swap(b3 ? x[0][e] : x[1][e], std::integral_constant<int, 0x128>{});  // row_ror:8
#pragma unroll
    for (int e = 0; e < 2; ++e)
        z[e] = (b1 ? y[e + 2] : y[e]) + swap(b1 ? y[e] : y[e + 2], std::integral_constant<int, 0x4E>{});  // quad_perm 2,3,0,1
    return (b0 ? z[1] : z[0]) + swap(b0 ? z[0] : z[1], std::integral_constant<int, 0xB1>{});  // quad_perm 1,0,3,2
}
__device__ __forceinline__ int token_of(int col, int g) { return 16 * (2 * (col >> 2 & 1) + (col >> 3)) + 4 * g + (col & 3); }

__device__ __forceinline__ rsrc_t page_record(const Attend& a, int page, int h, int bytes, bool& ok) {
    ok = page >= 0 && page < a.pages;
    return make_rsrc(a.cache + ((int64_t)(ok ? page : 0) * a.heads + h) * bytes, ok ? bytes : 0);
}

// Few rows, up to 16 or 64 (ONE: their operand stays in registers, else in LDS): each
// workgroup brings them once and then streams its share of a sequence's pages, a
// page a wave, the next one's codes on their way.  Workgroup n of a sequence takes
// pages 4 n .. 4 n + 3 and those `groups` workgroups further on: an even share of whatever
// length it has, below whatever limit.
template <int D, int BITS, int NQ, bool ONE>
__global__ __launch_bounds__(64 * WAVES, D == 256 ? 1 : 2) void weights_few_kernel(AttendWeights w) {
    constexpr int KS = D / 32, TILES = ONE ? 1 : 4;
    const Attend& a = w.a;
    __shared__ float qs[ONE ? 1 : WAVES][ROWS][D + 4];
    __shared__ uint4 op[TILES][NQ][ONE ? 1 : KS][64];
    __shared__ RowInfo info[TILES][ROWS];
    __shared__ float scales[WAVES][KV_PAGE];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int h = (int)(blockIdx.x % a.heads);
    const int64_t id = blockIdx.x / a.heads, b = id / w.groups;
    const int c0 = (int)(id % w.groups) * WAVES, step = w.groups * WAVES;
    const int32_t* table = a.table + b * a.max_pages;
    // (of the table's, whatever the length: it then needs not be waited for)
    const int first_page = __builtin_amdgcn_readfirstlane(table[min((int64_t)c0 + wave, a.max_pages - 1)]);
    const Sequence seq = sequence_of_lane(sequence_of(a, b), 0);
    const int pages = (seq.len + KV_PAGE - 1) / KV_PAGE;
    if (c0 >= pages) return;
    constexpr int bytes = kv_record_of(BITS, D);
    const Widen masks;
    PageKeys<D, BITS> keys;
    bool ok = false, next_ok;
    int p = c0 + wave;
    const auto page_at = [&](int64_t p) { return __builtin_amdgcn_readfirstlane(p < pages ? table[p] : -1); };
    // a row's values and the first page set out together
    const int rows = seq.nq * a.group, tiles = (rows + ROWS - 1) / ROWS;
    h8_t qf[NQ][KS];
    RowInfo mine{1.0f, INFINITY, 0, -1};
    if constexpr (ONE) {
        constexpr int NI = (ROWS * (D / 8) + 64 * WAVES - 1) / (64 * WAVES);
        const Tile tile = item_tile(a, seq, 0);
        QueryItem qi[NI];
#pragma unroll
        for (int n = 0; n < NI; ++n) {
            const int i = threadIdx.x + 64 * WAVES * n, r = i / (D / 8);
            if (r < rows && r < ROWS) fetch_q<D>(a, seq, h, row_of_tile(a, tile, r), i % (D / 8), qi[n]);
        }
        keys.fetch(page_record(a, p < pages ? first_page : -1, h, bytes, ok), lane);
        mine = info_of(w, seq, tile, h, col);
#pragma unroll
        for (int n = 0; n < NI; ++n) {
            const int i = threadIdx.x + 64 * WAVES * n, r = i / (D / 8), q = i % (D / 8);
            if (r >= ROWS) continue;
            if (r < rows) {
                fetch_turn(a, q, qi[n]);
                put_q(a, q, qi[n], qs[0][r]);
            } else {
                *reinterpret_cast<float4*>(&qs[0][r][8 * q]) = make_float4(0, 0, 0, 0);
                *reinterpret_cast<float4*>(&qs[0][r][8 * q + 4]) = make_float4(0, 0, 0, 0);
            }
        }
        __syncthreads();
        mine.unit = query_operand<D, NQ>(a, qs[0][col], g, qf);
    } else {
        keys.fetch(page_record(a, p < pages ? first_page : -1, h, bytes, ok), lane);
        if (wave < tiles) {
            mine = stage_rows<D, NQ>(w, seq, h, wave, lane, qs[wave], qf);
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int s = 0; s < KS; ++s) op[wave][n][s][lane] = __builtin_bit_cast(uint4, qf[n][s]);
            if (g == 0) info[wave][col] = mine;
        }
        __syncthreads();
    }
    const int64_t row = (b * a.heads + h) * w.stride;
    for (; p < pages; p += step) {
        const int j0 = p * KV_PAGE, j = j0 + token_of(col, g);
        const float before = w.old && j < seq.len - seq.n ? w.old[row + j] : 0.0f;
        scales[wave][lane] = keys.scale;
        float sum[4][4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[q][i] = 0.0f;
        const rsrc_t rec = page_record(a, page_at((int64_t)p + step), h, bytes, next_ok);
        if constexpr (ONE) {
            f4_t s4[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) s4[q] = f4_t{0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < KS / 2; ++s) {
                h8_t kf[4][2];
#pragma unroll
                for (int q = 0; q < 4; ++q) keys.widen(masks, q, s, kf[q][0], kf[q][1]);
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            s4[q] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[q][t], qf[n][2 * s + t], s4[q], 0, 0, 0);
            }
            keys.fetch(rec, lane);
            if (ok) add_row(s4, scales[wave], mine, j0, g, sum);
        } else {
            h8_t kf[4][KS];
#pragma unroll
            for (int s = 0; s < KS / 2; ++s)
#pragma unroll
                for (int q = 0; q < 4; ++q) keys.widen(masks, q, s, kf[q][2 * s], kf[q][2 * s + 1]);
            keys.fetch(rec, lane);
            if (ok)
                for (int i = 0; i < tiles; ++i) {
                    f4_t s4[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) s4[q] = f4_t{0, 0, 0, 0};
#pragma unroll
                    for (int s = 0; s < KS; ++s)
#pragma unroll
                        for (int n = 0; n < NQ; ++n) {
                            const h8_t x = __builtin_bit_cast(h8_t, op[i][n][s][lane]);
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                s4[q] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[q][s], x, s4[q], 0, 0, 0);
                        }
                    add_row(s4, scales[wave], info[i][col], j0, g, sum);
                }
        }
        const float got = rows_sum(sum, col);
        if (j < seq.len) w.weights[row + j] = __builtin_fmaf(before, w.keep, got);
        ok = next_ok;
    }
}

// How many of a sequence's `groups` workgroups there are groups of pages for, and
// shares of the rows that leave the others something to do: by the lengths on the
// device, not by the limits that the grid was made for.
struct Shares {
    int groups, splits;
};
__device__ __forceinline__ Shares shares_of(const AttendWeights& w, const Sequence& seq, int group_pages) {
    const int64_t tokens = (int64_t)group_pages * KV_PAGE;
    Shares s;
    s.groups = (int)((seq.len + tokens - 1) / tokens);
    const int tiles = (seq.nq * w.a.group + ROWS - 1) / ROWS, most = max(1, (tiles + LEAST_TILES - 1) / LEAST_TILES);
    s.splits = s.groups > 0 ? max(1, min(w.groups / s.groups, most)) : 1;
    return s;
}

// Many rows: they become operands once, in the workspace, sixteen to a piece of
// NQ D/32 + 1 KB (the last: their RowInfo, four times over).
template <int D, int NQ>
constexpr int piece_kb() { return NQ * (D / 32) + 1; }
__device__ __forceinline__ int64_t first_piece(const Attend& a, const Sequence& seq, int64_t b) {
    return (int64_t)seq.q0 * a.group / ROWS + b;  // sequences' rows are ascending: pieces do not meet
}
template <int D, int NQ>
__global__ __launch_bounds__(64 * WAVES) void weights_rows_kernel(AttendWeights w) {
    const Attend& a = w.a;
    __shared__ float qs[WAVES][ROWS][D + 4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t id = (int64_t)blockIdx.x * WAVES + wave;
    const int h = (int)(id % a.heads);
    const int t = (int)(id / a.heads % a.tiles_max);
    const int64_t b = id / a.heads / a.tiles_max;
    if (b >= a.B) return;
    const Sequence seq = sequence_of_lane(sequence_of(a, b), 0);
    if (t * ROWS >= seq.nq * a.group) return;
    h8_t qf[NQ][D / 32];
    const RowInfo o = stage_rows<D, NQ>(w, seq, h, t, lane, qs[wave], qf);
    uint4* to = w.rows + ((first_piece(a, seq, b) + t) * a.heads + h) * (64 * piece_kb<D, NQ>()) + lane;
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int s = 0; s < D / 32; ++s) to[64 * (n * (D / 32) + s)] = __builtin_bit_cast(uint4, qf[n][s]);
    to[64 * NQ * (D / 32)] = __builtin_bit_cast(uint4, o);
}

// Then each workgroup holds the keys of PAGES pages a wave, widened once, and its share
// of the rows goes by: pieces by the buffer into LDS, TS at a time, the next ones on
// their way while these are multiplied, one barrier for TS.
template <int D, int BITS, int NQ>
__global__ __launch_bounds__(64 * WAVES, 2) void weights_many_kernel(AttendWeights w) {
    constexpr int KS = D / 32, PAGES = D == 256 ? 1 : 2, KB = piece_kb<D, NQ>(), TS = D == 256 ? 2 : 4;
    const Attend& a = w.a;
    __shared__ uint4 ops[2][TS][KB][64];
    __shared__ float scales[WAVES][PAGES][KV_PAGE];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    int64_t id = blockIdx.x;
    const int h = (int)(id % a.heads);
    id /= a.heads;
    const int64_t b = id / w.groups;
    const Sequence seq = sequence_of_lane(sequence_of(a, b), 0);
    const Shares sh = shares_of(w, seq, WAVES * PAGES);
    const int place = uni((int)(id % w.groups)), split = uni(sh.groups > 0 ? place / sh.groups : 1);
    if (split >= sh.splits) return;
    // (the two workgroups that a compute unit starts with: not in the same phase, attend_tile.hip)
    if (blockIdx.x >> 8 & 1) __builtin_amdgcn_s_setprio(1);
    const int c0 = (place - split * sh.groups) * (WAVES * PAGES);
    const int32_t* table = a.table + b * a.max_pages;
    constexpr int bytes = kv_record_of(BITS, D);
    // rows that may see one of these pages
    const int past = seq.len - seq.n, i0 = min(max(0, c0 * KV_PAGE - past), seq.nq);
    int64_t i1 = seq.nq;
    if (a.window > 0) i1 = min(i1, (int64_t)(c0 + WAVES * PAGES) * KV_PAGE - 1 + a.window - past);
    const int r0 = uni(i0 * a.group / ROWS), r1 = uni(i1 > i0 ? (int)((i1 * a.group + ROWS - 1) / ROWS) : r0);
    const int each = (r1 - r0 + sh.splits - 1) / sh.splits, t0 = r0 + split * each, t1 = min(r1, t0 + each);
    const uint4* pieces = w.rows + (first_piece(a, seq, b) * a.heads + h) * (64 * KB);
    const int64_t step = (int64_t)a.heads * (64 * KB);
    const auto bring = [&](int t, int buf) {
#pragma unroll
        for (int i = 0; i < (TS * KB + WAVES - 1) / WAVES; ++i) {
            const int x = wave + WAVES * i;
            if (x >= TS * KB) break;
            const rsrc_t src = make_rsrc(pieces + min(t + x / KB, t1 - 1) * step, KB * 1024);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void*)&ops[buf][x / KB][x % KB][0],
                                                     16, 16 * lane, (x % KB) * 1024, 0, 0);
        }
    };
    const Widen masks;
    h8_t kf[PAGES][4][KS];
    bool ok[PAGES];
    float sum[PAGES][4][4];
#pragma unroll
    for (int n = 0; n < PAGES; ++n) {
        const int p = c0 + wave * PAGES + n;
        PageKeys<D, BITS> keys;
        const int page = __builtin_amdgcn_readfirstlane(p * KV_PAGE < seq.len ? table[p] : -1);
        keys.fetch(page_record(a, page, h, bytes, ok[n]), lane);
        if (n == 0 && t0 < t1) bring(t0, 0);
#pragma unroll
        for (int s = 0; s < KS / 2; ++s)
#pragma unroll
            for (int q = 0; q < 4; ++q) keys.widen(masks, q, s, kf[n][q][2 * s], kf[n][q][2 * s + 1]);
        scales[wave][n][lane] = keys.scale;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[n][q][e] = 0.0f;
    }
    for (int t = t0, buf = 0; t < t1; t += TS, buf ^= 1) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (t + TS < t1) bring(t + TS, buf ^ 1);
        for (int i = 0; i < TS && t + i < t1; ++i) {
            const RowInfo row = __builtin_bit_cast(RowInfo, ops[buf][i][KB - 1][lane]);
            f4_t s4[PAGES][4];
#pragma unroll
            for (int n = 0; n < PAGES; ++n)
#pragma unroll
                for (int q = 0; q < 4; ++q) s4[n][q] = f4_t{0, 0, 0, 0};
#pragma unroll
            for (int m = 0; m < NQ; ++m)
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const h8_t x = __builtin_bit_cast(h8_t, ops[buf][i][m * KS + s][lane]);
#pragma unroll
                    for (int n = 0; n < PAGES; ++n)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            s4[n][q] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[n][q][s], x, s4[n][q], 0, 0, 0);
                }
            __builtin_amdgcn_sched_barrier(0);  // keeps to two waves' registers
#pragma unroll
            for (int n = 0; n < PAGES; ++n)
                if (ok[n]) add_row(s4[n], scales[wave][n], row, (c0 + wave * PAGES + n) * KV_PAGE, g, sum[n]);
        }
    }
#pragma unroll
    for (int n = 0; n < PAGES; ++n) {
        const float got = rows_sum(sum[n], col);
        const int j = (c0 + wave * PAGES + n) * KV_PAGE + token_of(col, g);
        if (j >= seq.len) continue;
        if (sh.splits > 1) {
            w.part[((b * a.heads + h) * w.groups + place) * (WAVES * PAGES * KV_PAGE) + (j - c0 * KV_PAGE)] = got;
        } else {
            const int64_t at = (b * a.heads + h) * w.stride + j;
            w.weights[at] = __builtin_fmaf(w.old && j < past ? w.old[at] : 0.0f, w.keep, got);
        }
    }
}

// Adds up the shares of the rows, in order.
__global__ __launch_bounds__(256) void weights_join_kernel(AttendWeights w) {
    const Attend& a = w.a;
    const int64_t per = (a.max_len + 255) / 256, bh = blockIdx.x / per, b = bh / a.heads;
    const int64_t j = (blockIdx.x % per) * 256 + threadIdx.x;
    const Sequence seq = sequence_of(a, b);
    const Shares sh = shares_of(w, seq, w.group_pages);
    if (j >= seq.len || sh.splits == 1) return;
    const int64_t tokens = (int64_t)w.group_pages * KV_PAGE;
    const float* part = w.part + (bh * w.groups + j / tokens) * tokens + j % tokens;
    float got = 0.0f;
    for (int s = 0; s < sh.splits; ++s) got += part[s * sh.groups * tokens];
    const int64_t at = bh * w.stride + j;
    w.weights[at] = __builtin_fmaf(w.old && j < seq.len - seq.n ? w.old[at] : 0.0f, w.keep, got);
}

template <int D, int BITS, int NQ>
hipError_t weights_n(const WeightsPlan& p, const AttendWeights& w, hipStream_t s) {
    const dim3 grid((unsigned)p.workgroups), block(64 * WAVES);
    if (!p.many) {
        if (p.rows <= ROWS)
            Q8K_LAUNCH((weights_few_kernel<D, BITS, NQ, true>), grid, block, 0, s, w);
        else
            Q8K_LAUNCH((weights_few_kernel<D, BITS, NQ, false>), grid, block, 0, s, w);
        return hipGetLastError();
    }
    const int64_t waves = w.a.B * w.a.heads * w.a.tiles_max;
    Q8K_LAUNCH((weights_rows_kernel<D, NQ>), dim3((unsigned)((waves + WAVES - 1) / WAVES)), block, 0, s, w);
    Q8K_LAUNCH((weights_many_kernel<D, BITS, NQ>), grid, block, 0, s, w);
    if (p.split) Q8K_LAUNCH(weights_join_kernel, dim3((unsigned)p.join_workgroups), dim3(256), 0, s, w);
    return hipGetLastError();
}
template <int D, int BITS>
hipError_t weights_d(const WeightsPlan& p, const AttendWeights& w, hipStream_t s) {
    return w.a.dtype == DT_BF16 && !w.a.rope.table ? weights_n<D, BITS, 1>(p, w, s) : weights_n<D, BITS, 2>(p, w, s);
}

}  // namespace

// Up to FEW_ROWS rows a head, what four tiles in LDS hold: one launch (16 sequences of up to
// 8191 tokens, 32 heads over 8, 4 bits: of 5 new tokens, 20 rows, 24.7 us, as operands in the
// workspace 30.8; of 8 28.9 and 33.4; of 16, 64 rows, 35.6 and 38.2; one sequence of 16 over
// 8191 9.0 and 15.9), as many workgroups a sequence and head as make FEW_WGS (16 sequences of
// up to 8191 tokens, 8 bits: 20.2 us, 512 of them 24.4, 1536 22.6, 2048 23.1; 1 x 65537 12.5,
// 12.7, 14.2 and 14.4; 8 x 65537 64, 73, 64.5 and 63; 4 bits, 16 x up to 8191 17.5, by 512
// 21.3, by 2048 19.4, five new tokens each 24.7, 22.8 and 29.3; 16 x 16001 of heads of 64 26.5,
// 30.6 and 26.5, of 256 66.9, 65.8 and 72.3).  More rows: their operands in the workspace,
// groups of 2 WAVES pages (of 256 values WAVES), and the rows in as many shares as make
// MANY_WGS workgroups (2 x 1000 tokens over 8001, 32 heads over 4: 225 us, by 1024 230, by 4096
// 240, under a window of 1000 153, 150 and 160; of heads of 64 151, 149 and 154, of 256 409, 419
// and 419; up to 700 of three over up to 6000, 32 over 8: 129, 147 and 131; 1000 over 16001,
// fp32: 223, 230 and 229), each of LEAST_TILES tiles at least.
constexpr int64_t FEW_ROWS = 64, FEW_WGS = 1024, MANY_WGS = 2048;

WeightsPlan weights_plan(int64_t B, int64_t Tq, int64_t max_q, int64_t max_len, int q_heads, int heads, int D) {
    WeightsPlan p{};
    const int64_t group = q_heads / heads, pages = (max_len + KV_PAGE - 1) / KV_PAGE;
    p.rows = max_q * group;
    p.many = p.rows > FEW_ROWS;
    p.threads = 64 * WAVES;
    p.tiles_max = (p.rows + ROWS - 1) / ROWS;
    // workgroups that a sequence and head has pages for, and those that fill the device
    p.group_pages = p.many && D < 256 ? 2 * WAVES : WAVES;
    const int64_t most = (pages + p.group_pages - 1) / p.group_pages;
    const int64_t fill = ((p.many ? MANY_WGS : FEW_WGS) + B * heads - 1) / (B * heads);
    if (!p.many) {
        p.groups = most < fill ? most : fill;
    } else {
        p.split = p.tiles_max > LEAST_TILES;
        p.groups = p.split && fill > most ? fill : most;
        p.rows_bytes = (Tq * group / ROWS + B + 1) * heads * (2 * (D / 32) + 1) * 1024;
        p.join_workgroups = B * heads * ((max_len + 255) / 256);
        p.ws_bytes = p.rows_bytes + (p.split ? B * heads * p.groups * p.group_pages * KV_PAGE * 4 : 0);
    }
    p.workgroups = B * heads * p.groups;
    return p;
}

hipError_t launch_attend_weights(int bits, int D, const WeightsPlan& p, AttendWeights w, void* ws, hipStream_t s) {
    w.a.tile_rows = ROWS;
    w.a.tiles_max = (int)p.tiles_max;
    w.a.inv_group = 1.0f / (float)w.a.group;
    w.groups = (int)p.groups;
    w.group_pages = (int)p.group_pages;
    w.rows = static_cast<uint4*>(ws);
    w.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + p.rows_bytes);
    if (bits == 8) return D == 64 ? weights_d<64, 8>(p, w, s) : D == 128 ? weights_d<128, 8>(p, w, s) : weights_d<256, 8>(p, w, s);
    return D == 64 ? weights_d<64, 4>(p, w, s) : D == 128 ? weights_d<128, 4>(p, w, s) : weights_d<256, 4>(p, w, s);
}

}  // namespace q8k
