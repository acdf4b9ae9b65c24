// What each cached token gets of the new tokens' attention, per key head:
//   w_j = keep old_j + sum over rows r that see j of e^(s_rj - lse_r),  s_rj = scale <q_r, key_j>,
// rows being the key head's query heads times the new tokens, lse their log sums
// as attention left them.  With lse known no row needs its other tokens, so the
// sum over rows stays where the tokens are: a wave holds the keys of one page, widened
// once, and adds up its 64 tokens while the rows go by.  No atomics: one order always.
#include "attend.h"

namespace q8k {

namespace {

constexpr int WAVES = 4, ROWS = 16;

// A page's keys of one head as the product's operand.
template <int D, int BITS>
__device__ __forceinline__ void page_keys(rsrc_t rec, int lane, h8_t (&kf)[4][D / 32]) {
    const int col = lane & 15, g = lane >> 4, off = col * 64 + g * 16;
    if constexpr (BITS == 8) {
        uint4 raw[4][D / 64];
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int s = 0; s < D / 64; ++s) raw[q][s] = load16_nt(rec, off + s * 4096 + q * 1024);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int s = 0; s < D / 64; ++s) {
                kf[q][2 * s] = codes_f16(raw[q][s].x, raw[q][s].y);
                kf[q][2 * s + 1] = codes_f16(raw[q][s].z, raw[q][s].w);
            }
    } else {
        uint4 raw[D / 32];
        uint32_t fac[D / 64];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) raw[i] = load16_nt(rec, off + i * 1024);
        load_words<D / 64>(rec, KV4_KF(D) + (col * 2 + (g >> 1)) * (D / 16), fac);
#pragma unroll
        for (int p = 0; p < D / 16; ++p) {
            const int q = p / (D / 64), s = p % (D / 64);
            const uint4 c = raw[p >> 1];
            const Factors f = kv4_key_factors(fac[p >> 2] >> (8 * (p & 3)) & 255u);
            kf[q][2 * s] = kv4_widen_keys(p & 1 ? c.z : c.x, f);
            kf[q][2 * s + 1] = kv4_widen_keys(p & 1 ? c.w : c.y, f);
        }
    }
}

struct RowInfo {
    float unit, lse;  // of the products, and log2 of the sum; inf where the row sees nothing
    int first, last;  // the tokens that it sees
};

// One workgroup: four pages of one sequence and head, and its share of the rows.
// Sixteen rows a wave become operands in LDS, which all waves then multiply.
template <int D, int BITS, int NQ>
__global__ __launch_bounds__(64 * WAVES, 1) void attend_weights_kernel(AttendWeights w) {
    constexpr int KS = D / 32;
    const Attend& a = w.a;
    __shared__ float qs[WAVES][ROWS][D + 4];
    __shared__ uint4 op[WAVES][NQ][KS][64];
    __shared__ RowInfo info[WAVES][ROWS];
    __shared__ float scales[WAVES][KV_PAGE];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    int64_t id = blockIdx.x;
    const int h = (int)(id % a.heads);
    id /= a.heads;
    const int split = (int)(id % w.splits);
    id /= w.splits;
    const int64_t b = id / w.page_groups;
    const int p0 = (int)(id % w.page_groups) * WAVES;
    const Sequence seq = sequence_of_lane(sequence_of(a, b), 0);
    if (p0 * KV_PAGE >= seq.len) return;
    const int p = p0 + wave, j0 = p * KV_PAGE;
    const int page = __builtin_amdgcn_readfirstlane(j0 < seq.len ? a.table[b * a.max_pages + p] : -1);
    const bool ok = page >= 0 && page < a.pages;
    constexpr int bytes = kv_record_of(BITS, D);
    const rsrc_t rec = make_rsrc(a.cache + ((int64_t)(ok ? page : 0) * a.heads + h) * bytes, ok ? bytes : 0);
    h8_t kf[4][KS];
    page_keys<D, BITS>(rec, lane, kf);
    scales[wave][lane] = __builtin_bit_cast(float, load4(rec, bytes - 8 * KV_PAGE + 4 * lane));
    float ks[4][4], sum[4][4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float4 k = *reinterpret_cast<const float4*>(&scales[wave][16 * q + 4 * g]);
        ks[q][0] = k.x, ks[q][1] = k.y, ks[q][2] = k.z, ks[q][3] = k.w;
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[q][i] = 0.0f;
    }
    const int rows = seq.nq * a.group, tiles = (rows + ROWS - 1) / ROWS;
    const int each = (tiles + w.splits - 1) / w.splits, t0 = split * each, t1 = min(tiles, t0 + each);
    for (int t = t0; t < t1; t += WAVES) {
        if (t + wave < t1) {
            const Tile tile = item_tile(a, seq, t + wave);
            float(*q_s)[D + 4] = qs[wave];
#pragma unroll
            for (int n = 0; n < D / 32; ++n) {
                const int i = lane + 64 * n, r = i / (D / 8), it = i % (D / 8);
                QueryItem qi;
                fetch_q<D>(a, seq, h, row_of_tile(a, tile, min(r, rows - 1 - tile.row0)), it, qi);
                fetch_turn(a, it, qi);
                put_q(a, it, qi, q_s[r]);
            }
            __builtin_amdgcn_wave_barrier();
            h8_t qf[NQ][KS];
            const float unit = query_operand<D, NQ>(a, q_s[col], g, qf);
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int s = 0; s < KS; ++s) op[wave][n][s][lane] = __builtin_bit_cast(uint4, qf[n][s]);
            if (g == 0) {
                RowInfo o{unit, INFINITY, 0, -1};
                if (tile.row0 + col < rows) {
                    const TileRow tr = row_of_tile(a, tile, col);
                    const Span sp = span_of(a, seq, tr.tok);
                    const float lse = w.lse[q_row_of(a, seq, h, tr)];
                    // (a row of -inf sees nothing that counts)
                    o = RowInfo{unit, lse == -INFINITY ? INFINITY : lse * LOG2E, sp.first, sp.last};
                }
                info[wave][col] = o;
            }
        }
        __syncthreads();
        for (int i = 0; i < WAVES && t + i < t1; ++i) {
            const RowInfo row = info[i][col];
            const bool sees = ok && row.first < j0 + KV_PAGE && row.last >= j0;
            if (!__any(sees)) continue;
            f4_t s4[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) s4[q] = f4_t{0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    const h8_t qf = __builtin_bit_cast(h8_t, op[i][n][s][lane]);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        s4[q] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[q][s], qf, s4[q], 0, 0, 0);
                }
            const bool whole = !__any(row.first > j0 || row.last < j0 + KV_PAGE - 1);
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s4[q][e] * ks[q][e], row.unit, -row.lse));
                    const int j = j0 + 16 * q + 4 * g + e;
                    sum[q][e] += whole || (j >= row.first && j <= row.last) ? x : 0.0f;
                }
        }
        __syncthreads();
    }
    if (j0 >= seq.len) return;
    // over the sixteen rows' lanes, then lane (col, g) keeps token 16 (col / 4) + 4 g + col % 4
    float mine = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float v = sum[q][e];
#pragma unroll
            for (int k = 0; k < 4; ++k) v += dpp_f(v, k);
            mine = col == 4 * q + e ? v : mine;
        }
    const int j = j0 + 16 * (col >> 2) + 4 * g + (col & 3);
    if (j >= seq.len) return;
    if (w.splits > 1) {
        w.part[((split * a.B + b) * a.heads + h) * (int64_t)w.page_groups * (WAVES * KV_PAGE) + j] = mine;
        return;
    }
    const int64_t at = (b * a.heads + h) * w.stride + j;
    w.weights[at] = w.old && j < seq.len - seq.n ? __builtin_fmaf(w.old[at], w.keep, mine) : mine;
}

template <int D, int BITS>
hipError_t weights_d(const AttendWeights& w, unsigned grid, hipStream_t s) {
    if (w.a.dtype == DT_BF16 && !w.a.rope.table)
        Q8K_LAUNCH((attend_weights_kernel<D, BITS, 1>), dim3(grid), dim3(64 * WAVES), 0, s, w);
    else
        Q8K_LAUNCH((attend_weights_kernel<D, BITS, 2>), dim3(grid), dim3(64 * WAVES), 0, s, w);
    return hipGetLastError();
}

}  // namespace

WeightsPlan weights_plan(int64_t B, int64_t max_q, int64_t max_len, int q_heads, int heads, int D) {
    WeightsPlan p;
    p.page_groups = (max_len + WAVES * KV_PAGE - 1) / (WAVES * KV_PAGE);
    p.splits = 1;
    p.workgroups = B * heads * p.page_groups * p.splits;
    p.threads = 64 * WAVES;
    p.ws_bytes = 0;
    return p;
}

hipError_t launch_attend_weights(int bits, int D, const WeightsPlan& p, AttendWeights w, void* ws, hipStream_t s) {
    w.a.tile_rows = ROWS;
    w.a.inv_group = 1.0f / (float)w.a.group;
    w.page_groups = (int)p.page_groups;
    w.splits = p.splits;
    w.part = static_cast<float*>(ws);
    const unsigned grid = (unsigned)p.workgroups;
    if (bits == 8)
        return D == 64 ? weights_d<64, 8>(w, grid, s) : D == 128 ? weights_d<128, 8>(w, grid, s) : weights_d<256, 8>(w, grid, s);
    return D == 64 ? weights_d<64, 4>(w, grid, s) : D == 128 ? weights_d<128, 4>(w, grid, s) : weights_d<256, 4>(w, grid, s);
}

}  // namespace q8k
