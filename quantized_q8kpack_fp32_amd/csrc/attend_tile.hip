// Attention of many rows over the paged 8-bit cache: prompts and chunks of
// them.  The formula of attend_decode.hip; here the arithmetic bounds it, so the
// codes become fp16 once for 64 or 128 rows and are read by all waves from LDS.
//
// Chunks of up to 1000 tokens of three prompts over up to 16001 (32 heads of 128
// over 4, bf16, turned): 802 us, 575 TFLOP/s of the formula's, where a large matrix
// product reaches 1140.  A query of two fp16 pieces makes the first product twice as
// long as the formula's, so that the matrix work alone would take 607 us at that
// rate; matrix instructions are busy for 36% of the cycles and vector ones (some
// twelve a score) for 41%, and little of the two overlaps: each wave does a page's
// scores, probabilities and values in turn, and the waves of a unit are in the same
// phase behind one barrier a page (scheduling groups that put the instructions
// between each other, and wave priorities, gained nothing).  The 1000, 443 and 787
// tokens make 564 tiles with work, of unequal length, on 512 places, the longest
// first; four of 1024 over 8192, 1024 tiles of nearly one length, reach 695.
#include "attend.h"

namespace q8k {

namespace {

// Probabilities enter the second product as fp16 pieces of p * vscale / U, U a
// row's own power of two: R / 2^15 of attend_decode.hip.  1 / U lies in the
// exponent, e^(s - m) / U = 2^(s log2 e - m + K), so that it costs no
// instruction a score; m is kept whole, so that K - m is exact, and the sum of the
// probabilities has the same unit.  From 2^-100 on, so that no sum overflows.
constexpr int K_FIRST = 100;

// One page's operands in LDS, in the order in which the lanes of a wave read
// them: every read and write of 16 bytes a lane is 1 KB of consecutive bytes.
template <int D>
struct PageOps {
    uint4 k[4][D / 32][64];  // [16 tokens][k step][lane]
    uint4 v[D / 16][2][64];  // [16 values][32 tokens][lane]
    float ks[KV_PAGE], vs[KV_PAGE];
    // The largest of the vs that some row of the tile sees; NaN where one of these is
    // infinite or NaN: such ones are zeros in vs, and bits in `odd`.
    float vmax;
    uint32_t odd[2], pad;
};

// One workgroup: 64 RT rows of one key head over its split's pages, 16 RT rows
// a wave.  While a page is multiplied, the next one's codes, in registers since
// the page before, become fp16 in the other buffer, and the one after that is
// on its way from memory: one barrier a page.  HALVES == 2: as many waves again
// take every other page, with buffers of their own, and the two results are
// joined through LDS: for calls of few short tiles, where a tile's own time
// counts (512 tokens of one prompt, 32 heads of 128 over 8: 21.6 us when this was
// chosen and 24.3 with one half, 19.8 now; tiles that are split into chunks lose
// by it: 500 tokens over 16001 283 us, 275).  Heads of 64 values in 128-row tiles
// keep to the registers of three waves a SIMD (chunks of 1000 over 8000: 230 us, of
// two waves 300).
template <int D, int WAVES, int HALVES, int RT, int NQ, int NP>
__global__ __launch_bounds__(64 * WAVES * HALVES, D == 64 && RT == 2 ? 3 : 2) void attend_tile_kernel(Attend a) {
    constexpr int KS = D / 32, DB = D / 16, ROWS = 16 * RT * WAVES;
    constexpr int KC = D / 16 / WAVES;  // 1 KB pieces of a page's keys (and of its values) a wave brings
    __shared__ union {
        PageOps<D> ops[HALVES][2];
        float q[HALVES * WAVES][16][D + 4];  // the queries on their way to registers
        struct {
            float4 acc[RT][D / 16][64];
            float2 ml[RT][64];
        } join[WAVES];
    } sm;
    const int lane = threadIdx.x & 63, wave_of_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = wave_of_all / WAVES, wave = wave_of_all % WAVES;
    PageOps<D>* ops = sm.ops[half];
    const int col = lane & 15, g = lane >> 4;
    const int h = (int)(blockIdx.x % a.heads);
    const int64_t item = blockIdx.x / a.heads;
    Item it;
    if (!item_of(a, item, it)) return;
    const Sequence seq = it.seq;
    const Tile tile = item_tile(a, seq, it.tile);
    const int rows = tile.rows;
    if (tile.row0 >= rows) return;
    const int p0 = uni(tile.p0 + it.split * it.c), p1 = uni(min(tile.p1, p0 + it.c));
    if (it.splits > 1 && p0 >= p1) return;  // the join reads only chunks that some row's span meets

    // The wave's queries: all on their way at once, then 16 rows at a time
    // through its part of LDS into the registers that the products take.
    h8_t qf[RT][NQ][KS];
    float unit[RT];
    int last[RT];  // the last token that the row sees; it sees those less than `window` before it
    const uint32_t window = a.window > 0 ? (uint32_t)a.window : 0x7fffffffu;
    {
        constexpr int NI = D / 32;  // items of 16 rows a lane
        float(*qs)[D + 4] = sm.q[wave_of_all];
        QueryItem qi[RT][NI];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int n = 0; n < NI; ++n) {
                const int i = lane + 64 * n, r = (wave * RT + rt) * 16 + i / (D / 8);
                fetch_q<D>(a, seq, h, row_of_tile(a, tile, min(r, rows - 1 - tile.row0)), i % (D / 8), qi[rt][n]);
            }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int n = 0; n < NI; ++n) fetch_turn(a, (lane + 64 * n) % (D / 8), qi[rt][n]);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
            for (int n = 0; n < NI; ++n) {
                const int i = lane + 64 * n;
                put_q(a, i % (D / 8), qi[rt][n], qs[i / (D / 8)]);
            }
            unit[rt] = query_operand<D, NQ>(a, qs[col], g, qf[rt]);
            last[rt] = span_of(a, seq, row_of_tile(a, tile, min((wave * RT + rt) * 16 + col, rows - 1 - tile.row0)).tok).last;
        }
    }
    __syncthreads();

    // A page's codes on their way: wave w brings pieces w, w + WAVES, ... of the
    // keys (16 tokens of one plane each) and of the values (16 rows each), wave
    // 0 the keys' scales and wave 1 the values'.  Reads go through a buffer
    // descriptor of one record, an empty one where the page selects nothing.
    // Page numbers come 64 at a time, one a lane.
    const int32_t* pages = a.table + it.b * a.max_pages;
    int ids = p0 + lane < p1 ? pages[p0 + lane] : -1;
    const int lane_off = col * 64 + g * 16;
    uint4 kraw[KC], vraw[KC];
    float sc_raw;
    int at_p;  // the page that the registers hold
    bool raw_ok;
    const auto fetch = [&](int p) {
        const int n = p - p0;
        // (tiles of two halves have at most 33 pages: attend_plan)
        if (HALVES == 1 && n > 0 && (n & 63) == 0) ids = p + lane < p1 ? pages[p + lane] : -1;
        const int page = __builtin_amdgcn_readlane(ids, n & 63);
        at_p = p;
        raw_ok = p < p1 && page >= 0 && page < a.pages;
        const rsrc_t rec = make_rsrc(a.cache + ((int64_t)(raw_ok ? page : 0) * a.heads + h) * kv_record(D),
                                     raw_ok ? kv_record(D) : 0);
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            kraw[c] = load16(rec, lane_off + (wave + WAVES * c) * 1024);
            vraw[c] = load16(rec, lane_off + KV_PAGE * D + (wave + WAVES * c) * 1024);
        }
        sc_raw = __builtin_bit_cast(float, load4(rec, 2 * KV_PAGE * D + 4 * (threadIdx.x & 127)));
    };
    const auto put = [&](PageOps<D>& o) {
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            // piece i of the keys: plane i / 4, tokens 16 (i % 4) and on
            const int i = wave + WAVES * c;
            o.k[i & 3][2 * (i >> 2)][lane] = __builtin_bit_cast(uint4, codes_f16(kraw[c].x, kraw[c].y));
            o.k[i & 3][2 * (i >> 2) + 1][lane] = __builtin_bit_cast(uint4, codes_f16(kraw[c].z, kraw[c].w));
            o.v[i][0][lane] = __builtin_bit_cast(uint4, codes_f16(vraw[c].x, vraw[c].y));
            o.v[i][1][lane] = __builtin_bit_cast(uint4, codes_f16(vraw[c].z, vraw[c].w));
        }
        if (wave == 0) o.ks[lane] = sc_raw;
        if (wave == 1) {
            // what lies in places that no row sees may be anything, NaN scales included
            const int j = at_p * KV_PAGE + lane;
            float v = j >= tile.lo.first && j <= tile.hi.last ? sc_raw : 0.0f;
            const uint64_t odd = __ballot(!(fabsf(v) < INFINITY));
            v = fabsf(v) < INFINITY ? v : 0.0f;
            o.vs[lane] = v;
            const float most = wave_max_dpp(v);
            if (lane == 0) {
                o.vmax = odd ? __builtin_nanf("") : most;
                o.odd[0] = (uint32_t)odd;
                o.odd[1] = (uint32_t)(odd >> 32);
            }
        }
    };

    float m[RT], l[RT], c[RT];  // l: the sum / U; c: K - m, or K where m is -inf or far
    bool far = false;           // some row's m is: is_far
    float U_least = pow2f(-K_FIRST);  // of the wave's rows
    const auto shift_of = [](float m) { return m == -INFINITY || is_far(m) ? 0.0f : m; };
    const auto unit_of = [&](int rt) { return pow2f(-(int)(c[rt] + shift_of(m[rt]))); };
    f4_t acc[RT][DB];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        m[rt] = -INFINITY, l[rt] = 0.0f, c[rt] = K_FIRST;
#pragma unroll
        for (int d = 0; d < DB; ++d) acc[rt][d] = f4_t{0, 0, 0, 0};
    }
    fetch(p0 + half);
    put(ops[0]);
    bool ok = raw_ok;
    fetch(p0 + half + HALVES);
    __syncthreads();
    for (int p = p0 + half, turn = 0; p - half < p1; p += HALVES, turn ^= 1) {
        const PageOps<D>& o = ops[turn];
        const bool next_ok = raw_ok;
        put(ops[turn ^ 1]);
        fetch(p + 2 * HALVES);
        if (ok) {
            // scores, the next 16 tokens' keys on their way while these are multiplied
            f4_t s4[RT][4];
            h8_t kf[2][KS];
#pragma unroll
            for (int s = 0; s < KS; ++s) kf[0][s] = __builtin_bit_cast(h8_t, o.k[0][s][lane]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (q < 3)
#pragma unroll
                    for (int s = 0; s < KS; ++s) kf[(q + 1) & 1][s] = __builtin_bit_cast(h8_t, o.k[q + 1][s][lane]);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) s4[rt][q] = f4_t{0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt)
                            s4[rt][q] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[q & 1][s], qf[rt][n][s], s4[rt][q], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 k = *reinterpret_cast<const float4*>(&o.ks[16 * q + 4 * g]);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    s4[rt][q][0] *= k.x;
                    s4[rt][q][1] *= k.y;
                    s4[rt][q][2] *= k.z;
                    s4[rt][q][3] *= k.w;
                }
            }
            // pages that some row sees only in part
            const bool in_part = p * KV_PAGE < tile.hi.first || p * KV_PAGE + KV_PAGE - 1 > tile.lo.last;
            if (in_part) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = p * KV_PAGE + 16 * q + 4 * g + i;
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt)
                            s4[rt][q][i] = (uint32_t)(last[rt] - j) < window ? s4[rt][q][i] : -INFINITY;
                    }
            }
            const float vmax = o.vmax;
            float tmax[RT];
            const bool more = !(vmax * 0x1p-15f <= U_least);
            bool grew = more || far;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                tmax[rt] = s4[rt][0][0];
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i) tmax[rt] = fmaxf(tmax[rt], s4[rt][q][i]);
                tmax[rt] *= unit[rt];
                grew |= tmax[rt] > m[rt];
            }
            if (__any(grew)) {
                float both[RT];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const float mn = fmaxf(m[rt], ceilf(groups_max(tmax[rt])));
                    both[rt] = __builtin_amdgcn_exp2f(m[rt] - (mn == -INFINITY ? 0.0f : mn));
                    c[rt] += shift_of(m[rt]) - shift_of(mn);
                    m[rt] = mn;
                    far |= __any(is_far(mn));
                }
                if (__any(more)) {
                    // The page's largest value scale that the row sees (not one that only other
                    // rows of the tile see: it would take this row's bits); NaN or infinite where
                    // it sees one that is not finite, and its result is NaN from here on.
                    float most[RT], least = INFINITY;
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) most[rt] = in_part ? 0.0f : vmax;
                    if (in_part) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const f4_t v = *reinterpret_cast<const f4_t*>(&o.vs[16 * q + 4 * g]);
                            const uint32_t odd = o.odd[q / 2] >> (16 * (q & 1) + 4 * g);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int j = p * KV_PAGE + 16 * q + 4 * g + i;
                                const float w = odd >> i & 1u ? INFINITY : v[i];
#pragma unroll
                                for (int rt = 0; rt < RT; ++rt)
                                    most[rt] = (uint32_t)(last[rt] - j) < window ? fmaxf(most[rt], w) : most[rt];
                            }
                        }
                    }
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        const float v = groups_max(most[rt]), U = unit_of(rt);
                        const bool odd = !(v < INFINITY);
                        if (__any(odd))
#pragma unroll
                            for (int d = 0; d < DB; ++d) acc[rt][d] *= odd ? __builtin_nanf("") : 1.0f;
                        const int e = exponent_of(v) - 14;
                        const bool raise = v > U * 0x1p15f && !odd;
                        both[rt] *= raise ? U * pow2f(-e) : 1.0f;
                        c[rt] = raise ? (float)-e - shift_of(m[rt]) : c[rt];
                        least = fminf(least, unit_of(rt));
                    }
                    U_least = uni_f(-wave_max_dpp(-least));
                }
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    l[rt] *= both[rt];
#pragma unroll
                    for (int d = 0; d < DB; ++d) acc[rt][d] *= both[rt];
                }
                if (far)
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        const float inv = 1.0f / unit[rt];
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                s4[rt][q][i] = is_far(m[rt]) ? far_score(s4[rt][q][i], unit[rt], inv, m[rt]) : s4[rt][q][i];
                    }
            }
            // The second product by halves of the page's tokens (all probabilities
            // first: 1.4% longer), its values two row blocks ahead.
            constexpr int AHEAD = 2;
            h8_t vf[AHEAD + 1];
#pragma unroll
            for (int d = 0; d < AHEAD; ++d) vf[d] = __builtin_bit_cast(h8_t, o.v[d][0][lane]);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                h8_t pf[RT][NP];
                uint32_t w[RT][2][2][2];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int q = 2 * t + b;
                    if (b && D == 64) __builtin_amdgcn_sched_barrier(0);  // keeps to three waves' registers
                    const f4_t v = *reinterpret_cast<const f4_t*>(&o.vs[16 * q + 4 * g]);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        float e[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s4[rt][q][i], unit[rt], c[rt]));
                            l[rt] += e[i];
                            e[i] *= v[i];
                        }
                        f16_pieces<NP>(e[0], e[1], w[rt][b][0]);
                        f16_pieces<NP>(e[2], e[3], w[rt][b][1]);
                    }
                }
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int n = 0; n < NP; ++n)
                        pf[rt][n] = __builtin_bit_cast(
                            h8_t, make_uint4(w[rt][0][0][n], w[rt][0][1][n], w[rt][1][0][n], w[rt][1][1][n]));
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    const int i = t * DB + d, k = i + AHEAD;
                    if (k < 2 * DB) vf[k % (AHEAD + 1)] = __builtin_bit_cast(h8_t, o.v[k % DB][k / DB][lane]);
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int n = 0; n < NP; ++n)
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt)
                            acc[rt][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[i % (AHEAD + 1)], pf[rt][n],
                                                                                acc[rt][d], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        ok = next_ok;
        __syncthreads();
    }

    if (HALVES == 2) {
        auto& join = sm.join[wave];
        if (half == 1) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const float u = unit_of(rt);
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    join.acc[rt][d][lane] = make_float4(acc[rt][d][0] * u, acc[rt][d][1] * u, acc[rt][d][2] * u,
                                                        acc[rt][d][3] * u);
                join.ml[rt][lane] = make_float2(m[rt], l[rt] * u);
            }
        }
        __syncthreads();
        if (half == 1) return;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const float2 ml = join.ml[rt][lane];
            const float mn = fmaxf(m[rt], ml.x), base = mn == -INFINITY ? 0.0f : mn;
            const float f0 = __builtin_amdgcn_exp2f(m[rt] - base) * unit_of(rt), f1 = __builtin_amdgcn_exp2f(ml.x - base);
            l[rt] = l[rt] * f0 + ml.y * f1;
            m[rt] = mn;
#pragma unroll
            for (int d = 0; d < DB; ++d) {
                const float4 v = join.acc[rt][d][lane];
                acc[rt][d] = acc[rt][d] * f0 + f4_t{v.x, v.y, v.z, v.w} * f1;
            }
        }
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int r = (wave * RT + rt) * 16 + col;
        const float lr = groups_sum(l[rt]);
        if (tile.row0 + r >= rows) continue;
        const int64_t qr = q_row_of(a, seq, h, row_of_tile(a, tile, r));
        const float base = m[rt] == -INFINITY ? 0.0f : m[rt];
        const float u = HALVES == 2 ? 1.0f : unit_of(rt);
        if (it.splits > 1) {
            const int64_t at = (item * a.heads + h) * ROWS + r;
#pragma unroll
            for (int d = 0; d < DB; ++d)
                *reinterpret_cast<float4*>(a.part + at * D + 16 * d + 4 * g) =
                    make_float4(acc[rt][d][0] * u, acc[rt][d][1] * u, acc[rt][d][2] * u, acc[rt][d][3] * u);
            if (g == 0) a.ml[at] = make_float2(m[rt], lr * u);
        } else {
            const float f = lr == 0.0f ? 0.0f : 1.0f / lr;
#pragma unroll
            for (int d = 0; d < DB; ++d)
                store4f(a.out, qr * D + 16 * d + 4 * g, a.dtype,
                        make_float4(acc[rt][d][0] * f, acc[rt][d][1] * f, acc[rt][d][2] * f, acc[rt][d][3] * f));
            if (g == 0 && a.lse) a.lse[qr] = lr == 0.0f ? -INFINITY : (base + __builtin_amdgcn_logf(lr * u)) * LN2;
        }
    }
}

template <int D, int WAVES, int HALVES, int RT>
hipError_t tile_w(const Attend& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.items * a.heads)), block(64 * WAVES * HALVES);
    if (a.dtype != DT_BF16)
        Q8K_LAUNCH((attend_tile_kernel<D, WAVES, HALVES, RT, 2, 2>), grid, block, 0, s, a);
    else if (a.rope.table)
        Q8K_LAUNCH((attend_tile_kernel<D, WAVES, HALVES, RT, 2, 1>), grid, block, 0, s, a);
    else
        Q8K_LAUNCH((attend_tile_kernel<D, WAVES, HALVES, RT, 1, 1>), grid, block, 0, s, a);
    return hipGetLastError();
}
template <int D>
hipError_t tile_d(const Attend& a, hipStream_t s) {
    if (a.tile_rows == ATTEND_TILE_FEW) {
        // two pages at a time in tiles that are not split; 256 values' operands fill LDS
        if constexpr (D < 256)
            if (a.target == 0) return tile_w<D, 4, 2, 1>(a, s);
        return tile_w<D, 4, 1, 1>(a, s);
    }
    // heads of 256 values: eight waves of 16 rows (four of 32 do not fit the register file)
    return tile_w<D, D == 256 ? 8 : 4, 1, D == 256 ? 1 : 2>(a, s);
}

}  // namespace

hipError_t launch_attend_tiles(int D, const Attend& a, hipStream_t s) {
    return D == 64 ? tile_d<64>(a, s) : D == 128 ? tile_d<128>(a, s) : tile_d<256>(a, s);
}

}  // namespace q8k
