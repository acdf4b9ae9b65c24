// Attention of few rows over the paged cache of 8 or 4 bits: decode steps, a few drafted
// tokens, and prompts too short to fill the device with tiles of 64 rows; the
// join of chunks; and the choice between the kernels (attend_plan).
//
// For the rows of one key head (its query heads times the new tokens), over
// the tokens j each row sees:
//   s_j = scale <q, kcode_j> kscale_j,  out = sum_j e^(s_j - m) vscale_j vcode_j / sum_j e^(s_j - m)
// in one pass with a running maximum m.  It is bound by the cache's bytes
// (2 D + 8 a token and head), which go from memory to the registers that the
// matrix instructions read: 8 x 65537 tokens of 8 heads of 128 in 171 us, 6.4
// TB/s (a streaming read of as many bytes reaches 6.7), 16 of up to 8191 in 37.9,
// 4.4 TB/s, 5 us of it the join; from the 4-bit cache 103 us (5.9 TB/s, near what its
// vector instructions take) and 30.  Short sequences are bound by the chain of loads
// before the first product and by what one compute unit draws: 513 tokens 8.8 us.
#include "attend.h"

namespace q8k {

namespace {

constexpr int ROWS = 16;

__device__ __forceinline__ h2_t h2(uint32_t w) { return __builtin_bit_cast(h2_t, w); }
__device__ __forceinline__ uint2 pair_of(h2_t a, h2_t b) {
    return make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
}

// Probabilities enter the second product as fp16 pieces of p * vscale / R *
// 2^15, R a power of two at least the largest vscale that the row has seen in
// this wave: at most 2^15 (fp16 ends at 65504), and what fp16's smallest step
// then loses of a token is 2^-40 of the largest one's share.  R is the row's own
// (its accumulators lie in the lanes that hold it): what other rows of the tile
// see, of whatever size, infinite or NaN, does not touch it.
constexpr float P_UP = 32768.0f, P_DOWN = 1.0f / 32768.0f;

// A product's steps go round four accumulators, so that no instruction waits
// for the one before it (1024 tokens: 13.1 us, 14.0 one chain after the other).
// One workgroup: 16 rows of one key head over `chunk` pages, wave w taking
// pages w, w + WAVES, ...  S^T = K Q^T leaves a lane the scores of one row
// (lane % 16) and 16 of a page's 64 tokens, in the layout that P^T has to have
// as the second product's operand (kv_cache.h): nothing moves between lanes
// but the running maximum, and that only where it grew.
// Of SLICES workgroups each makes its part of the row's values, the scores all of them.
// NQ and NP: fp16 pieces of the queries and of the probabilities (f16_pieces).
template <int D, int BITS, int WAVES, int SLICES, int NQ, int NP>
__global__ __launch_bounds__(64 * WAVES, D == 256 ? 1 : 2) void attend_decode_kernel(Attend a) {
    constexpr int KS = D / 32;  // k steps of the first product
    constexpr int DV = D / SLICES;  // values of the result
    constexpr int DB = DV / 16;     // row blocks of the second product
    constexpr int VB = DB < 4 ? DB : 4;  // of them, by turns
    __shared__ float qs[ROWS][D + 4];
    __shared__ float red[WAVES][ROWS][2];
    __shared__ float acc_s[WAVES][ROWS][DV + 4];
    __shared__ float scales[WAVES][2 * KV_PAGE];
    // of a page's values, for each word of codes two pairs; and what comes off (kv4_cache.h)
    __shared__ __attribute__((aligned(16))) uint2 factors[WAVES][3][BITS == 4 ? DV / 2 : 2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int h = (int)(blockIdx.x % a.heads);
    const int64_t item_slice = blockIdx.x / a.heads;
    const int64_t item = SLICES == 1 ? item_slice : item_slice % a.items;
    const int slice = SLICES == 1 ? 0 : (int)(item_slice / a.items);
    Item it;
    if (!item_of(a, item, it)) return;
    const Sequence seq = it.seq;
    const Tile tile = item_tile(a, seq, it.tile);
    if (tile.row0 >= tile.rows) return;
    const int p0 = uni(tile.p0 + it.split * it.c), p1 = uni(min(tile.p1, p0 + it.c));
    if (it.splits > 1 && p0 >= p1) return;  // the join reads only chunks that some row's span meets

    // the queries and the first page set out together
    constexpr int NI = (ROWS * (D / 8) + 64 * WAVES - 1) / (64 * WAVES);
    QueryItem qi[NI];
#pragma unroll
    for (int n = 0; n < NI; ++n) {
        const int i = threadIdx.x + 64 * WAVES * n, r = i / (D / 8);
        if (i < ROWS * (D / 8) && tile.row0 + r < tile.rows)
            fetch_q<D>(a, seq, h, row_of_tile(a, tile, r), i % (D / 8), qi[n]);
    }
    const Widen masks;
    const int32_t* pages = a.table + it.b * a.max_pages;
    const int lane_off = col * 64 + g * 16;
    // A page's codes and scales on their way, one page ahead of the arithmetic:
    // the keys' registers are loaded again as soon as the scores are there, the
    // values' as soon as the second product is.
    // The codes are read once, which the loads say (non-temporal: 8 x 65537
    // tokens at 6.1 TB/s and 5.4 without, when this was chosen; 6.4 now).
    // Reads go through a buffer descriptor of one record; a page that selects
    // nothing has an empty one, whose reads return zeros and touch no memory.
    // 4 bits: KB blocks of two pieces of the keys, one of two row blocks of the values; the
    // factors of a lane's pieces, and those of the values, a word or two a lane, which become
    // pairs with what comes off once for the wave, by LDS (8 x 65537 tokens 101 us; by every
    // lane for itself 120, the pairs alone by LDS 104).
    constexpr int KB = D / 32, VF = DV / 128 < 1 ? 1 : DV / 128;
    uint4 kraw[4][KS / 2], vraw[DB];
    uint4 kraw4[KB], vraw4[DB / 2];
    uint32_t kfac[KB / 2], vfac[VF];
    float ksc, vsc;
    bool ok, next_ok;
    const auto record_of = [&](int p, bool& good) {
        const int page = __builtin_amdgcn_readfirstlane(p < p1 ? pages[p] : -1);
        good = page >= 0 && page < a.pages;
        constexpr int bytes = kv_record_of(BITS, D);
        return make_rsrc(a.cache + ((int64_t)(good ? page : 0) * a.heads + h) * bytes, good ? bytes : 0);
    };
    constexpr int SCALES = kv_record_of(BITS, D) - 8 * KV_PAGE;
    const auto load_keys = [&](rsrc_t rec) {
        if constexpr (BITS == 8) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int s = 0; s < KS / 2; ++s) kraw[q][s] = load16_nt(rec, lane_off + s * 4096 + q * 1024);
        } else {
#pragma unroll
            for (int i = 0; i < KB; ++i) kraw4[i] = load16_nt(rec, lane_off + i * 1024);
            load_words<KB / 2>(rec, KV4_KF(D) + (col * 2 + (g >> 1)) * (D / 16), kfac);
        }
        ksc = __builtin_bit_cast(float, load4(rec, 4 * lane + SCALES));
    };
    const auto load_values = [&](rsrc_t rec) {
        if constexpr (BITS == 8) {
#pragma unroll
            for (int d = 0; d < DB; ++d) vraw[d] = load16_nt(rec, lane_off + KV_PAGE * D + (slice * DB + d) * 1024);
        } else {
#pragma unroll
            for (int e = 0; e < DB / 2; ++e) vraw4[e] = load16_nt(rec, lane_off + KV4_V(D) + (slice * (DB / 2) + e) * 1024);
            load_words<VF>(rec, KV4_VF(D) + slice * 2 * DV + 4 * VF * (lane % (DV / 2 / VF)), vfac);
        }
        vsc = __builtin_bit_cast(float, load4(rec, 4 * lane + SCALES + 4 * KV_PAGE));
    };
    float* sc = scales[wave];
    {
        const rsrc_t rec = record_of(p0 + wave, ok);
        load_keys(rec);
        load_values(rec);
    }
#pragma unroll
    for (int n = 0; n < NI; ++n) {
        const int i = threadIdx.x + 64 * WAVES * n, r = i / (D / 8), q = i % (D / 8);
        if (i >= ROWS * (D / 8)) continue;
        if (tile.row0 + r < tile.rows) {
            fetch_turn(a, q, qi[n]);
            put_q(a, q, qi[n], qs[r]);
        } else {
            *reinterpret_cast<float4*>(&qs[r][8 * q]) = make_float4(0, 0, 0, 0);
            *reinterpret_cast<float4*>(&qs[r][8 * q + 4]) = make_float4(0, 0, 0, 0);
        }
    }
    __syncthreads();
    h8_t qf[NQ][KS];
    const float unit = query_operand<D, NQ>(a, qs[col], g, qf);
    const Span span = span_of(a, seq, row_of_tile(a, tile, min(col, tile.rows - 1 - tile.row0)).tok);
    float m = -INFINITY, l = 0.0f, R = pow2f(-100), Rinv = pow2f(100) * P_UP;
    bool far = false;  // some row's m is: is_far
    f4_t acc[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d) acc[d] = f4_t{0, 0, 0, 0};
    for (int p = p0 + wave; p < p1; p += WAVES) {
        const rsrc_t rec = record_of(p + WAVES, next_ok);
        sc[lane] = ksc;
        float t[4][4];
        {
            f4_t s4[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) s4[q] = f4_t{0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < KS / 2; ++s) {
                h8_t kf[4][2];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if constexpr (BITS == 8) {
                        const uint4 c = kraw[q][s];
                        kf[q][0] = codes_f16(c.x, c.y);
                        kf[q][1] = codes_f16(c.z, c.w);
                    } else {
                        const int e = q * (D / 64) + s;
                        const uint4 c = kraw4[e >> 1];
                        const Factors f = kv4_key_factors(kfac[e >> 2] >> (8 * (e & 3)) & 255u);
                        kf[q][0] = kv4_widen_keys(masks, e & 1 ? c.z : c.x, f);
                        kf[q][1] = kv4_widen_keys(masks, e & 1 ? c.w : c.y, f);
                    }
                }
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            s4[q] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[q][t], qf[n][2 * s + t], s4[q], 0, 0, 0);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 ks = *reinterpret_cast<const float4*>(&sc[16 * q + 4 * g]);
                t[q][0] = s4[q][0] * ks.x;
                t[q][1] = s4[q][1] * ks.y;
                t[q][2] = s4[q][2] * ks.z;
                t[q][3] = s4[q][3] * ks.w;
            }
        }
        load_keys(rec);
        __builtin_amdgcn_sched_barrier(0);
        sc[KV_PAGE + lane] = vsc;
        if constexpr (BITS == 4) {
#pragma unroll
            for (int i = 0; i < VF; ++i) {
                const FactorPairs f = kv4_value_factors(vfac[i]);
                const int at = VF * (lane % (DV / 2 / VF)) + i;
                factors[wave][0][at] = pair_of(f.first.f, f.second.f);
                factors[wave][1][at] = pair_of(f.first.low, f.second.low);
                factors[wave][2][at] = pair_of(f.first.high, f.second.high);
            }
        }
        float vs[4][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float4 v = *reinterpret_cast<const float4*>(&sc[KV_PAGE + 16 * q + 4 * g]);
            vs[q][0] = v.x, vs[q][1] = v.y, vs[q][2] = v.z, vs[q][3] = v.w;
        }
        // pages that some row sees only in part (what lies in unseen places may
        // be anything, NaN scales included)
        if (!ok || p * KV_PAGE < tile.hi.first || p * KV_PAGE + KV_PAGE - 1 > tile.lo.last) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = p * KV_PAGE + 16 * q + 4 * g + i;
                    const bool seen = ok && j >= span.first && j <= span.last;
                    t[q][i] = seen ? t[q][i] : -INFINITY;
                    vs[q][i] = seen ? vs[q][i] : 0.0f;
                }
        }
        float tmax = t[0][0], vmax = vs[0][0];
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) tmax = fmaxf(tmax, t[q][i]), vmax = fmaxf(vmax, vs[q][i]);
        tmax *= unit;
        if (__any(tmax > m || vmax > R)) {
            const float mn = fmaxf(m, groups_max(tmax));
            float Rn = R;
            if (__any(vmax > R)) {
                const float v = groups_max(vmax);
                Rn = v > R ? pow2f(exponent_of(v) + 1) : R;
            }
            const float base = mn == -INFINITY ? 0.0f : mn;
            const float down = __builtin_amdgcn_exp2f(m - base);
            l *= down;
            const float both = down * (R / Rn);
#pragma unroll
            for (int d = 0; d < DB; ++d) acc[d] *= both;
            m = mn;
            R = Rn;
            Rinv = P_UP / Rn;
            far |= __any(is_far(mn));
        }
        float mb = m == -INFINITY ? 0.0f : m;
        if (far && is_far(m)) {
            const float inv = 1.0f / unit;
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) t[q][i] = far_score(t[q][i], unit, inv, m);
            mb = 0.0f;
        }
        uint32_t pw[NP][4][2];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(t[q][i], unit, -mb));
                l += e[i];
                e[i] *= vs[q][i] * Rinv;
            }
            uint32_t w0[2], w1[2];
            f16_pieces<NP>(e[0], e[1], w0);
            f16_pieces<NP>(e[2], e[3], w1);
#pragma unroll
            for (int n = 0; n < NP; ++n) pw[n][q][0] = w0[n], pw[n][q][1] = w1[n];
        }
#pragma unroll
        for (int d0 = 0; d0 < DB; d0 += VB) {
            h8_t vf[VB][2];
#pragma unroll
            for (int d = 0; d < VB; ++d) {
                if constexpr (BITS == 8) {
                    vf[d][0] = codes_f16(vraw[d0 + d].x, vraw[d0 + d].y);
                    vf[d][1] = codes_f16(vraw[d0 + d].z, vraw[d0 + d].w);
                } else if (d % 2 == 0) {
                    const uint4 c = vraw4[(d0 + d) / 2];
                    const int at = (d0 + d) * 8 + 4 * g;
                    FactorPairs f[4];
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        const uint4 x = *reinterpret_cast<const uint4*>(&factors[wave][0][at + i]);
                        const uint4 y = *reinterpret_cast<const uint4*>(&factors[wave][1][at + i]);
                        const uint4 z = *reinterpret_cast<const uint4*>(&factors[wave][2][at + i]);
                        f[i] = {{h2(x.x), h2(y.x), h2(z.x)}, {h2(x.y), h2(y.y), h2(z.y)}};
                        f[i + 1] = {{h2(x.z), h2(y.z), h2(z.z)}, {h2(x.w), h2(y.w), h2(z.w)}};
                    }
                    kv4_widen_values(masks, c.x, c.y, f[0], f[1], vf[d][0], vf[d + 1][0]);
                    kv4_widen_values(masks, c.z, c.w, f[2], f[3], vf[d][1], vf[d + 1][1]);
                }
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int n = 0; n < NP; ++n) {
                    const h8_t pf = __builtin_bit_cast(h8_t, make_uint4(pw[n][2 * t][0], pw[n][2 * t][1],
                                                                        pw[n][2 * t + 1][0], pw[n][2 * t + 1][1]));
#pragma unroll
                    for (int d = 0; d < VB; ++d)
                        acc[d0 + d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[d][t], pf, acc[d0 + d], 0, 0, 0);
                }
        }
        load_values(rec);
        __builtin_amdgcn_sched_barrier(0);
        ok = next_ok;
    }

    // join the waves
    l = groups_sum(l);
    if (g == 0) red[wave][col][0] = m, red[wave][col][1] = l;
    __syncthreads();
    float mt = red[0][col][0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) mt = fmaxf(mt, red[w][col][0]);
    const float base = mt == -INFINITY ? 0.0f : mt;
    const float f = __builtin_amdgcn_exp2f(m - base) * R * P_DOWN;
    if (tile.row0 + col < tile.rows)
#pragma unroll
        for (int d = 0; d < DB; ++d)
            *reinterpret_cast<float4*>(&acc_s[wave][col][16 * d + 4 * g]) =
                make_float4(acc[d][0] * f, acc[d][1] * f, acc[d][2] * f, acc[d][3] * f);
    __syncthreads();
    for (int i = threadIdx.x; i < ROWS * (DV / 4); i += 64 * WAVES) {
        const int r = i / (DV / 4), c = 4 * (i % (DV / 4));
        if (tile.row0 + r >= tile.rows) break;
        float mr = red[0][r][0];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) mr = fmaxf(mr, red[w][r][0]);
        const float br = mr == -INFINITY ? 0.0f : mr;
        float lr = 0.0f;
        float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            lr += red[w][r][1] * __builtin_amdgcn_exp2f(red[w][r][0] - br);
            const float4 v = *reinterpret_cast<const float4*>(&acc_s[w][r][c]);
            o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
        }
        const int64_t qr = q_row_of(a, seq, h, row_of_tile(a, tile, r));
        if (it.splits > 1) {
            const int64_t at = (item * a.heads + h) * ROWS + r;
            *reinterpret_cast<float4*>(a.part + at * D + slice * DV + c) = o;
            if (c == 0 && slice == 0) a.ml[at] = make_float2(mr, lr);
        } else {
            const float inv = lr == 0.0f ? 0.0f : 1.0f / lr;
            store4f(a.out, qr * D + slice * DV + c, a.dtype, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
            if (c == 0 && slice == 0 && a.lse) a.lse[qr] = lr == 0.0f ? -INFINITY : (br + __builtin_amdgcn_logf(lr)) * LN2;
        }
    }
}

// Joins the chunks of each row, always in the same order.  W waves a row (four
// where rows are few and chunks many, one where it is the other way round):
// wave w adds chunks w, w + W, ...  Lanes first take a chunk each (its maximum
// and sum), then D/64 values of every chunk's result.  5 us for 512 rows of some
// five chunks (1.3 MB): a launch and three dependent loads.
template <int D, int W>
__global__ __launch_bounds__(256) void attend_join_kernel(Attend a) {
    constexpr int N = D / 64;
    __shared__ float o_s[4][D];
    __shared__ float2 ml_s[4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t per = (int64_t)a.max_q * a.group;  // rows a sequence and head, at most
    const int64_t id = W == 4 ? blockIdx.x : (int64_t)blockIdx.x * 4 + wave;
    const int64_t bh = id / per;
    if (bh >= a.B * a.heads) return;
    const int row = (int)(id % per), h = (int)(bh % a.heads);
    const Item it = items_of(a, bh / a.heads);
    if (it.splits == 1) return;
    const Sequence seq = it.seq;
    if (row >= seq.nq * a.group) return;
    const int ti = row / a.tile_rows, r = row % a.tile_rows;
    const Tile tile = item_tile(a, seq, ti);
    const TileRow tr = row_of_tile(a, tile, r);
    const Span span = span_of(a, seq, tr.tok);
    const int s0 = uni((span.first / KV_PAGE - tile.p0) / it.c);
    const int s1 = uni(span.last >= 0 ? (span.last / KV_PAGE - tile.p0) / it.c + 1 : s0);
    const int64_t first = it.first + (int64_t)ti * it.splits, step = (int64_t)a.heads * a.tile_rows;
    float m = -INFINITY, l = 0.0f, o[N];
#pragma unroll
    for (int n = 0; n < N; ++n) o[n] = 0.0f;
    const int w = W == 4 ? wave : 0;
    for (int s = s0 + w; s < s1; s += 64 * W) {
        const int64_t at = ((first + s) * a.heads + h) * a.tile_rows + r;
        const int count = min(64, (s1 - s + W - 1) / W);
        float2 ml = make_float2(-INFINITY, 0.0f);
        if (lane < count) ml = a.ml[at + lane * W * step];
        const float* part = a.part + at * D + N * lane;
        const float mn = fmaxf(m, wave_max_dpp(ml.x)), base = mn == -INFINITY ? 0.0f : mn;
        const float down = __builtin_amdgcn_exp2f(m - base), y = __builtin_amdgcn_exp2f(ml.x - base);
        l = l * down + wave_sum_dpp(ml.y * y);
#pragma unroll
        for (int n = 0; n < N; ++n) o[n] *= down;
#pragma unroll 8
        for (int i = 0; i < count; ++i) {
            const float f = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, y), i));
            const float* x = part + i * W * step * D;
#pragma unroll
            for (int n = 0; n < N; ++n) o[n] += x[n] * f;
        }
        m = mn;
    }
    if (W == 4) {
#pragma unroll
        for (int n = 0; n < N; ++n) o_s[wave][N * lane + n] = o[n];
        if (lane == 0) ml_s[wave] = make_float2(m, l);
        __syncthreads();
        if (wave != 0) return;
        m = fmaxf(fmaxf(ml_s[0].x, ml_s[1].x), fmaxf(ml_s[2].x, ml_s[3].x));
        const float base = m == -INFINITY ? 0.0f : m;
        l = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) o[n] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float y = __builtin_amdgcn_exp2f(ml_s[i].x - base);
            l += ml_s[i].y * y;
#pragma unroll
            for (int n = 0; n < N; ++n) o[n] += o_s[i][N * lane + n] * y;
        }
    }
    const int64_t qr = q_row_of(a, seq, h, tr);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l, base = m == -INFINITY ? 0.0f : m;
    const int64_t to = qr * D + N * lane;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const float v = o[n] * inv;
        if (a.dtype == DT_F32)
            static_cast<float*>(a.out)[to + n] = v;
        else
            static_cast<uint16_t*>(a.out)[to + n] = (uint16_t)(a.dtype == DT_BF16 ? to_bf16(v) : to_f16(v));
    }
    if (lane == 0 && a.lse) a.lse[qr] = l == 0.0f ? -INFINITY : (base + __builtin_amdgcn_logf(l)) * LN2;
}

template <int D, int BITS, int WAVES, int SLICES, int NQ, int NP>
hipError_t decode_n(const Attend& a, hipStream_t s) {
    Q8K_LAUNCH((attend_decode_kernel<D, BITS, WAVES, SLICES, NQ, NP>), dim3((unsigned)(a.items * a.heads * SLICES)),
               dim3(64 * WAVES), 0, s, a);
    return hipGetLastError();
}
template <int D, int BITS, int WAVES, int SLICES>
hipError_t decode_w(const Attend& a, hipStream_t s) {
    if (a.dtype != DT_BF16) return decode_n<D, BITS, WAVES, SLICES, 2, 2>(a, s);
    return a.rope.table ? decode_n<D, BITS, WAVES, SLICES, 2, 1>(a, s) : decode_n<D, BITS, WAVES, SLICES, 1, 1>(a, s);
}
template <int D, int BITS>
hipError_t decode_d(const Attend& a, const AttendPlan& p, hipStream_t s) {
    // eight waves' accumulators of 256 values would not fit; 64 values by four
    // are one row block each
    if constexpr (D < 256)
        if (p.waves == 8) return decode_w<D, BITS, 8, 1>(a, s);
    if constexpr (D > 64)
        if (p.slices == 4) return decode_w<D, BITS, 4, 4>(a, s);
    return p.slices == 2 ? decode_w<D, BITS, 4, 2>(a, s) : decode_w<D, BITS, 4, 1>(a, s);
}
template <int BITS>
hipError_t decode_of(int D, const Attend& a, const AttendPlan& p, hipStream_t s) {
    return D == 64 ? decode_d<64, BITS>(a, p, s) : D == 128 ? decode_d<128, BITS>(a, p, s) : decode_d<256, BITS>(a, p, s);
}
template <int D>
hipError_t join_d(const Attend& a, bool tiles, hipStream_t s) {
    const int64_t rows = a.B * a.heads * a.max_q * a.group;
    if (tiles)
        Q8K_LAUNCH((attend_join_kernel<D, 1>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, s, a);
    else
        Q8K_LAUNCH((attend_join_kernel<D, 4>), dim3((unsigned)rows), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

// Which kernel and how many work items.  Times are of one key/value cache with
// 8 key heads of 128 and 32 query heads unless it says otherwise.
//
// Chunks are of a size for TARGET_WGS workgroups, two a compute unit: more and
// smaller ones measured slower (each has its queries to bring and its results
// to join), fewer leave units idle where lengths differ.  A call that has
// several times as many tiles is not split, nor is one of more sequences than
// the workgroups care to look through: of lengths spread from a tenth to the
// longest (8 query heads over one), 64 of up to 8191 tokens take 26 us in chunks
// and 48 whole, 256 of up to 4000 take 50 and 38, 512 of them 113 and 64, of up to
// 16000 272 and 216.  What the limit gives away is a sequence far longer than the
// rest: 65537 tokens among 255 of up to 2000 take 50 us, among 256 of them, whole,
// 412 (in chunks 52).
constexpr int64_t TARGET_WGS = 512;
// Heads of 256 values in 4 bits: a compute unit takes one workgroup of them at a time, so
// that 512 come in two turns (32 query heads over 8, bf16: 16 x 2000 tokens 25.4 us, with 512
// 32.7, with 384 36.3; 16 x 8191 57.4, 66.2 and 78.2; 2 x 60000 55.2, 66.5 and 78.2).
constexpr int64_t TARGET_WGS_256 = 256;
constexpr int64_t SPLIT_MAX_BATCH = 256;
// A chunk has at least this many pages (4096 tokens of one sequence: 15.6 us;
// with 16 pages 17.2, with 4 15.3, but 16000 tokens then 22.6 and not 20.8).
constexpr int LEAST_PAGES = 8;
// The join costs a launch: up to UNSPLIT_PAGES pages (UNSPLIT_PAGES_256 of the
// larger records) a tile is one workgroup's (16 x 1500 tokens: 16.3 us, in
// chunks 19.4; 1 x 2000 15.3 and 14.6, 1 x 3000 19.7 and 15.2; 256 values,
// 1 x 1000: 14.5 and 16.9, 1 x 2000: 21.1 and 17.6; tiles of 64 rows, 1000 new
// tokens over 2000: 97 and 107).
constexpr int64_t UNSPLIT_PAGES = 32, UNSPLIT_PAGES_256 = 24;
// A compute unit alone draws no more than some 50 GB/s of codes it has not met, so
// few workgroups share a tile's values between them, each with all of the keys:
// four up to 64 workgroups, two up to 128 (513 tokens: 9.4 us, by two 9.9, alone
// 10.8; 256 values: 13.3, 15.1, 18.4; 16 x 2000 tokens by two 19.2, alone 22.2;
// 32 x 2000 by two 29.5, alone 24.6).
constexpr int64_t FOUR_SLICES_TO = 64, TWO_SLICES_TO = 128;
// Where one workgroup a compute unit is all there is, it has eight waves if there are
// pages for them (12 sequences of 1000 tokens, five tokens each: 12.3 us, of
// four waves 13.6; 24 of 500: 13.2 and 11.8, of 640 13.8 and 13.4, of 768 and up
// within 3% of each other; heads of 64 values, 640: 9.9 and 10.2, 832: 11.1 and
// 11.7, 1500: 13.9 and 15.6); where there are more, four (64 x 2000: 36 us, of
// eight 43).
constexpr int64_t EIGHT_WAVES_TO = 256, EIGHT_WAVES_FROM_PAGES = 13;
// Rows of one key head by the sixteen, each 16 with the whole cache before
// them, or by the 64 or 128 that share a page's conversion but leave compute
// units without work where there are few of them, and half a tile where the rows
// are.  Up to SHORT_PAGES pages the sixteens are the faster for up to 48 rows and
// up to SIXTEENS tiles (64 new tokens over 1000, 128 tiles: 12.8 us, by 64 rows
// 29.2; 256 over 256, 512 tiles: 11.8 and 14.5; 384 over 384, 768: 21.3 and
// 18.0; 64 sequences of 500 tokens, 12 new ones each: 40 and 41, 16: 55 and 42);
// over more for up to 96 rows (16 sequences of 8191 tokens, nine new ones each: 67 us
// and 115, 16: 94 and 115, 24: 123 and 122; 64 of 2000, 20 each: 98 and 111) and up to
// SIXTEENS_PAGES pages of all tiles together (32 over 4000, 64 tiles: 24 and
// 39, over 16000 43 and 49, over 65000 133 and 108; 64 over 8000, 128 tiles: 44 and
// 46, over 16000 67 and 66).
constexpr int64_t SHORT_PAGES = 16, SIXTEENS = 512, SIXTEENS_PAGES = 16384;
// 128 rows a tile where they fill the compute units or are cut into enough chunks
// to, else 64 (32 heads over 4, 250 new tokens, over 2500: 44 us, by 128 rows 51;
// over 4000 56 and 55, over 16001 149 and 132; 1000 over 16001: 503 and 435, of
// 256 values 1244 and 729).
constexpr int64_t SMALL_TILES_BELOW = 256, SMALL_TILES_PAGES = 48;

static AttendPlan plan_for(int bits, int64_t B, int64_t max_q, int64_t max_len, int q_heads, int heads, int D,
                           int64_t window) {
    AttendPlan p;
    const int64_t group = q_heads / heads, rows = max_q * group, pages = (max_len + KV_PAGE - 1) / KV_PAGE;
    // what a tile reads at most
    const auto live_of = [&](int64_t tile_rows) {
        const int64_t seen = (window + tile_rows / group + KV_PAGE) / KV_PAGE + 1;
        return window > 0 && seen < pages ? seen : pages;
    };
    const int64_t sixteens = (rows + ROWS - 1) / ROWS * B * heads, few = live_of(ROWS);
    p.tiles = few <= SHORT_PAGES ? rows > 3 * ROWS && sixteens > SIXTEENS
                                 : rows > 6 * ROWS && sixteens > SIXTEENS_PAGES / few;
    p.tile_rows = ROWS;
    if (p.tiles) {
        const int64_t large = (rows + ATTEND_TILE_ROWS - 1) / ATTEND_TILE_ROWS * B * heads;
        p.tile_rows = large < SMALL_TILES_BELOW && few <= SMALL_TILES_PAGES ? ATTEND_TILE_FEW : ATTEND_TILE_ROWS;
    }
    p.tiles_max = (int)((rows + p.tile_rows - 1) / p.tile_rows);
    p.least = LEAST_PAGES;
    const int64_t tiles = B * p.tiles_max, live = live_of(p.tile_rows);
    p.split = live > (D == 256 && !p.tiles ? UNSPLIT_PAGES_256 : UNSPLIT_PAGES) && B <= SPLIT_MAX_BATCH &&
              tiles * heads < (p.tiles ? 1 : 4) * TARGET_WGS;
    const int64_t wgs_wanted = bits == 4 && D == 256 && !p.tiles ? TARGET_WGS_256 : TARGET_WGS;
    p.target = p.split ? (int)((wgs_wanted + heads - 1) / heads) : 0;
    p.items = tiles;
    if (p.split) {
        const int64_t most = tiles * (1 + pages / p.least);
        p.items = tiles + p.target < most ? tiles + p.target : most;
    }
    const int64_t wgs = p.items * heads;
    p.slices = p.tiles ? 1 : wgs <= FOUR_SLICES_TO && D > 64 ? 4 : wgs <= TWO_SLICES_TO ? 2 : 1;
    // finding the longest takes a workgroup up to 1 us (58 sequences of 513 tokens,
    // eight new ones each: 30.6 us, 35.0 ordered; 64 of 8191, 16 each: 287 and 251)
    p.order = !p.split && B > 1 && B <= 64 && (p.tiles || live > UNSPLIT_PAGES);
    p.waves = D < 256 && p.slices == 1 && wgs <= EIGHT_WAVES_TO && !p.split && live >= EIGHT_WAVES_FROM_PAGES ? 8 : 4;
    // (decode_d, tile_d: two halves or eight waves of a tile)
    p.threads = !p.tiles ? 64 * p.waves : (p.tile_rows == ATTEND_TILE_FEW ? D < 256 && !p.split : D == 256) ? 512 : 256;
    p.ws_bytes = 0;
    if (p.split) {
        const int64_t parts = p.items * heads * p.tile_rows;
        p.ws_bytes = align256(parts * D * 4) + parts * 8;
    }
    return p;
}

// Callers size the workspace without a window: a plan that a window changes to
// one of a larger workspace is not taken (either serves any window).
AttendPlan attend_plan(int bits, int64_t B, int64_t max_q, int64_t max_len, int q_heads, int heads, int D, int64_t window) {
    const AttendPlan all = plan_for(bits, B, max_q, max_len, q_heads, heads, D, 0);
    if (window == 0) return all;
    const AttendPlan p = plan_for(bits, B, max_q, max_len, q_heads, heads, D, window);
    return p.ws_bytes > all.ws_bytes ? all : p;
}

hipError_t launch_attend(int bits, int D, const AttendPlan& p, Attend a, void* ws, hipStream_t s) {
    a.tile_rows = p.tile_rows;
    a.tiles_max = p.tiles_max;
    a.least = p.least;
    a.target = p.target;
    a.items = p.items;
    a.order = p.order;
    a.inv_group = 1.0f / (float)a.group;
    a.part = static_cast<float*>(ws);
    if (p.split)
        a.ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + align256(p.items * a.heads * p.tile_rows * D * 4));
    const hipError_t e = p.tiles     ? launch_attend_tiles(bits, D, a, s)
                         : bits == 8 ? decode_of<8>(D, a, p, s)
                                     : decode_of<4>(D, a, p, s);
    if (e != hipSuccess || !p.split) return e;
    return D == 64    ? join_d<64>(a, p.tiles, s)
           : D == 128 ? join_d<128>(a, p.tiles, s)
                      : join_d<256>(a, p.tiles, s);
}

}  // namespace q8k
