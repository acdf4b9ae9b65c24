// Attention of few rows over the paged 8-bit cache: decode steps, a few drafted
// tokens, and anything whose rows a key head fill no 128-row tile.
//
// For the rows of one key head (its query heads times the new tokens), over
// the tokens j each row sees:
//   s_j = scale <q, kcode_j> kscale_j,  out = sum_j e^(s_j - m) vscale_j vcode_j / sum_j e^(s_j - m)
// in one pass with a running maximum m.  It is bound by the cache's bytes
// (2 D + 8 a token and head), which go from memory to the registers that the
// matrix instructions read.
#include "attend.h"

namespace q8k {

namespace {

constexpr int WAVES = 4;
constexpr int ROWS = 16;

// Probabilities enter the second product as fp16 pieces of p * vscale / R *
// 2^15, R a power of two at least the largest vscale a wave has met: at most
// 2^15 (fp16 ends at 65504), and what fp16's smallest step then loses of a
// token is 2^-40 of the largest one's share.
constexpr float P_UP = 32768.0f, P_DOWN = 1.0f / 32768.0f;

// One workgroup: 16 rows of one key head over `chunk` pages, wave w taking
// pages w, w + 4, ...  S^T = K Q^T leaves a lane the scores of one row
// (lane % 16) and 16 of a page's 64 tokens, in the layout that P^T has to have
// as the second product's operand (kv_cache.h): nothing moves between lanes
// but the running maximum, and that only where it grew.
// NQ and NP: fp16 pieces of the queries and of the probabilities (f16_pieces).
template <int D, int NQ, int NP>
__global__ __launch_bounds__(64 * WAVES, D == 256 ? 1 : 2) void attend_decode_kernel(Attend a) {
    constexpr int KS = D / 32;  // k steps of the first product
    constexpr int DB = D / 16;  // row blocks of the second
    __shared__ float qs[ROWS][D + 4];
    __shared__ float red[WAVES][ROWS][2];
    __shared__ float acc_s[WAVES][ROWS][D + 4];
    __shared__ float scales[WAVES][2 * KV_PAGE];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    // block -> (row tile, split, sequence, head): tiles of the same pages are a
    // multiple of the units apart
    const int64_t units = (int64_t)a.splits * a.B * a.heads;
    const int tile = (int)(blockIdx.x / units);
    const int64_t u = blockIdx.x % units;
    const int split = (int)(u % a.splits);
    const int h = (int)(u / a.splits % a.heads);
    const int64_t b = u / a.splits / a.heads;
    const Sequence seq = sequence_of(a, b);
    const int rows = seq.nq * a.group;
    if (tile * ROWS >= rows) return;
    const int last_row = min(rows, tile * ROWS + ROWS) - 1;
    const Span lo = span_of(a, seq, tile * ROWS / a.group), hi = span_of(a, seq, last_row / a.group);
    int p0 = lo.first / KV_PAGE, p1 = hi.last >= 0 ? hi.last / KV_PAGE + 1 : 0;
    const int first_page = (p0 / a.chunk + split) * a.chunk;  // splits start at multiples of the chunk
    p0 = max(p0, first_page);
    p1 = min(p1, first_page + a.chunk);
    if (a.splits > 1 && p0 >= p1) return;  // the join reads only splits that some row's span meets

    for (int i = threadIdx.x; i < ROWS * (D / 8); i += 64 * WAVES) {
        const int r = i / (D / 8), row = tile * ROWS + r;
        if (row < rows)
            load_q_item<D>(a, seq, h, row, i % (D / 8), qs[r]);
        else {
            *reinterpret_cast<float4*>(&qs[r][8 * (i % (D / 8))]) = make_float4(0, 0, 0, 0);
            *reinterpret_cast<float4*>(&qs[r][8 * (i % (D / 8)) + 4]) = make_float4(0, 0, 0, 0);
        }
    }
    __syncthreads();
    // Q^T operands: step 2 s + t of lane group g holds values 64 s + 16 g + 8 t + j
    float amax = 0.0f;
#pragma unroll
    for (int s = 0; s < KS / 2; ++s)
#pragma unroll
        for (int c = 0; c < 4; ++c) amax = fmaxf(amax, max4(*reinterpret_cast<const float4*>(&qs[col][64 * s + 16 * g + 4 * c])));
    amax = groups_max(amax);
    const int qe = 12 - exponent_of(amax);  // the row's largest value goes to [2^12, 2^13)
    const float qup = pow2f(qe), unit = score_unit(a, qe);
    h8_t qf[NQ][KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        uint32_t w[4][2];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float2 v = *reinterpret_cast<const float2*>(&qs[col][64 * (s / 2) + 16 * g + 8 * (s & 1) + 2 * c]);
            f16_pieces<NQ>(v.x * qup, v.y * qup, w[c]);
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n)
            qf[n][s] = __builtin_bit_cast(h8_t, make_uint4(w[0][n], w[1][n], w[2][n], w[3][n]));
    }

    const int row = tile * ROWS + col;
    Span span = span_of(a, seq, min(row, rows - 1) / a.group);
    float m = -INFINITY, l = 0.0f, R = pow2f(-100), Rinv = pow2f(100) * P_UP;
    f4_t acc[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d) acc[d] = f4_t{0, 0, 0, 0};
    const int32_t* pages = a.table + b * a.max_pages;
    const int lane_off = col * 64 + g * 16;
    // A page's codes and scales on their way, one page ahead of the arithmetic:
    // the keys' registers are loaded again as soon as the scores are there, the
    // values' as soon as the second product is.
    // Reads go through a buffer descriptor of one record; a page that selects
    // nothing has an empty one, whose reads return zeros and touch no memory.
    uint4 kraw[4][KS / 2], vraw[DB];
    float ksc, vsc;
    bool ok, next_ok;
    const auto record_of = [&](int p, bool& good) {
        const int page = p < p1 ? pages[p] : -1;
        good = page >= 0 && page < a.pages;
        return make_rsrc(a.cache + ((int64_t)(good ? page : 0) * a.heads + h) * kv_record(D), good ? kv_record(D) : 0);
    };
    const auto load_keys = [&](rsrc_t rec) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int s = 0; s < KS / 2; ++s) kraw[q][s] = load16(rec, lane_off + s * 4096 + q * 1024);
        ksc = __builtin_bit_cast(float, load4(rec, 4 * lane + 2 * KV_PAGE * D));
    };
    const auto load_values = [&](rsrc_t rec) {
#pragma unroll
        for (int d = 0; d < DB; ++d) vraw[d] = load16(rec, lane_off + KV_PAGE * D + d * 1024);
        vsc = __builtin_bit_cast(float, load4(rec, 4 * lane + 2 * KV_PAGE * D + 4 * KV_PAGE));
    };
    float* sc = scales[wave];
    {
        const rsrc_t rec = record_of(p0 + wave, ok);
        load_keys(rec);
        load_values(rec);
    }
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
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint4 c = kraw[q][s];
                    const h8_t k0 = codes_f16(c.x, c.y), k1 = codes_f16(c.z, c.w);
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        s4[q] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, qf[n][2 * s], s4[q], 0, 0, 0);
                        s4[q] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, qf[n][2 * s + 1], s4[q], 0, 0, 0);
                    }
                    if (q & 1) __builtin_amdgcn_sched_barrier(0);
                }
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
        float vs[4][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float4 v = *reinterpret_cast<const float4*>(&sc[KV_PAGE + 16 * q + 4 * g]);
            vs[q][0] = v.x, vs[q][1] = v.y, vs[q][2] = v.z, vs[q][3] = v.w;
        }
        // pages that some row sees only in part (what lies in unseen places may
        // be anything, NaN scales included)
        if (!ok || p * KV_PAGE < hi.first || p * KV_PAGE + KV_PAGE - 1 > lo.last) {
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
                const float v = wave_max(vmax);
                Rn = fmaxf(R, pow2f(exponent_of(v) + 1));
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
        }
        const float mb = m == -INFINITY ? 0.0f : m;
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
        for (int d = 0; d < DB; ++d) {
            const h8_t v0 = codes_f16(vraw[d].x, vraw[d].y), v1 = codes_f16(vraw[d].z, vraw[d].w);
#pragma unroll
            for (int n = 0; n < NP; ++n) {
                const h8_t q0 = __builtin_bit_cast(h8_t, make_uint4(pw[n][0][0], pw[n][0][1], pw[n][1][0], pw[n][1][1]));
                const h8_t q1 = __builtin_bit_cast(h8_t, make_uint4(pw[n][2][0], pw[n][2][1], pw[n][3][0], pw[n][3][1]));
                acc[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, q0, acc[d], 0, 0, 0);
                acc[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, q1, acc[d], 0, 0, 0);
            }
            if (d & 1) __builtin_amdgcn_sched_barrier(0);
        }
        load_values(rec);
        __builtin_amdgcn_sched_barrier(0);
        ok = next_ok;
    }

    // join the four waves
    l = groups_sum(l);
    if (g == 0) red[wave][col][0] = m, red[wave][col][1] = l;
    __syncthreads();
    float mt = red[0][col][0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) mt = fmaxf(mt, red[w][col][0]);
    const float base = mt == -INFINITY ? 0.0f : mt;
    const float f = __builtin_amdgcn_exp2f(m - base) * R * P_DOWN;
#pragma unroll
    for (int d = 0; d < DB; ++d)
        *reinterpret_cast<float4*>(&acc_s[wave][col][16 * d + 4 * g]) =
            make_float4(acc[d][0] * f, acc[d][1] * f, acc[d][2] * f, acc[d][3] * f);
    __syncthreads();
    for (int i = threadIdx.x; i < ROWS * (D / 4); i += 64 * WAVES) {
        const int r = i / (D / 4), c = 4 * (i % (D / 4));
        if (tile * ROWS + r >= rows) break;
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
        const int64_t qr = q_row_of(a, seq, h, tile * ROWS + r);
        if (a.splits > 1) {
            const int64_t at = (int64_t)split * a.Tq * a.q_heads + qr;
            *reinterpret_cast<float4*>(a.part + at * D + c) = o;
            if (c == 0) a.ml[at] = make_float2(mr, lr);
        } else {
            const float inv = lr == 0.0f ? 0.0f : 1.0f / lr;
            store4f(a.out, qr * D + c, a.dtype, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
            if (c == 0 && a.lse) a.lse[qr] = lr == 0.0f ? -INFINITY : (br + __builtin_amdgcn_logf(lr)) * LN2;
        }
    }
}

// Joins the splits of each row, in their order.  One workgroup a row, four
// values a lane: wave w adds splits w, w + 4, ... and the waves' sums are
// added in their order.
template <int D>
__global__ __launch_bounds__(256) void attend_join_kernel(Attend a) {
    constexpr int L = D / 4;        // lanes a split
    constexpr int N = 256 / L;      // splits at a time
    __shared__ float4 o_s[N][L];
    __shared__ float2 ml_s[N];
    const int64_t per = a.max_q * a.group;  // rows a head, at most
    const int64_t bh = blockIdx.x / per;
    const int row = (int)(blockIdx.x % per), h = (int)(bh % a.heads);
    const Sequence seq = sequence_of(a, bh / a.heads);
    if (row >= seq.nq * a.group) return;
    const Span span = span_of(a, seq, row / a.group);
    const int c = 4 * (threadIdx.x % L), n = threadIdx.x / L;
    const int64_t qr = q_row_of(a, seq, h, row), rows = a.Tq * a.q_heads;
    // the splits that the row's span meets, counted from its tile's first
    const int base_split = span_of(a, seq, row / a.tile_rows * a.tile_rows / a.group).first / KV_PAGE / a.chunk;
    const int s0 = span.first / KV_PAGE / a.chunk - base_split;
    const int s1 = span.last >= 0 ? span.last / KV_PAGE / a.chunk + 1 - base_split : s0;
    float m = -INFINITY, l = 0.0f;
    float4 o = make_float4(0, 0, 0, 0);
    for (int s = s0 + n; s < s1; s += N) {
        const int64_t at = s * rows + qr;
        const float2 ml = a.ml[at];
        const float4 v = *reinterpret_cast<const float4*>(a.part + at * D + c);
        const float mn = fmaxf(m, ml.x), base = mn == -INFINITY ? 0.0f : mn;
        const float x = __builtin_amdgcn_exp2f(m - base), y = __builtin_amdgcn_exp2f(ml.x - base);
        l = l * x + ml.y * y;
        o.x = o.x * x + v.x * y, o.y = o.y * x + v.y * y, o.z = o.z * x + v.z * y, o.w = o.w * x + v.w * y;
        m = mn;
    }
    o_s[n][threadIdx.x % L] = o;
    if (c == 0) ml_s[n] = make_float2(m, l);
    __syncthreads();
    if (n != 0) return;
    float mt = ml_s[0].x;
#pragma unroll
    for (int i = 1; i < N; ++i) mt = fmaxf(mt, ml_s[i].x);
    const float base = mt == -INFINITY ? 0.0f : mt;
    l = 0.0f;
    o = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float y = __builtin_amdgcn_exp2f(ml_s[i].x - base);
        const float4 v = o_s[i][threadIdx.x];
        l += ml_s[i].y * y;
        o.x += v.x * y, o.y += v.y * y, o.z += v.z * y, o.w += v.w * y;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    store4f(a.out, qr * D + c, a.dtype, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    if (c == 0 && a.lse) a.lse[qr] = l == 0.0f ? -INFINITY : (base + __builtin_amdgcn_logf(l)) * LN2;
}

template <int D, int NQ, int NP>
hipError_t decode_n(const Attend& a, hipStream_t s) {
    const int64_t tiles = (a.max_q * a.group + ROWS - 1) / ROWS;
    Q8K_LAUNCH((attend_decode_kernel<D, NQ, NP>), dim3((unsigned)(tiles * a.splits * a.B * a.heads)), dim3(64 * WAVES), 0, s,
               a);
    return hipGetLastError();
}
template <int D>
hipError_t decode_d(const Attend& a, hipStream_t s) {
    if (a.dtype != DT_BF16) return decode_n<D, 2, 2>(a, s);
    return a.rope.table ? decode_n<D, 2, 1>(a, s) : decode_n<D, 1, 1>(a, s);
}
template <int D>
hipError_t join_d(const Attend& a, hipStream_t s) {
    Q8K_LAUNCH(attend_join_kernel<D>, dim3((unsigned)(a.B * a.heads * a.max_q * a.group)), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

// Which kernel and which splits.  The tile kernel's workgroups fill the device
// once they are two a compute unit; the 16-row kernel's are short and hide
// their ends behind each other.
constexpr int64_t DECODE_WGS = 2048, TILE_WGS = 512;
constexpr int64_t TILE_FROM_ROWS = 33;

AttendPlan attend_plan(int64_t B, int64_t Tq, int64_t max_q, int64_t max_len, int q_heads, int heads, int D,
                       int64_t window) {
    AttendPlan p;
    const int64_t group = q_heads / heads;
    p.tiles = max_q * group >= TILE_FROM_ROWS;
    p.tile_rows = p.tiles ? ATTEND_TILE_ROWS : ROWS;
    const int64_t target = p.tiles ? TILE_WGS : DECODE_WGS, least = p.tiles ? 2 : WAVES;
    const int64_t tiles = (max_q * group + p.tile_rows - 1) / p.tile_rows;
    const int64_t pages = (max_len + KV_PAGE - 1) / KV_PAGE, units = tiles * B * heads;
    const auto chunk_of = [&](int64_t live) {
        const int64_t c = (units * live + target - 1) / target;
        return c < least ? least : (c + least - 1) / least * least;
    };
    // the whole sequence; a window changes the chunk, never to more splits
    int64_t chunk = chunk_of(pages), splits = (pages + chunk - 1) / chunk;
    if (splits > 1 && window > 0) {
        // pages that a tile's rows see: at most the window and the tile's own tokens, from anywhere in a page
        const int64_t most = p.tile_rows / group + 2, tokens = max_q < most ? max_q : most;
        const int64_t live = (window + tokens + KV_PAGE - 2) / KV_PAGE + 1;
        if (live < pages) {
            chunk = chunk_of(live);
            while ((live + chunk - 2) / chunk + 1 > splits) chunk += least;
            splits = (live + chunk - 2) / chunk + 1;
        }
    }
    if (splits < 1) splits = 1;
    if (splits == 1) chunk = pages > 0 ? pages : 1;
    p.chunk = (int)chunk;
    p.splits = (int)splits;
    p.ws_bytes = splits > 1 ? align256((size_t)splits * Tq * q_heads * D * 4) + (size_t)splits * Tq * q_heads * 8 : 0;
    return p;
}

hipError_t launch_attend(int D, const AttendPlan& p, Attend a, void* ws, hipStream_t s) {
    a.splits = p.splits;
    a.chunk = p.chunk;
    a.tile_rows = p.tile_rows;
    a.part = static_cast<float*>(ws);
    a.ml = p.splits > 1 ? reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) +
                                                    align256((size_t)p.splits * a.Tq * a.q_heads * D * 4))
                        : nullptr;
    const hipError_t e = p.tiles     ? launch_attend_tiles(D, a, s)
                         : D == 64   ? decode_d<64>(a, s)
                         : D == 128  ? decode_d<128>(a, s)
                                     : decode_d<256>(a, s);
    if (e != hipSuccess || p.splits == 1) return e;
    return D == 64 ? join_d<64>(a, s) : D == 128 ? join_d<128>(a, s) : join_d<256>(a, s);
}

}  // namespace q8k
