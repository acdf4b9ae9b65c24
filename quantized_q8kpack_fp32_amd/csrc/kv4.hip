// Appending to the paged 4-bit key/value cache, and reading it back.
//
// Append, for each token and head: the key turns by its position, then key and
// value each become D codes of 4 bits, D/32 factors and one scale:
//   scale = amax/7,  factor_y = the least 8-bit float >= max|x_y| / amax,
//   code = round(x / (factor_y scale)).
// 4 D or 8 D bytes a token and head in, D + D/16 + 8 out: 8191 tokens of 8 heads of 128,
// bf16, half turned, 45 MB, take 16 us, about 11 of them vector instructions (twelve
// divisions a lane, which the four lanes of a group repeat, and the codes); the read back,
// 43 MB, 11 (3.8 TB/s).  Few tokens are bound by the launch and two chained loads (61
// tokens 3.4 us, the read back 3.9).
#include "kv4_cache.h"
#include "kv_tile.h"
#include "q8k_launch.h"

namespace q8k {

namespace {

// Codes of lanes two apart in a group of four.
__device__ __forceinline__ uint32_t other_half(uint32_t w) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0x4E, 0xF, 0xF, false);  // quad_perm 2,3,0,1
}

// Eight values of a row (D/8 = L lanes) and what their group and row decide.
struct Row4 {
    float scale, inverse;
    uint32_t factor;
};
// Magnitudes compare as whole numbers do: an infinity or a NaN shows in the largest one,
// and no maximum has to quieten its operands.
constexpr uint32_t INF_BITS = 0x7f800000u;
__device__ __forceinline__ uint32_t magnitude(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t most_of(float4 x, float4 y) {
    const uint32_t a = max(max(magnitude(x.x), magnitude(x.y)), magnitude(x.z));
    const uint32_t b = max(max(magnitude(x.w), magnitude(y.x)), magnitude(y.y));
    return max(max(a, b), max(magnitude(y.z), magnitude(y.w)));
}
template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false));
}
// (passes NaN over, as group_max does; leaves 0 in the place of what has code 0: a NaN, and
// an infinity, whose row's scale is infinite)
template <int L>
__device__ __forceinline__ Row4 quantise_row(float4& x, float4& y) {
    float* const v[8] = {&x.x, &x.y, &x.z, &x.w, &y.x, &y.y, &y.z, &y.w};
    uint32_t most = most_of(x, y);
    const bool odd = __any(most >= INF_BITS);
    if (odd) {
#pragma unroll
        for (int i = 0; i < 8; ++i) *v[i] = magnitude(*v[i]) > INF_BITS ? 0.0f : *v[i];
        most = most_of(x, y);
    }
    const uint32_t top = max_dpp<0x4E>(max_dpp<0xB1>(most));  // of the group: quad_perm 1,0,3,2 and 2,3,0,1
    uint32_t all = max_dpp<0x141>(top);                       // row_half_mirror
    if (L >= 16) all = max_dpp<0x128>(all);                   // row_ror:8
    if (L == 32) all = max(all, (uint32_t)__shfl_xor((int)all, 16, WAVE));
    if (odd)
#pragma unroll
        for (int i = 0; i < 8; ++i) *v[i] = magnitude(*v[i]) == INF_BITS ? 0.0f : *v[i];
    const float amax = __builtin_bit_cast(float, all);
    Row4 r;
    r.scale = amax / 7.0f;
    r.factor = kv4_factor(__builtin_bit_cast(float, top) / amax);
    r.inverse = kv4_inverse(r.factor, r.scale);
    return r;
}
// Values that turned half a rotation apart, by way of LDS (the row's lanes are of one
// wave) to where eight consecutive ones lie.
template <int D>
__device__ __forceinline__ void natural_order(float* row_s, int oa, int ob, int item, float4& x, float4& y) {
    *reinterpret_cast<float4*>(row_s + oa) = x;
    *reinterpret_cast<float4*>(row_s + ob) = y;
    __builtin_amdgcn_wave_barrier();
    x = *reinterpret_cast<const float4*>(row_s + 8 * item);
    y = *reinterpret_cast<const float4*>(row_s + 8 * item + 4);
    __builtin_amdgcn_wave_barrier();
}
// Four bytes of a value row: lanes 0 and 1 of a group of four lanes hold its first sixteen
// values, 2 and 3 the others, which lie beside them.  Lane i makes the bytes of values
// 8 (i % 2) + 4 (i / 2) and on of the first sixteen.
__device__ __forceinline__ uint32_t value_bytes(float4 x, float4 y, float inverse, int item) {
    const uint64_t codes = kv4_codes8<0, 8, 16, 24, 32, 40, 48, 56>(x, y, inverse);
    const uint32_t lo = (uint32_t)codes, hi = (uint32_t)(codes >> 32);
    const uint32_t lo2 = other_half(lo), hi2 = other_half(hi);
    return item & 2 ? hi2 | hi << 4 : lo | lo2 << 4;
}

// D/8 lanes a row (a token's key or value of one head), eight consecutive values
// a lane: a key's word, a fourth of a group.  Pairs that turn half a rotation apart go
// through LDS to where their values lie.
template <int D>
__global__ __launch_bounds__(256) void kv4_append_kernel(KvAppend a) {
    constexpr int L = D / 8, ROWS = 256 / L;
    __shared__ float turned[ROWS][D + 4];
    const int item = threadIdx.x % L;
    const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / L;
    if (row >= a.T * 2 * a.heads) return;  // uniform over the row's lanes
    const int64_t t = row / (2 * a.heads);
    const int hv = (int)(row % (2 * a.heads));
    const bool is_v = hv >= a.heads;
    const int h = is_v ? hv - a.heads : hv;
    RopeView r = a.rope;
    if (is_v) r.table = nullptr;
    int oa, ob;
    kv_item(r, item, oa, ob);
    // the slot, the position and the row set out together
    const int slot = a.slots[t], p = a.rope.table ? a.pos[t] : 0;
    const void* src = is_v ? a.v : a.k;
    const int64_t base = t * (is_v ? a.v_stride : a.k_stride) + (int64_t)h * D;
    const uint4 raw_x = load4raw(src, base + oa, a.dtype == DT_F32), raw_y = load4raw(src, base + ob, a.dtype == DT_F32);
    if (slot < 0 || slot >= a.pages * KV_PAGE) return;
    if (a.rope.table && (p < 0 || p >= a.rope.len)) return;  // neither key nor value: the token selects nothing
    const int64_t page = slot / KV_PAGE;
    const int token = slot % KV_PAGE;
    const float* turn = r.table ? r.table + (int64_t)p * r.dim : nullptr;
    float4 x = raw4f(raw_x, a.dtype), y = raw4f(raw_y, a.dtype);
    if (turn && 8 * item < r.dim) {
        kv_turn(r, *reinterpret_cast<const float4*>(turn + 4 * item),
                *reinterpret_cast<const float4*>(turn + r.dim / 2 + 4 * item), x, y);
    }
    if (turn && !r.adjacent) natural_order<D>(turned[threadIdx.x / L], oa, ob, item, x, y);
    const Row4 q = quantise_row<L>(x, y);
    uint8_t* rec = a.cache + (page * a.heads + h) * kv4_record(D);
    const int group = item >> 2;
    if (!is_v) {
        *reinterpret_cast<uint32_t*>(rec + kv4_key_word<D>(token, item)) = kv4_key_codes(x, y, q.inverse);
        if ((item & 3) == 0) rec[kv4_key_factor<D>(token, group)] = (uint8_t)q.factor;
    } else {
        const uint32_t w = value_bytes(x, y, q.inverse, item);
        uint8_t* v = rec + KV4_V(D) + group * 1024 + (8 * (item & 1) + 2 * (item & 2)) * KV_PAGE + kv4_place(token);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e * KV_PAGE] = (uint8_t)(w >> (8 * e));
        if ((item & 3) == 0) rec[KV4_VF(D) + group * KV_PAGE + kv4_place(token)] = (uint8_t)q.factor;
    }
    if (item == 0) reinterpret_cast<float*>(rec + KV4_S(D))[(is_v ? KV_PAGE : 0) + token] = q.scale;
}

// Many tokens: one workgroup takes 32 tokens of one head.  Keys go as above, 32 to 128
// consecutive bytes a token.  The values' bytes meet in LDS: those of four tokens
// that follow each other from a multiple of four on lie side by side in each row of
// places and leave as words, the others' (a run's ends, slots in no order) as bytes.
// Made for each type: where the type was looked at for every value, 19.2 us for 17.0.
template <int D, int DT>
__global__ __launch_bounds__(256) void kv4_append_tile_kernel(KvAppend a) {
    constexpr int L = D / 8, ROWS = 256 / L, N = TILE / ROWS, W = D / 8;  // words of a token's values
    __shared__ float turned[ROWS][D + 4];
    __shared__ uint32_t codes[TILE][W + 1];
    __shared__ int slots[TILE], fours[FOURS];
    const int h = (int)(blockIdx.x % a.heads);
    const int64_t t0 = (int64_t)(blockIdx.x / a.heads) * TILE;
    const int n = (int)(a.T - t0 < TILE ? a.T - t0 : TILE);
    const int item = threadIdx.x % L, group = item >> 2;
    int oa, ob;
    kv_item(a.rope, item, oa, ob);
    // all rows of the tile (the last one's again behind the last)
    uint4 raw[N][4];
    int slot_of[N], pos[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t t = t0 + min(i * ROWS + (int)threadIdx.x / L, n - 1);
        slot_of[i] = a.slots[t];
        pos[i] = a.rope.table ? a.pos[t] : 0;
        const int64_t kb = t * a.k_stride + (int64_t)h * D, vb = t * a.v_stride + (int64_t)h * D;
        raw[i][0] = load4raw(a.k, kb + oa, DT == DT_F32);
        raw[i][1] = load4raw(a.k, kb + ob, DT == DT_F32);
        raw[i][2] = load4raw(a.v, vb + 8 * item, DT == DT_F32);
        raw[i][3] = load4raw(a.v, vb + 8 * item + 4, DT == DT_F32);
    }
    float4 c[N], s[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const bool there = i * ROWS + (int)threadIdx.x / L < n;
        // a token that selects nothing: behind the last, its slot or its position outside
        if (!there || slot_of[i] >= a.pages * KV_PAGE) slot_of[i] = -1;
        if (a.rope.table) {
            if (pos[i] < 0 || pos[i] >= a.rope.len) slot_of[i] = -1;
            if (slot_of[i] >= 0 && 8 * item < a.rope.dim) {
                const float* turn = a.rope.table + (int64_t)pos[i] * a.rope.dim + 4 * item;
                c[i] = *reinterpret_cast<const float4*>(turn);
                s[i] = *reinterpret_cast<const float4*>(turn + a.rope.dim / 2);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int t = i * ROWS + threadIdx.x / L, slot = slot_of[i];
        if (item == 0) slots[t] = slot;
        if (slot < 0) continue;  // uniform over the row's lanes
        uint8_t* rec = a.cache + ((int64_t)(slot / KV_PAGE) * a.heads + h) * kv4_record(D);
        const int token = slot % KV_PAGE;
        float4 x = raw4f(raw[i][0], DT), y = raw4f(raw[i][1], DT);
        float4 u = raw4f(raw[i][2], DT), w = raw4f(raw[i][3], DT);
        if (a.rope.table && 8 * item < a.rope.dim) kv_turn(a.rope, c[i], s[i], x, y);
        if (a.rope.table && !a.rope.adjacent) natural_order<D>(turned[threadIdx.x / L], oa, ob, item, x, y);
        const Row4 k = quantise_row<L>(x, y), v = quantise_row<L>(u, w);
        *reinterpret_cast<uint32_t*>(rec + kv4_key_word<D>(token, item)) = kv4_key_codes(x, y, k.inverse);
        codes[t][4 * group + 2 * (item & 1) + (item >> 1 & 1)] = value_bytes(u, w, v.inverse, item);
        if ((item & 3) == 0) {
            rec[kv4_key_factor<D>(token, group)] = (uint8_t)k.factor;
            rec[KV4_VF(D) + group * KV_PAGE + kv4_place(token)] = (uint8_t)v.factor;
        }
        if (item == 0) {
            float* sc = reinterpret_cast<float*>(rec + KV4_S(D));
            sc[token] = k.scale;
            sc[KV_PAGE + token] = v.scale;
        }
    }
    __syncthreads();
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Groups g = groups_of(slots, lane);
    if (wave == 0) list_groups(g.fours, lane, fours);
    __syncthreads();
    const int first = fours[lane % FOURS];
    if (first >= 0) {
        const int sl = slots[first];
        uint8_t* v = a.cache + ((int64_t)(sl / KV_PAGE) * a.heads + h) * kv4_record(D) + KV4_V(D) + kv4_place(sl % KV_PAGE);
#pragma unroll
        for (int y = 64 / FOURS * wave + lane / FOURS; y < W; y += 256 / FOURS) {
            // places hold tokens 0, 2, 1, 3 of a group
            uint32_t w[4] = {codes[first][y], codes[first + 2][y], codes[first + 1][y], codes[first + 3][y]};
            transpose4(w);
#pragma unroll
            for (int e = 0; e < 4; ++e) *reinterpret_cast<uint32_t*>(v + (4 * y + e) * KV_PAGE) = w[e];
        }
    }
    if (g.singles >> lane & 1) {
        const int sl = slots[lane];
        uint8_t* v = a.cache + ((int64_t)(sl / KV_PAGE) * a.heads + h) * kv4_record(D) + KV4_V(D) + kv4_place(sl % KV_PAGE);
        for (int y = wave; y < W; y += 4) {
            const uint32_t q = codes[lane][y];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[(4 * y + e) * KV_PAGE] = (uint8_t)(q >> (8 * e));
        }
    }
}

// Rounded to fp32 and then to the type.  (The compiler would take a product and its
// conversion to fp16 as one instruction, which rounds once.)
__device__ __forceinline__ float4 scaled(float4 c, float factor, float s) {
    float4 v = make_float4(c.x * factor * s, c.y * factor * s, c.z * factor * s, c.w * factor * s);
    asm("" : "+v"(v.x), "+v"(v.y), "+v"(v.z), "+v"(v.w));
    return v;
}

// The codes of four bytes' low (at 0) or high (at 4) halves.
__device__ __forceinline__ float4 value_codes(uint32_t w, int at) {
    const auto c = [w, at](int e) { return (float)((int)(w >> (8 * e + at) & 15u) - 8); };
    return make_float4(c(0), c(1), c(2), c(3));
}

template <int D>
__global__ __launch_bounds__(256) void kv4_read_kernel(KvRead a) {
    constexpr int L = D / 8, ROWS = 256 / L;
    const int item = threadIdx.x % L;
    const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / L;
    if (row >= a.T * a.heads) return;
    const int64_t t = row / a.heads;
    const int h = (int)(row % a.heads);
    const int slot = a.slots[t];
    float4 k0 = make_float4(0, 0, 0, 0), k1 = k0, v0 = k0, v1 = k0;
    if (slot >= 0 && slot < a.pages * KV_PAGE) {
        const int token = slot % KV_PAGE, group = item >> 2;
        const uint8_t* rec = a.cache + ((int64_t)(slot / KV_PAGE) * a.heads + h) * kv4_record(D);
        const float* sc = reinterpret_cast<const float*>(rec + KV4_S(D)) + token;
        const float kf = kv4_factor_value(rec[kv4_key_factor<D>(token, group)]);
        const float vf = kv4_factor_value(rec[KV4_VF(D) + group * KV_PAGE + kv4_place(token)]);
        kv4_key_values(*reinterpret_cast<const uint32_t*>(rec + kv4_key_word<D>(token, item)), k0, k1);
        const uint8_t* v = rec + KV4_V(D) + group * 1024 + 8 * (item & 1) * KV_PAGE + kv4_place(token);
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e / 4] |= (uint32_t)v[e * KV_PAGE] << (8 * (e % 4));
        k0 = scaled(k0, kf, sc[0]);
        k1 = scaled(k1, kf, sc[0]);
        v0 = scaled(value_codes(w[0], item & 2 ? 4 : 0), vf, sc[KV_PAGE]);
        v1 = scaled(value_codes(w[1], item & 2 ? 4 : 0), vf, sc[KV_PAGE]);
    }
    const int64_t o = row * D + 8 * item;
    store4f(a.k, o, a.dtype, k0);
    store4f(a.k, o + 4, a.dtype, k1);
    store4f(a.v, o, a.dtype, v0);
    store4f(a.v, o + 4, a.dtype, v1);
}

// Many tokens, as kv4_append_tile_kernel's: 32 tokens of one head.
template <int D, int DT>
__global__ __launch_bounds__(256) void kv4_read_tile_kernel(KvRead a) {
    constexpr int L = D / 8, ROWS = 256 / L, W = D / 8;
    __shared__ uint32_t codes[TILE][W + 1];
    __shared__ int slots[TILE], fours[FOURS];
    const int h = (int)(blockIdx.x % a.heads);
    const int64_t t0 = (int64_t)(blockIdx.x / a.heads) * TILE;
    const int n = (int)(a.T - t0 < TILE ? a.T - t0 : TILE);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (wave == 0 && lane < TILE) {
        const int s = lane < n ? a.slots[t0 + lane] : -1;
        slots[lane] = s >= a.pages * KV_PAGE ? -1 : s;
    }
    __syncthreads();
    const Groups g = groups_of(slots, lane);
    if (wave == 0) list_groups(g.fours, lane, fours);
    // the keys' words, factors and scales set out before the values' codes are waited for
    const int item = threadIdx.x % L, group = item >> 2;
    constexpr int N = TILE / ROWS;
    uint32_t kw[N], kf[N], vf[N];
    float ks[N], vs[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int t = i * ROWS + threadIdx.x / L, s = slots[t];
        if (s < 0) continue;
        const int token = s % KV_PAGE;
        const uint8_t* rec = a.cache + ((int64_t)(s / KV_PAGE) * a.heads + h) * kv4_record(D);
        const float* sc = reinterpret_cast<const float*>(rec + KV4_S(D)) + token;
        kw[i] = *reinterpret_cast<const uint32_t*>(rec + kv4_key_word<D>(token, item));
        kf[i] = rec[kv4_key_factor<D>(token, group)];
        vf[i] = rec[KV4_VF(D) + group * KV_PAGE + kv4_place(token)];
        ks[i] = sc[0];
        vs[i] = sc[KV_PAGE];
    }
    __syncthreads();
    const int first = fours[lane % FOURS];
    if (first >= 0) {
        const int s = slots[first];
        const uint8_t* v = a.cache + ((int64_t)(s / KV_PAGE) * a.heads + h) * kv4_record(D) + KV4_V(D) +
                           kv4_place(s % KV_PAGE);
#pragma unroll
        for (int y = 64 / FOURS * wave + lane / FOURS; y < W; y += 256 / FOURS) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = *reinterpret_cast<const uint32_t*>(v + (4 * y + e) * KV_PAGE);
            transpose4(w);
            codes[first][y] = w[0];
            codes[first + 2][y] = w[1];
            codes[first + 1][y] = w[2];
            codes[first + 3][y] = w[3];
        }
    }
    if (g.singles >> lane & 1) {
        const int s = slots[lane];
        const uint8_t* v = a.cache + ((int64_t)(s / KV_PAGE) * a.heads + h) * kv4_record(D) + KV4_V(D) +
                           kv4_place(s % KV_PAGE);
        for (int y = wave; y < W; y += 4) {
            uint32_t q = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) q |= (uint32_t)v[(4 * y + e) * KV_PAGE] << (8 * e);
            codes[lane][y] = q;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int t = i * ROWS + threadIdx.x / L;
        if (t >= n) break;
        float4 k0 = make_float4(0, 0, 0, 0), k1 = k0, v0 = k0, v1 = k0;
        if (slots[t] >= 0) {
            kv4_key_values(kw[i], k0, k1);
            const float f = kv4_factor_value(kf[i]), e = kv4_factor_value(vf[i]);
            k0 = scaled(k0, f, ks[i]);
            k1 = scaled(k1, f, ks[i]);
            const int at = item & 2 ? 4 : 0;
            v0 = scaled(value_codes(codes[t][4 * group + 2 * (item & 1)], at), e, vs[i]);
            v1 = scaled(value_codes(codes[t][4 * group + 2 * (item & 1) + 1], at), e, vs[i]);
        }
        const int64_t o = ((t0 + t) * a.heads + h) * D + 8 * item;
        store4f(a.k, o, DT, k0);
        store4f(a.k, o + 4, DT, k1);
        store4f(a.v, o, DT, v0);
        store4f(a.v, o + 4, DT, v1);
    }
}

// Tokens times heads from which on the tiles take less time where slots run on: appends
// of 512 tokens of 8 heads of 128, fp32, take 5.9 us and 5.0 in the simple form, 1024 6.3
// and 6.9, 2048 7.5 and 11.0 (reads 5.3 and 4.4, 6.3 and 6.4, 9.1 and 9.6); heads of 64,
// bf16, 1024: 4.7 and 5.0; heads of 256, fp32, 512: 9.3 and 8.7, 1024: 10.0 and 14.4.
// Slots apart, one a page, cost either form its single bytes: 1024 of 8 heads of 128, fp32,
// 12.7 and 10.8, 2048 20.6 and 18.7.
constexpr int64_t TILE_FROM_ROWS = 8192;

template <int D, int DT>
hipError_t append_tiles(const KvAppend& a, hipStream_t s) {
    Q8K_LAUNCH((kv4_append_tile_kernel<D, DT>), dim3((unsigned)kv_workgroups(a.T, a.heads)), dim3(256), 0, s, a);
    return hipGetLastError();
}
template <int D>
hipError_t append_d(const KvAppend& a, hipStream_t s) {
    if (a.T * a.heads >= TILE_FROM_ROWS)
        return a.dtype == DT_F32 ? append_tiles<D, DT_F32>(a, s)
               : a.dtype == DT_BF16 ? append_tiles<D, DT_BF16>(a, s) : append_tiles<D, DT_F16>(a, s);
    const int64_t rows = a.T * 2 * a.heads, per = 256 / (D / 8);
    Q8K_LAUNCH((kv4_append_kernel<D>), dim3((unsigned)((rows + per - 1) / per)), dim3(256), 0, s, a);
    return hipGetLastError();
}
template <int D, int DT>
hipError_t read_tiles(const KvRead& a, hipStream_t s) {
    Q8K_LAUNCH((kv4_read_tile_kernel<D, DT>), dim3((unsigned)kv_workgroups(a.T, a.heads)), dim3(256), 0, s, a);
    return hipGetLastError();
}
template <int D>
hipError_t read_d(const KvRead& a, hipStream_t s) {
    if (a.T * a.heads >= TILE_FROM_ROWS)
        return a.dtype == DT_F32 ? read_tiles<D, DT_F32>(a, s)
               : a.dtype == DT_BF16 ? read_tiles<D, DT_BF16>(a, s) : read_tiles<D, DT_F16>(a, s);
    const int64_t rows = a.T * a.heads, per = 256 / (D / 8);
    Q8K_LAUNCH((kv4_read_kernel<D>), dim3((unsigned)((rows + per - 1) / per)), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv4_append(int D, const KvAppend& a, hipStream_t s) {
    return D == 64 ? append_d<64>(a, s) : D == 128 ? append_d<128>(a, s) : append_d<256>(a, s);
}
hipError_t launch_kv4_read(int D, const KvRead& a, hipStream_t s) {
    return D == 64 ? read_d<64>(a, s) : D == 128 ? read_d<128>(a, s) : read_d<256>(a, s);
}

}  // namespace q8k
