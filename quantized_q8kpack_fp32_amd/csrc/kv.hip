// Appending to the paged 8-bit key/value cache, and reading it back.
//
// Append, for each token and head: the key turns by its position,
//   (a, b) -> (a cos - b sin, a sin + b cos),
// then key and value each become D codes and one scale by q8_K's rule with the
// head's row as the block: scale = amax/127, code = round(x * 127/amax).  One
// scale a token (not a page): an append touches no other token's codes, so
// tokens appended one by one and in one call leave the same bytes.
//
// Bound by bytes and by how they are cut: 4 D or 8 D a token and head in, 2 D + 8
// out (8191 tokens of 8 heads of 128, bf16: 51 MB in 17.7 us, 2.9 TB/s; the read
// back 14.7 us, 3.5 TB/s), and for few tokens by the launch and the slot's, the row's
// and the table's loads (one token 2.7 us, its read back 2.1).
#include "kv_cache.h"
#include "kv_tile.h"
#include "q8k_launch.h"

namespace q8k {

namespace {

// The simple form: D/8 lanes a row (a token's key or value of one head), eight
// values a lane.  A value's codes lie 64 bytes apart (one row of places for
// each of the head's D values), so each leaves as a byte.
template <int D>
__global__ __launch_bounds__(256) void kv_append_kernel(KvAppend a) {
    constexpr int L = D / 8, ROWS = 256 / L;
    const int item = threadIdx.x % L;
    const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / L;
    if (row >= a.T * 2 * a.heads) return;  // uniform over the row's lanes
    const int64_t t = row / (2 * a.heads);
    const int hv = (int)(row % (2 * a.heads));
    const bool is_v = hv >= a.heads;
    const int h = is_v ? hv - a.heads : hv;
    const int slot = a.slots[t];
    if (slot < 0 || slot >= a.pages * KV_PAGE) return;
    const int64_t page = slot / KV_PAGE;
    const int token = slot % KV_PAGE;
    RopeView r = a.rope;
    const float* turn = nullptr;
    if (r.table) {
        const int p = a.pos[t];
        if (p < 0 || p >= r.len) return;  // neither key nor value: the token selects nothing
        turn = r.table + (int64_t)p * r.dim;
    }
    if (is_v) r.table = turn = nullptr;
    int oa, ob;
    kv_item(r, item, oa, ob);
    const void* src = is_v ? a.v : a.k;
    const int64_t base = t * (is_v ? a.v_stride : a.k_stride) + (int64_t)h * D;
    float4 x = load4f(src, base + oa, a.dtype), y = load4f(src, base + ob, a.dtype);
    if (turn && 8 * item < r.dim)
        kv_turn(r, *reinterpret_cast<const float4*>(turn + 4 * item),
                *reinterpret_cast<const float4*>(turn + r.dim / 2 + 4 * item), x, y);
    const float amax = group_max<L>(fmaxf(max4(x), max4(y)));
    const float iscale = 127.0f / amax;
    const uint32_t cx = kv_codes4(x, iscale), cy = kv_codes4(y, iscale);
    uint8_t* rec = a.cache + (page * a.heads + h) * kv_record(D);
    if (!is_v) {
        *reinterpret_cast<uint32_t*>(rec + (oa >> 6) * 4096 + token * 64 + (oa & 63)) = cx;
        *reinterpret_cast<uint32_t*>(rec + (ob >> 6) * 4096 + token * 64 + (ob & 63)) = cy;
    } else {
        uint8_t* v = rec + KV_PAGE * D + kv_place(token);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[(oa + e) * KV_PAGE] = (uint8_t)(cx >> (8 * e));
            v[(ob + e) * KV_PAGE] = (uint8_t)(cy >> (8 * e));
        }
    }
    if (item == 0)
        reinterpret_cast<float*>(rec + 2 * KV_PAGE * D)[(is_v ? KV_PAGE : 0) + token] = amax / 127.0f;
}

// Many tokens: one workgroup takes 32 tokens of one head.  Keys go as above.
// The values' codes first meet in LDS.  Four tokens that follow each other from
// a multiple of four on have places that follow each other, and a wave then
// stores the four codes of eight such groups to four rows of places at a time: of
// 32 tokens that begin at a multiple of 32, four pieces of eight consecutive bytes
// of each row.  The tokens that are left (a run's ends, or slots in no order) go byte
// by byte.  Tiles are cut by the call's order and not by pages: a run that begins in
// the middle of four has such tokens in every tile (1024 tokens of 8 heads of 128,
// bf16: 6.6 us, from the start of a page 5.8), and a page's values, 64 D consecutive
// bytes, are written by two or three workgroups.  8191 tokens take 17.7 us for the
// simple form's 49; tiles of 64 tokens, cut the same way, take as long there, and
// longer where tokens are fewer.
template <int D>
__global__ __launch_bounds__(256) void kv_append_tile_kernel(KvAppend a) {
    constexpr int L = D / 8, ROWS = 256 / L;
    constexpr int N = TILE / ROWS;
    __shared__ uint32_t codes[TILE][D / 4 + 1];
    __shared__ float scales[TILE];
    __shared__ int slots[TILE], fours[FOURS];
    const int h = (int)(blockIdx.x % a.heads);
    const int64_t t0 = (int64_t)(blockIdx.x / a.heads) * TILE;
    const int n = (int)(a.T - t0 < TILE ? a.T - t0 : TILE);
    const int item = threadIdx.x % L;
    int oa, ob;
    kv_item(a.rope, item, oa, ob);
    // all rows of the tile (the last one's again behind the last)
    uint4 raw[N][4];
    int slot_of[N], pos[N];
    const auto fetch = [&](bool f32) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t t = t0 + min(i * ROWS + (int)threadIdx.x / L, n - 1);
            const int64_t kb = t * a.k_stride + (int64_t)h * D, vb = t * a.v_stride + (int64_t)h * D;
            raw[i][0] = load4raw(a.k, kb + oa, f32);
            raw[i][1] = load4raw(a.k, kb + ob, f32);
            raw[i][2] = load4raw(a.v, vb + 8 * item, f32);
            raw[i][3] = load4raw(a.v, vb + 8 * item + 4, f32);
        }
    };
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t t = t0 + min(i * ROWS + (int)threadIdx.x / L, n - 1);
        slot_of[i] = a.slots[t];
        pos[i] = a.rope.table ? a.pos[t] : 0;
    }
    if (a.dtype == DT_F32)
        fetch(true);
    else
        fetch(false);
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
        uint8_t* rec = a.cache + ((int64_t)(slot / KV_PAGE) * a.heads + h) * kv_record(D);
        const int token = slot % KV_PAGE;
        float4 x = raw4f(raw[i][0], a.dtype), y = raw4f(raw[i][1], a.dtype);
        const float4 u = raw4f(raw[i][2], a.dtype), w = raw4f(raw[i][3], a.dtype);
        if (a.rope.table && 8 * item < a.rope.dim) kv_turn(a.rope, c[i], s[i], x, y);
        const float kmax = group_max<L>(fmaxf(max4(x), max4(y))), vmax = group_max<L>(fmaxf(max4(u), max4(w)));
        const float ks = 127.0f / kmax, vs = 127.0f / vmax;
        *reinterpret_cast<uint32_t*>(rec + (oa >> 6) * 4096 + token * 64 + (oa & 63)) = kv_codes4(x, ks);
        *reinterpret_cast<uint32_t*>(rec + (ob >> 6) * 4096 + token * 64 + (ob & 63)) = kv_codes4(y, ks);
        codes[t][2 * item] = kv_codes4(u, vs);
        codes[t][2 * item + 1] = kv_codes4(w, vs);
        if (item == 0) {
            reinterpret_cast<float*>(rec + 2 * KV_PAGE * D)[token] = kmax / 127.0f;
            scales[t] = vmax / 127.0f;
        }
    }
    __syncthreads();
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, slot = lane < TILE ? slots[lane] : -1;
    const Groups g = groups_of(slots, lane);
    if (wave == 0) {
        list_groups(g.fours, lane, fours);
        if (slot >= 0)
            reinterpret_cast<float*>(a.cache + ((int64_t)(slot / KV_PAGE) * a.heads + h) * kv_record(D) +
                                     2 * KV_PAGE * D)[KV_PAGE + slot % KV_PAGE] = scales[lane];
    }
    __syncthreads();
    const int first = fours[lane % FOURS];
    if (first >= 0) {
        const int s = slots[first];
        uint8_t* v = a.cache + ((int64_t)(s / KV_PAGE) * a.heads + h) * kv_record(D) + KV_PAGE * D + kv_place(s % KV_PAGE);
#pragma unroll
        for (int c = 64 / FOURS * wave + lane / FOURS; c < D / 4; c += 256 / FOURS) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = codes[first + e][c];
            transpose4(w);
#pragma unroll
            for (int e = 0; e < 4; ++e) *reinterpret_cast<uint32_t*>(v + (4 * c + e) * KV_PAGE) = w[e];
        }
    }
    if (g.singles >> lane & 1) {
        uint8_t* v = a.cache + ((int64_t)(slot / KV_PAGE) * a.heads + h) * kv_record(D) + KV_PAGE * D +
                     kv_place(slot % KV_PAGE);
        for (int c = wave; c < D / 4; c += 4) {
            const uint32_t q = codes[lane][c];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[(4 * c + e) * KV_PAGE] = (uint8_t)(q >> (8 * e));
        }
    }
}

__device__ __forceinline__ float4 dequant4(uint32_t c, float s) {
    return make_float4((float)(int8_t)c * s, (float)(int8_t)(c >> 8) * s, (float)(int8_t)(c >> 16) * s,
                       (float)(int8_t)(c >> 24) * s);
}

template <int D>
__global__ __launch_bounds__(256) void kv_read_kernel(KvRead a) {
    constexpr int L = D / 8, ROWS = 256 / L;
    const int item = threadIdx.x % L;
    const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / L;
    if (row >= a.T * a.heads) return;
    const int64_t t = row / a.heads;
    const int h = (int)(row % a.heads);
    const int slot = a.slots[t];
    float4 k0 = make_float4(0, 0, 0, 0), k1 = k0, v0 = k0, v1 = k0;
    if (slot >= 0 && slot < a.pages * KV_PAGE) {
        const int token = slot % KV_PAGE;
        const uint8_t* rec = a.cache + ((int64_t)(slot / KV_PAGE) * a.heads + h) * kv_record(D);
        const float* sc = reinterpret_cast<const float*>(rec + 2 * KV_PAGE * D) + token;
        const uint2 kc = *reinterpret_cast<const uint2*>(rec + (item >> 3) * 4096 + token * 64 + 8 * (item & 7));
        const uint8_t* v = rec + KV_PAGE * D + 8 * item * KV_PAGE + kv_place(token);
        uint32_t c0 = 0, c1 = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            c0 |= (uint32_t)v[e * KV_PAGE] << (8 * e);
            c1 |= (uint32_t)v[(e + 4) * KV_PAGE] << (8 * e);
        }
        k0 = dequant4(kc.x, sc[0]);
        k1 = dequant4(kc.y, sc[0]);
        v0 = dequant4(c0, sc[KV_PAGE]);
        v1 = dequant4(c1, sc[KV_PAGE]);
    }
    const int64_t o = row * D + 8 * item;
    store4f(a.k, o, a.dtype, k0);
    store4f(a.k, o + 4, a.dtype, k1);
    store4f(a.v, o, a.dtype, v0);
    store4f(a.v, o + 4, a.dtype, v1);
}

// Many tokens, as kv_append_tile_kernel's: 32 tokens of one head.
template <int D>
__global__ __launch_bounds__(256) void kv_read_tile_kernel(KvRead a) {
    constexpr int L = D / 8, ROWS = 256 / L;
    __shared__ uint32_t codes[TILE][D / 4 + 1];
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
    __syncthreads();
    const int first = fours[lane % FOURS];
    if (first >= 0) {
        const int s = slots[first];
        const uint8_t* v = a.cache + ((int64_t)(s / KV_PAGE) * a.heads + h) * kv_record(D) + KV_PAGE * D +
                           kv_place(s % KV_PAGE);
#pragma unroll
        for (int c = 64 / FOURS * wave + lane / FOURS; c < D / 4; c += 256 / FOURS) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = *reinterpret_cast<const uint32_t*>(v + (4 * c + e) * KV_PAGE);
            transpose4(w);
#pragma unroll
            for (int e = 0; e < 4; ++e) codes[first + e][c] = w[e];
        }
    }
    if (g.singles >> lane & 1) {
        const int s = slots[lane];
        const uint8_t* v = a.cache + ((int64_t)(s / KV_PAGE) * a.heads + h) * kv_record(D) + KV_PAGE * D +
                           kv_place(s % KV_PAGE);
        for (int c = wave; c < D / 4; c += 4) {
            uint32_t q = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) q |= (uint32_t)v[(4 * c + e) * KV_PAGE] << (8 * e);
            codes[lane][c] = q;
        }
    }
    __syncthreads();
    const int item = threadIdx.x % L;
#pragma unroll
    for (int i = 0; i < TILE / ROWS; ++i) {
        const int t = i * ROWS + threadIdx.x / L;
        if (t >= n) break;
        const int s = slots[t];
        float4 k0 = make_float4(0, 0, 0, 0), k1 = k0, v0 = k0, v1 = k0;
        if (s >= 0) {
            const int token = s % KV_PAGE;
            const uint8_t* rec = a.cache + ((int64_t)(s / KV_PAGE) * a.heads + h) * kv_record(D);
            const float* sc = reinterpret_cast<const float*>(rec + 2 * KV_PAGE * D) + token;
            const uint2 kc = *reinterpret_cast<const uint2*>(rec + (item >> 3) * 4096 + token * 64 + 8 * (item & 7));
            k0 = dequant4(kc.x, sc[0]);
            k1 = dequant4(kc.y, sc[0]);
            v0 = dequant4(codes[t][2 * item], sc[KV_PAGE]);
            v1 = dequant4(codes[t][2 * item + 1], sc[KV_PAGE]);
        }
        const int64_t o = ((t0 + t) * a.heads + h) * D + 8 * item;
        store4f(a.k, o, a.dtype, k0);
        store4f(a.k, o + 4, a.dtype, k1);
        store4f(a.v, o, a.dtype, v0);
        store4f(a.v, o + 4, a.dtype, v1);
    }
}

// Tokens times heads from which on the tiles take less time where slots run on:
// appends of 512 tokens of 8 heads of 128, fp32, take 6.6 us, 7.5 in the simple
// form, 256 tokens 6.0 and 4.9; heads of 64, bf16, 512: 4.1 and 4.8; heads of 256,
// fp32, 512: 10.6 and 14.7.  A step of many sequences has its slots apart, one a
// page, and every value code goes by itself either way: 61 tokens (simple) 4.2 us,
// 512 of 8 heads of 128, fp32, 19.6 in tiles and 17.7 in the simple form, bf16 17.7
// and 16.0, 1024 39.8 both, 2048 73.5 and 75.2, heads of 64 7.9 and 6.9, of 256 43.3
// and 44.6.  The host does not know the slots, so the rule goes by the runs.
constexpr int64_t TILE_FROM_ROWS = 4096;

template <int D>
hipError_t append_d(const KvAppend& a, hipStream_t s) {
    if (a.T * a.heads >= TILE_FROM_ROWS) {
        Q8K_LAUNCH((kv_append_tile_kernel<D>), dim3((unsigned)kv_workgroups(a.T, a.heads)), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    const int64_t rows = a.T * 2 * a.heads, per = 256 / (D / 8);
    Q8K_LAUNCH((kv_append_kernel<D>), dim3((unsigned)((rows + per - 1) / per)), dim3(256), 0, s, a);
    return hipGetLastError();
}
template <int D>
hipError_t read_d(const KvRead& a, hipStream_t s) {
    if (a.T * a.heads >= TILE_FROM_ROWS) {
        Q8K_LAUNCH((kv_read_tile_kernel<D>), dim3((unsigned)kv_workgroups(a.T, a.heads)), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    const int64_t rows = a.T * a.heads, per = 256 / (D / 8);
    Q8K_LAUNCH((kv_read_kernel<D>), dim3((unsigned)((rows + per - 1) / per)), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

int64_t kv_workgroups(int64_t T, int64_t heads) { return (T + TILE - 1) / TILE * heads; }

hipError_t launch_kv_append(int D, const KvAppend& a, hipStream_t s) {
    return D == 64 ? append_d<64>(a, s) : D == 128 ? append_d<128>(a, s) : append_d<256>(a, s);
}
hipError_t launch_kv_read(int D, const KvRead& a, hipStream_t s) {
    return D == 64 ? read_d<64>(a, s) : D == 128 ? read_d<128>(a, s) : read_d<256>(a, s);
}

}  // namespace q8k
