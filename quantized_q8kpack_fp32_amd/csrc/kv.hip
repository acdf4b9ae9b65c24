// Appending to the paged 8-bit key/value cache, and reading it back.
//
// Append, for each token and head: the key turns by its position,
//   (a, b) -> (a cos - b sin, a sin + b cos),
// then key and value each become D codes and one scale by q8_K's rule with the
// head's row as the block: scale = amax/127, code = round(x * 127/amax).  One
// scale a token (not a page): an append touches no other token's codes, so
// tokens appended one by one and in one call leave the same bytes.
#include "kv_cache.h"
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
    const uint32_t cx = amax != 0.0f ? kv_codes4(x, iscale) : 0u, cy = amax != 0.0f ? kv_codes4(y, iscale) : 0u;
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
        reinterpret_cast<float*>(rec + 2 * KV_PAGE * D)[(is_v ? KV_PAGE : 0) + token] = amax != 0.0f ? amax / 127.0f : 0.0f;
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

template <int D>
hipError_t append_d(const KvAppend& a, hipStream_t s) {
    const int64_t rows = a.T * 2 * a.heads, per = 256 / (D / 8);
    Q8K_LAUNCH((kv_append_kernel<D>), dim3((unsigned)((rows + per - 1) / per)), dim3(256), 0, s, a);
    return hipGetLastError();
}
template <int D>
hipError_t read_d(const KvRead& a, hipStream_t s) {
    const int64_t rows = a.T * a.heads, per = 256 / (D / 8);
    Q8K_LAUNCH((kv_read_kernel<D>), dim3((unsigned)((rows + per - 1) / per)), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(int D, const KvAppend& a, hipStream_t s) {
    return D == 64 ? append_d<64>(a, s) : D == 128 ? append_d<128>(a, s) : append_d<256>(a, s);
}
hipError_t launch_kv_read(int D, const KvRead& a, hipStream_t s) {
    return D == 64 ? read_d<64>(a, s) : D == 128 ? read_d<128>(a, s) : read_d<256>(a, s);
}

}  // namespace q8k
