// Appending to the paged 4-bit key/value cache, and reading it back.
//
// Append, for each token and head: the key turns by its position, then key and
// value each become D codes of 4 bits, D/32 factors and one scale:
//   scale = amax/7,  factor_y = the least 8-bit float >= max|x_y| / amax,
//   code = round(x / (factor_y scale)).
// Bound by bytes: 4 D or 8 D a token and head in, D + D/16 + 8 out.
#include "kv4_cache.h"
#include "q8k_launch.h"

namespace q8k {

namespace {

// Maximum over aligned groups of four lanes, of magnitudes (group_max's rule).
__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, dpp_f(v, 0));
    v = fmaxf(v, dpp_f(v, 1));
    return fmaxf(v, 0.0f);
}
// Codes of lanes two apart in a group of four.
__device__ __forceinline__ uint32_t other_half(uint32_t w) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0x4E, 0xF, 0xF, false);  // quad_perm 2,3,0,1
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
    if (turn && 8 * item < r.dim) {
        kv_turn(r, *reinterpret_cast<const float4*>(turn + 4 * item),
                *reinterpret_cast<const float4*>(turn + r.dim / 2 + 4 * item), x, y);
    }
    if (turn && !r.adjacent) {
        float* row_s = turned[threadIdx.x / L];  // the row's lanes are of one wave
        *reinterpret_cast<float4*>(row_s + oa) = x;
        *reinterpret_cast<float4*>(row_s + ob) = y;
        __builtin_amdgcn_wave_barrier();
        x = *reinterpret_cast<const float4*>(row_s + 8 * item);
        y = *reinterpret_cast<const float4*>(row_s + 8 * item + 4);
    }
    const float most = fmaxf(max4(x), max4(y)), top = quad_max(most), amax = group_max<L>(most);
    const float scale = amax / 7.0f;
    const uint32_t factor = kv4_factor(top / amax);
    const float inverse = kv4_inverse(factor, scale);
    uint8_t* rec = a.cache + (page * a.heads + h) * kv4_record(D);
    const int group = item >> 2;
    if (!is_v) {
        *reinterpret_cast<uint32_t*>(rec + kv4_key_word<D>(token, item)) = kv4_key_codes(x, y, inverse);
        if ((item & 3) == 0) rec[kv4_key_factor<D>(token, group)] = (uint8_t)factor;
    } else {
        // lanes 0 and 1 of a group hold its first sixteen values, 2 and 3 the others, which lie beside them
        const uint32_t lo = kv4_code(x.x, inverse) | kv4_code(x.y, inverse) << 8 | kv4_code(x.z, inverse) << 16 |
                            kv4_code(x.w, inverse) << 24;
        const uint32_t hi = kv4_code(y.x, inverse) | kv4_code(y.y, inverse) << 8 | kv4_code(y.z, inverse) << 16 |
                            kv4_code(y.w, inverse) << 24;
        const uint32_t lo2 = other_half(lo), hi2 = other_half(hi);
        const bool second = item & 2;
        const uint32_t w = second ? hi2 | hi << 4 : lo | lo2 << 4;
        uint8_t* v = rec + KV4_V(D) + group * 1024 + (8 * (item & 1) + (second ? 4 : 0)) * KV_PAGE + kv4_place(token);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e * KV_PAGE] = (uint8_t)(w >> (8 * e));
        if ((item & 3) == 0) rec[KV4_VF(D) + group * KV_PAGE + kv4_place(token)] = (uint8_t)factor;
    }
    if (item == 0) reinterpret_cast<float*>(rec + KV4_S(D))[(is_v ? KV_PAGE : 0) + token] = scale;
}

__device__ __forceinline__ float4 scaled(float4 c, float factor, float s) {
    return make_float4(c.x * factor * s, c.y * factor * s, c.z * factor * s, c.w * factor * s);
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
        const int at = item & 2 ? 4 : 0;
        float c[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = (float)((int)(v[e * KV_PAGE] >> at & 15u) - 8);
        k0 = scaled(k0, kf, sc[0]);
        k1 = scaled(k1, kf, sc[0]);
        v0 = scaled(make_float4(c[0], c[1], c[2], c[3]), vf, sc[KV_PAGE]);
        v1 = scaled(make_float4(c[4], c[5], c[6], c[7]), vf, sc[KV_PAGE]);
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
    Q8K_LAUNCH((kv4_append_kernel<D>), dim3((unsigned)((rows + per - 1) / per)), dim3(256), 0, s, a);
    return hipGetLastError();
}
template <int D>
hipError_t read_d(const KvRead& a, hipStream_t s) {
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
