// Eviction from a paged key/value cache of 8 or 4 bits: of each sequence longer
// than the budget, every key head keeps its first and last tokens and, of the
// others, those of the largest weights (equal ones by ascending index), in order;
// what the cache holds of these moves to the front of the sequence's new pages.
//
// Two launches: the choice (one workgroup a sequence and head: the least weight kept
// by its digits, eight bits a pass over the weights, then one pass in order), and
// the move.  A page's places beyond the kept tokens are left as they were.
#include "kv4_cache.h"
#include "q8k_launch.h"

namespace q8k {

namespace {

constexpr int THREADS = 1024;

// Weights as whole numbers of the same order; NaN below all, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
    return v != v ? 0u : b >> 31 ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ int lanes_below(uint64_t mask, int lane) { return __popcll(mask & ((1ull << lane) - 1)); }

__global__ __launch_bounds__(THREADS) void kv_evict_choose_kernel(KvEvict a) {
    __shared__ int hist[256], found[2], counts[2][2][THREADS / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = blockIdx.x, b = row / a.heads;
    int64_t l = a.kv_len[b];
    const int len = (int)(l < 0 ? 0 : l > a.max_len ? a.max_len : l), budget = (int)a.budget;
    const float* in = a.weights + row * a.w_stride;
    float* out = a.out_weights ? a.out_weights + row * a.out_stride : nullptr;
    int* kept = a.kept + row * a.budget;
    if (row % a.heads == 0 && threadIdx.x == 0) a.new_len[b] = min(len, budget);
    if (len <= budget) {
        for (int i = threadIdx.x; i < budget; i += THREADS) {
            kept[i] = i < len ? i : -1;
            if (i < len && out && out != in) out[i] = in[i];
        }
        return;
    }
    const int c0 = (int)a.first, c1 = len - (int)a.last, want = budget - (int)(a.first + a.last);
    // the want-th largest key among the candidates, digit by digit
    uint32_t prefix = 0, mask = 0;
    int rest = want;
    if (want > 0)
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = threadIdx.x; i < 256; i += THREADS) hist[i] = 0;
            __syncthreads();
            for (int i = c0 + threadIdx.x; i < c1; i += THREADS) {
                const uint32_t k = key_of(in[i]);
                if ((k & mask) == prefix) atomicAdd(&hist[k >> shift & 255u], 1);
            }
            __syncthreads();
            if (threadIdx.x == 0) {
                int above = 0, d = 255;
                while (above + hist[d] < rest) above += hist[d--];
                found[0] = d;
                found[1] = rest - above;
            }
            __syncthreads();
            prefix |= (uint32_t)found[0] << shift;
            mask |= 255u << shift;
            rest = found[1];
            __syncthreads();
        }
    // in order: all above it, and the first `rest` of those equal to it
    int done = 0, ties = 0;
    for (int i0 = 0, turn = 0; i0 < len; i0 += THREADS, turn ^= 1) {
        const int i = i0 + threadIdx.x;
        const bool inside = i < len, fixed = inside && (i < c0 || i >= c1);
        const float v = inside ? in[i] : 0.0f;
        const uint32_t k = key_of(v);
        const bool above = inside && (fixed || (want > 0 && k > prefix)), tie = inside && !fixed && want > 0 && k == prefix;
        const uint64_t ma = __ballot(above), mt = __ballot(tie);
        if (lane == 0) counts[turn][0][wave] = __popcll(ma), counts[turn][1][wave] = __popcll(mt);
        __syncthreads();
        int before = 0, tied = 0, all = 0, all_tied = 0;
        for (int w = 0; w < THREADS / 64; ++w) {
            const int x = counts[turn][0][w], y = counts[turn][1][w];
            before += w < wave ? x : 0, tied += w < wave ? y : 0;
            all += x, all_tied += y;
        }
        const int t = ties + tied + lanes_below(mt, lane);  // ties before this one
        const int at = done + before + lanes_below(ma, lane) + min(t, rest) - 0;
        if (above || (tie && t < rest)) {
            kept[at] = i;
            if (out) out[at] = v;
        }
        done += all;
        ties += all_tied;
    }
}

// The move.  What a page holds of its tokens is cut into parts, a wave each: lane t
// brings token kept[64 P + t] of the new page P.  In place the pages go one after
// another: a kept token's new place is never behind its old one, so that a page's
// tokens, all loaded before any is stored, come from places that no earlier page
// was stored to.
//   parts of 64 bytes a token of the keys' codes, of 32 rows of places (the values' codes
//   and, in 4 bits, their factors), and one of the scales and the keys' factors
template <int D, int BITS, bool IN_PLACE>
__global__ __launch_bounds__(64) void kv_evict_move_kernel(KvEvict a) {
    constexpr int bytes = kv_record_of(BITS, D);
    constexpr int KEYS = BITS == 8 ? D / 64 : D == 256 ? 2 : 1, ROWS = 32, VALUES = (BITS == 8 ? D : D / 2) / ROWS;
    constexpr int PARTS = KEYS + VALUES + 1;
    const int lane = threadIdx.x;
    int64_t id = blockIdx.x;
    const int part = (int)(id % PARTS);
    id /= PARTS;
    const int h = (int)(id % a.heads);
    id /= a.heads;
    const int64_t pages = (a.budget + KV_PAGE - 1) / KV_PAGE;
    const int64_t b = IN_PLACE ? id : id / pages;
    const int64_t l = a.kv_len[b];
    const int len = (int)(l < 0 ? 0 : l > a.max_len ? a.max_len : l), n = min(len, (int)a.budget);
    const int* kept = a.kept + (b * a.heads + h) * a.budget;
    const int P0 = IN_PLACE ? 0 : (int)(id % pages), P1 = IN_PLACE ? (n + KV_PAGE - 1) / KV_PAGE : P0 + 1;
    for (int P = P0; P < P1; ++P) {
        const int i = P * KV_PAGE + lane;
        const bool there = i < n;
        const int from = there ? kept[i] : 0;
        if (IN_PLACE && __all(!there || from == i)) continue;
        const int to_page = a.out_table[b * a.out_pages + P];
        if (P * KV_PAGE >= n || to_page < 0 || to_page >= a.pages) continue;
        const int src_page = a.table[b * a.max_pages + from / KV_PAGE], token = from % KV_PAGE;
        const bool good = there && src_page >= 0 && src_page < a.pages;
        const uint8_t* src = a.cache + ((int64_t)(good ? src_page : 0) * a.heads + h) * bytes;
        uint8_t* dst = a.cache + ((int64_t)to_page * a.heads + h) * bytes;
        if (part < KEYS) {
            // four pieces of 16 bytes; in 4 bits and 64 values of 8
            constexpr bool small = BITS == 4 && D == 64;
            const auto at = [&](int t, int c) {
                if (BITS == 8) return part * 4096 + t * 64 + c * 16;
                if (small) return (t >> 5) * 1024 + (t & 15) * 64 + c * 16 + ((t >> 4) & 1) * 8;
                return ((t >> 4) * (D / 128) + part) * 1024 + (t & 15) * 64 + c * 16;
            };
            uint4 v[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                v[c] = make_uint4(0, 0, 0, 0);
                if (!good) continue;
                if constexpr (small) {
                    const uint2 x = *reinterpret_cast<const uint2*>(src + at(token, c));
                    v[c].x = x.x, v[c].y = x.y;
                } else {
                    v[c] = *reinterpret_cast<const uint4*>(src + at(token, c));
                }
            }
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            if (there)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if constexpr (small)
                        *reinterpret_cast<uint2*>(dst + at(lane, c)) = make_uint2(v[c].x, v[c].y);
                    else
                        *reinterpret_cast<uint4*>(dst + at(lane, c)) = v[c];
                }
        } else if (part < KEYS + VALUES) {
            const int base = (BITS == 8 ? KV_PAGE * D : KV4_V(D)) + (part - KEYS) * ROWS * KV_PAGE;
            const int p = BITS == 8 ? kv_place(token) : kv4_place(token), to = BITS == 8 ? kv_place(lane) : kv4_place(lane);
            uint32_t v[ROWS];
#pragma unroll
            for (int r = 0; r < ROWS; ++r) v[r] = good ? src[base + r * KV_PAGE + p] : 0;
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            if (there)
#pragma unroll
                for (int r = 0; r < ROWS; ++r) dst[base + r * KV_PAGE + to] = (uint8_t)v[r];
        } else {
            const float* s = reinterpret_cast<const float*>(src + bytes - 8 * KV_PAGE) + token;
            const float k = good ? s[0] : 0.0f, v = good ? s[KV_PAGE] : 0.0f;
            uint32_t kf[BITS == 4 ? D / 32 : 1], vf[BITS == 4 ? D / 32 : 1];
            if constexpr (BITS == 4)
#pragma unroll
                for (int y = 0; y < D / 32; ++y) {
                    kf[y] = good ? src[kv4_key_factor<D>(token, y)] : 0;
                    vf[y] = good ? src[KV4_VF(D) + y * KV_PAGE + kv4_place(token)] : 0;
                }
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            if (there) {
                float* d = reinterpret_cast<float*>(dst + bytes - 8 * KV_PAGE) + lane;
                d[0] = k;
                d[KV_PAGE] = v;
                if constexpr (BITS == 4)
#pragma unroll
                    for (int y = 0; y < D / 32; ++y) {
                        dst[kv4_key_factor<D>(lane, y)] = (uint8_t)kf[y];
                        dst[KV4_VF(D) + y * KV_PAGE + kv4_place(lane)] = (uint8_t)vf[y];
                    }
            }
        }
    }
}

constexpr int parts_of(int bits, int D) {
    return (bits == 8 ? D / 64 : D == 256 ? 2 : 1) + (bits == 8 ? D : D / 2) / 32 + 1;
}

template <int D, int BITS>
hipError_t move_d(const KvEvict& a, bool in_place, hipStream_t s) {
    const unsigned grid = (unsigned)evict_workgroups(BITS, D, a.B, a.heads, a.budget, in_place);
    if (in_place)
        Q8K_LAUNCH((kv_evict_move_kernel<D, BITS, true>), dim3(grid), dim3(64), 0, s, a);
    else
        Q8K_LAUNCH((kv_evict_move_kernel<D, BITS, false>), dim3(grid), dim3(64), 0, s, a);
    return hipGetLastError();
}

}  // namespace

int64_t evict_workgroups(int bits, int D, int64_t B, int64_t heads, int64_t budget, bool in_place) {
    return B * heads * parts_of(bits, D) * (in_place ? 1 : (budget + KV_PAGE - 1) / KV_PAGE);
}
int evict_threads() { return THREADS; }

hipError_t launch_kv_evict(int bits, int D, const KvEvict& a, bool in_place, hipStream_t s) {
    Q8K_LAUNCH(kv_evict_choose_kernel, dim3((unsigned)(a.B * a.heads)), dim3(THREADS), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (bits == 8) return D == 64 ? move_d<64, 8>(a, in_place, s) : D == 128 ? move_d<128, 8>(a, in_place, s) : move_d<256, 8>(a, in_place, s);
    return D == 64 ? move_d<64, 4>(a, in_place, s) : D == 128 ? move_d<128, 4>(a, in_place, s) : move_d<256, 4>(a, in_place, s);
}

}  // namespace q8k
