// Eviction from a paged key/value cache of 8 or 4 bits: of each sequence longer
// than the budget, every key head keeps its first and last tokens and, of the
// others, those of the largest weights (equal ones by ascending index), in order;
// what the cache holds of these moves to the front of the sequence's new pages.
//
// Two launches: the choice (one workgroup a sequence and head; 8 rows of 2111 weights 6.1
// us, a chain of barriers, 128 of up to 16001 14.9, 8 of 65537, read again for each digit,
// 68) and the move (4000 of up to 16001 tokens of 128 rows, 8 bits, heads of 128: 96 us, 4.2
// TB/s of what it touches, since a page's values lie row by row and a line of 64 tokens is
// read for one; 2048 of 2111 tokens of 8 rows, 4 bits, 4.4).  In place the pages of a head go
// one after another, each behind a chain of loads and stores: 47 us for the 2048 of 2111,
// 184 for the 4000 of up to 16001.  A page's places beyond the kept tokens are left as they
// were.
#include "attend.h"
#include "q8k_launch.h"

namespace q8k {

namespace {

constexpr int THREADS = 1024, WAVES = THREADS / 64;

// Weights as whole numbers of the same order, 1 to ALWAYS - 1; NaN below all, -0 as 0.
// A token that is kept whatever its weight has ALWAYS, a place behind the last NEVER.
constexpr uint32_t ALWAYS = 0xffffffffu, NEVER = 0;
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
    return v != v ? 1u : b >> 31 ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ int lanes_below(uint64_t mask) {
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// The least key that is kept, digit by digit from the top (11, 11 and 10 bits, each with
// the counts of all its values), then one pass in order.  The weights are read once:
// EACH a thread stay in registers beside their keys (longer rows are read again, 1024 EACH
// at a time), and what a place's index says is in its key, so that it is looked at once
// (at every digit: 16.9 us for 15.0).
template <int EACH>
__global__ __launch_bounds__(THREADS) void kv_evict_choose_kernel(KvEvict a) {
    constexpr int CHUNK = THREADS * EACH;
    __shared__ int hist[2048], sums[WAVES], found[3];
    __shared__ uint32_t counts[EACH * WAVES + 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = blockIdx.x, b = row / a.heads;
    const int64_t l = a.kv_len[b];
    const float* in = a.weights + row * a.w_stride;
    float* out = a.out_weights ? a.out_weights + row * a.out_stride : nullptr;
    int* kept = a.kept + row * a.budget;
    float v[EACH];
    uint32_t k[EACH];
    const auto load = [&](int c) {
#pragma unroll
        for (int r = 0; r < EACH; ++r) {
            const int64_t i = (int64_t)c * CHUNK + r * THREADS + (int)threadIdx.x;
            v[r] = i < a.max_len ? in[i] : 0.0f;  // (whatever the length, which needs not be waited for)
        }
    };
    load(0);
    const int len = (int)(l < 0 ? 0 : l > a.max_len ? a.max_len : l), budget = (int)a.budget;
    if (row % a.heads == 0 && threadIdx.x == 0) a.new_len[b] = min(len, budget);
    if (len <= budget) {
        for (int i = threadIdx.x; i < budget; i += THREADS) {
            kept[i] = i < len ? i : -1;
            if (i < len && out && out != in) out[i] = in[i];
        }
        return;
    }
    const int c0 = (int)a.first, c1 = len - (int)a.last, want = budget - (int)(a.first + a.last);
    const int chunks = (len + CHUNK - 1) / CHUNK;
    const auto keys = [&](int c) {
#pragma unroll
        for (int r = 0; r < EACH; ++r) {
            const int i = c * CHUNK + r * THREADS + (int)threadIdx.x;
            k[r] = i >= len ? NEVER : i < c0 || i >= c1 ? ALWAYS : key_of(v[r]);
        }
    };
    keys(0);
    uint32_t prefix = want > 0 ? 0 : ALWAYS - 1, mask = 0;
    int rest = want;
    if (want > 0)
        for (int digit = 0; digit < 3; ++digit) {
            const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
            const uint32_t most = digit == 2 ? 1023u : 2047u;
            hist[threadIdx.x] = hist[threadIdx.x + THREADS] = 0;
            __syncthreads();
            for (int c = 0; c < chunks; ++c) {
                if (chunks > 1) load(c), keys(c);
#pragma unroll
                for (int r = 0; r < EACH; ++r)
                    if (k[r] + 1 > NEVER + 1 && (k[r] & mask) == prefix) atomicAdd(&hist[k[r] >> shift & most], 1);
            }
            __syncthreads();
            // thread t: the counts of values 2047 - 2 t and 2046 - 2 t, and of all above them
            const int x = hist[2047 - 2 * threadIdx.x], y = hist[2046 - 2 * threadIdx.x], upto = wave_scan(x + y);
            if (lane == 63) sums[wave] = upto;
            __syncthreads();
            int above = upto - x - y;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) above += w < wave ? sums[w] : 0;
            if (above < rest && rest <= above + x + y) {
                const bool second = rest > above + x;
                found[0] = 2047 - 2 * (int)threadIdx.x - (second ? 1 : 0);
                found[1] = rest - above - (second ? x : 0);
                found[2] = second ? y : x;
            }
            __syncthreads();
            prefix |= (uint32_t)found[0] << shift;
            mask |= most << shift;
            rest = found[1];
            if (found[2] == rest) {
                // all of them are kept: those above what is just below (never below all keys: some token goes)
                prefix -= 1;
                rest = 0;
                break;
            }
        }
    // in order: all above it, and the first `rest` of those equal to it
    int done = 0, ties = 0;
    for (int c = 0; c < chunks; ++c) {
        if (chunks > 1) load(c), keys(c);
        uint64_t ma[EACH], mt[EACH];
#pragma unroll
        for (int r = 0; r < EACH; ++r) {
            ma[r] = __ballot(k[r] > prefix);
            mt[r] = __ballot(k[r] == prefix);
            if (lane == 0) counts[r * WAVES + wave] = (uint32_t)__popcll(ma[r]) | (uint32_t)__popcll(mt[r]) << 16;
        }
        __syncthreads();
        if (wave == 0) {
            constexpr int N = EACH * WAVES / 64;
            uint32_t n[N], sum = 0;
#pragma unroll
            for (int i = 0; i < N; ++i) n[i] = counts[N * lane + i], sum += n[i];
            uint32_t before = (uint32_t)wave_scan((int)sum) - sum;
#pragma unroll
            for (int i = 0; i < N; ++i) counts[N * lane + i] = before, before += n[i];
            if (lane == 63) counts[EACH * WAVES] = before;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < EACH; ++r) {
            const int i = c * CHUNK + r * THREADS + (int)threadIdx.x;
            const uint32_t before = counts[r * WAVES + wave];
            const int t = ties + (int)(before >> 16) + lanes_below(mt[r]);
            const int at = done + (int)(before & 0xffffu) + lanes_below(ma[r]) + min(t, rest);
            if ((ma[r] >> lane & 1) || ((mt[r] >> lane & 1) && t < rest)) {
                kept[at] = i;
                if (out) out[at] = v[r];
            }
        }
        const uint32_t all = counts[EACH * WAVES];
        done += (int)(all & 0xffffu);
        ties += (int)(all >> 16);
        __syncthreads();
    }
}

template <int CTRL>
__device__ __forceinline__ uint32_t quad(uint32_t w) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, CTRL, 0xF, 0xF, false);
}

// The move.  What a page holds of its tokens is cut into parts, a wave each: lane t
// brings token kept[64 P + t] of the new page P.  In place the pages go one after
// another: a kept token's new place is never behind its old one, so that a page's
// tokens, all loaded before any is stored, come from places that no earlier page
// was stored to.
//   parts of 64 bytes a token of the keys' codes, of 32 rows of places of the values'
//   codes, and one of the scales and, in 4 bits, the factors
// Four tokens of one group of four change places within the wave, so that their bytes of
// a row leave as a word.
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
    const int* kept = a.kept + (b * a.heads + h) * a.budget;
    const int P0 = IN_PLACE ? 0 : (int)(id % pages), P1 = IN_PLACE ? (int)pages : P0 + 1;
    const int place = BITS == 8 ? kv_place(lane) : kv4_place(lane);
    for (int P = P0; P < P1; ++P) {
        const int i = P * KV_PAGE + lane, old = i < a.budget ? kept[i] : -1;
        const int to_page = a.out_table[b * a.out_pages + P];
        const bool there = old >= 0, whole = __all(there);
        if (!__any(there)) return;
        if (IN_PLACE && __all(!there || old == i)) continue;
        const int from = there ? old : 0, n = __popcll(__ballot(there));  // the first n places
        if (to_page < 0 || to_page >= a.pages) continue;
        const int src_page = a.table[b * a.max_pages + from / KV_PAGE], token = from % KV_PAGE;
        const bool good = there && src_page >= 0 && src_page < a.pages;
        const int64_t rec = good ? ((int64_t)src_page * a.heads + h) * bytes : -1;
        uint8_t* dst = a.cache + ((int64_t)to_page * a.heads + h) * bytes;
        if (part < KEYS) {
            // four lanes a token, sixteen tokens at a time; 16 bytes a lane, in 4 bits and 64 values 8
            constexpr bool small = BITS == 4 && D == 64;
            const int piece = lane & 3;
            const auto at = [&](int t) {
                if (BITS == 8) return part * 4096 + t * 64 + piece * 16;
                if (small) return (t >> 5) * 1024 + (t & 15) * 64 + piece * 16 + ((t >> 4) & 1) * 8;
                return ((t >> 4) * (D / 128) + part) * 1024 + (t & 15) * 64 + piece * 16;
            };
            uint4 v[4];
            int64_t r[4];
            int t[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int who = 16 * c + (lane >> 2);
                r[c] = __shfl(rec, who, 64);
                t[c] = __shfl(token, who, 64);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                v[c] = make_uint4(0, 0, 0, 0);
                if (r[c] < 0) continue;
                if constexpr (small) {
                    const uint2 x = *reinterpret_cast<const uint2*>(a.cache + r[c] + at(t[c]));
                    v[c].x = x.x, v[c].y = x.y;
                } else {
                    v[c] = *reinterpret_cast<const uint4*>(a.cache + r[c] + at(t[c]));
                }
            }
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int who = 16 * c + (lane >> 2);
                if (who >= n) continue;
                if constexpr (small)
                    *reinterpret_cast<uint2*>(dst + at(who)) = make_uint2(v[c].x, v[c].y);
                else
                    *reinterpret_cast<uint4*>(dst + at(who)) = v[c];
            }
        } else if (part < KEYS + VALUES) {
            const int base = (BITS == 8 ? KV_PAGE * D : KV4_V(D)) + (part - KEYS) * ROWS * KV_PAGE;
            const uint8_t* src = a.cache + (good ? rec : 0) + base + (BITS == 8 ? kv_place(token) : kv4_place(token));
            uint32_t v[ROWS];
#pragma unroll
            for (int r = 0; r < ROWS; ++r) v[r] = good ? src[r * KV_PAGE] : 0;
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            if (whole) {
                // the four lanes of a group hold the bytes of places p .. p + 3, in their order 0, 1, 2, 3 or (4 bits)
                // 0, 2, 1, 3: lane k of places' order is left with the word of row 4 r + k
                const bool odd = place & 1, upper = place & 2;
                const uint32_t one = odd ? 0x03070105u : 0x06020400u, two = upper ? 0x03020706u : 0x05040100u;
#pragma unroll
                for (int r = 0; r < ROWS / 4; ++r) {
                    uint32_t w = v[4 * r] | v[4 * r + 1] << 8 | v[4 * r + 2] << 16 | v[4 * r + 3] << 24;
                    // with the neighbour in the places' lowest bit: bytes (mine, its) of rows 0 and 2, or 1 and 3
                    w = __builtin_amdgcn_perm(BITS == 8 ? quad<0xB1>(w) : quad<0x4E>(w), w, one);
                    w = __builtin_amdgcn_perm(BITS == 8 ? quad<0x4E>(w) : quad<0xB1>(w), w, two);
                    *reinterpret_cast<uint32_t*>(dst + base + (4 * r + (place & 3)) * KV_PAGE + (place & ~3)) = w;
                }
            } else if (there) {
#pragma unroll
                for (int r = 0; r < ROWS; ++r) dst[base + r * KV_PAGE + place] = (uint8_t)v[r];
            }
        } else {
            const uint8_t* src = a.cache + (good ? rec : 0);
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
                        dst[KV4_VF(D) + y * KV_PAGE + place] = (uint8_t)vf[y];
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

// Four weights a thread for rows that they hold, else sixteen (both launches, 200 kept, 8
// heads of 128, 4 bits: 8 rows of 2111 9.6 us, of sixteen a thread 13.3, 8 of 4096 10.0 and
// 13.7, 128 18.8 and 23.3; 8 of 5000 14.4, of four a thread, in two turns, 14.2, 8 of 16000
// 15.4 and 21.8, 128 33.8 and 40.2, 8 of 65537 66.5 and 63.9).
hipError_t launch_kv_evict(int bits, int D, const KvEvict& a, bool in_place, hipStream_t s) {
    if (a.max_len <= 4 * THREADS)
        Q8K_LAUNCH((kv_evict_choose_kernel<4>), dim3((unsigned)(a.B * a.heads)), dim3(THREADS), 0, s, a);
    else
        Q8K_LAUNCH((kv_evict_choose_kernel<16>), dim3((unsigned)(a.B * a.heads)), dim3(THREADS), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (bits == 8) return D == 64 ? move_d<64, 8>(a, in_place, s) : D == 128 ? move_d<128, 8>(a, in_place, s) : move_d<256, 8>(a, in_place, s);
    return D == 64 ? move_d<64, 4>(a, in_place, s) : D == 128 ? move_d<128, 4>(a, in_place, s) : move_d<256, 4>(a, in_place, s);
}

}  // namespace q8k
