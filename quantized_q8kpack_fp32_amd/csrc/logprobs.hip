// Log probabilities of given tokens, the entropy of each row of logits and its
// top alternatives, in one pass over the logits and one launch (two where few long
// rows are cut into parts).
//
//   m = max x, Z = sum e^(x - m), lse = m + log Z
//   logprob = x[target] - lse,  entropy = log Z - sum e^(x - m) (x - m) / Z
//   top: the topn largest, by (logit descending, id ascending)
//
// Bound by reading the logits once.  One workgroup a row (or a part of a long
// one where rows are few): every thread takes 32 logits at a time and keeps its
// own maximum and sums, which meet at the end.  The top list is kept in LDS and
// renewed from round to round (1024 threads' 32768 logits are one).  512 x 32000
// fp32 logits, eight of each on top: 16.2 us, 4.1 TB/s, with two workgroups a
// compute unit one round of loads and the selection behind it (some 4 us); one
// row 7.5 us, launch and latency; 48 x 128257 bf16, top 20, in five parts a row
// 14.2 us, 4 of them the join.
#include "kv_cache.h"
#include "q8k_launch.h"

namespace q8k {

namespace {

constexpr int PER = 32;       // logits a thread holds
constexpr int TOP_MAX = 32;
constexpr int CAND_MAX = 512; // candidates that are ranked against each other

// A logit as an unsigned integer that orders as the logits do; -0 counts as 0,
// a NaN is below every number, 0 is below everything.
__device__ __forceinline__ uint32_t order_of(float x) {
    uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);
    u = (u & 0x80000000u) ? ~u : u | 0x80000000u;
    return x != x ? 1u : u;
}
__device__ __forceinline__ float logit_of(uint32_t u) {
    if (u == 1u) return __builtin_nanf("");
    return __builtin_bit_cast(float, (u & 0x80000000u) ? u & 0x7fffffffu : ~u);
}
// With its id as one integer that orders as (logit, -id): distinct for every
// id, so that "larger" leaves no ties.
__device__ __forceinline__ uint64_t key_of(uint32_t u, int id) { return (uint64_t)u << 32 | (uint32_t)~(uint32_t)id; }
__device__ __forceinline__ int id_of(uint64_t k) { return (int)~(uint32_t)k; }

template <int DT>
struct Logits {
    static constexpr int SIZE = DT == DT_F32 ? 4 : 2;
    static constexpr int N = 16 / SIZE;     // logits of a 16-byte load
    static constexpr int REGS = PER / N * 4;  // the registers they take
};
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));
typedef u4_t u4_any __attribute__((aligned(2)));  // at any element's address

template <int DT>
__device__ __forceinline__ float load_one(const uint8_t* p) {
    if constexpr (DT == DT_F32) return *reinterpret_cast<const float*>(p);
    const uint32_t w = *reinterpret_cast<const uint16_t*>(p);
    return DT == DT_BF16 ? __builtin_bit_cast(float, w << 16) : half_bits_to_float(w);
}
// Logit j of a thread's registers.
template <int DT>
__device__ __forceinline__ float logit_at(const uint32_t (&r)[Logits<DT>::REGS], int j) {
    if constexpr (DT == DT_F32) return __builtin_bit_cast(float, r[j]);
    const uint32_t w = r[j / 2];
    if constexpr (DT == DT_BF16) return __builtin_bit_cast(float, j & 1 ? w & 0xffff0000u : w << 16);
    return half_bits_to_float(j & 1 ? w >> 16 : w & 0xffffu);
}
template <int DT>
__device__ __forceinline__ uint32_t low_bits() {  // -inf, as a register of logits
    return DT == DT_F32 ? 0xff800000u : DT == DT_BF16 ? 0xff80ff80u : 0xfc00fc00u;
}

// A part of a row: its maximum and its sums about it.
struct Sums {
    float m, z, e;
};

template <int THREADS>
struct Shared {
    static constexpr int WAVES = THREADS / 64;
    uint64_t cand[CAND_MAX];
    uint64_t top[TOP_MAX];  // sorted; 0: none
    int found, odd;          // candidates of the round; whether it has NaN
    uint32_t limit[WAVES];
    int count[WAVES];
    Sums sums[WAVES];
};

// Maximum over the wave, in every lane.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));   // quad_perm 1,0,3,2
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));   // quad_perm 2,3,0,1
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xF, 0xF, false));  // row_ror:4
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, false));  // row_ror:8
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    const uint32_t a0 = a[0], a1 = a[1];
    v = max(a0, a1);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    const uint32_t b0 = b[0], b1 = b[1];
    return max(b0, b1);
}

// The n-th largest of the wave's 64 values, equal ones counted one by one: at
// least n lanes hold it or more.
__device__ __forceinline__ uint32_t nth_of_wave(uint32_t u, int n) {
    for (;;) {
        const uint32_t t = wave_max_u32(u);
        const int c = __popcll(__ballot(u == t));
        if (c >= n || t == 0u) return t;
        n -= c;
        u = u == t ? 0u : u;
    }
}

template <int THREADS>
__device__ __forceinline__ int block_count(Shared<THREADS>& sh, int wave_count) {
    const int wave = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh.count[wave] = wave_count;
    __syncthreads();
    int c = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) c += sh.count[w];
    return c;
}

// Keeps the compiler from holding what it made of the logits (as many values
// again, or twice) until they are next used.
template <int REGS>
__device__ __forceinline__ void fresh(uint32_t (&r)[REGS]) {
#pragma unroll
    for (int k = 0; k < REGS; ++k) asm volatile("" : "+v"(r[k]));
}

// Puts into sh.cand the topn largest of the n logits at x (ids from `first`
// on) exactly, whatever their number of equals: the topn-th largest is found
// bit by bit, and among its equals the last id that still belongs.  The slow
// way, for rows of ties: it reads the logits again for every bit.
template <int DT, int THREADS>
__device__ __forceinline__ int exact_top(Shared<THREADS>& sh, const uint8_t* x, int first, int n, int topn) {
    constexpr int SIZE = Logits<DT>::SIZE;
    const int tid = threadIdx.x, want = topn < n ? topn : n;
    const auto count = [&](uint32_t from, uint32_t to, int below) {  // logits of order [from, to], ids below
        int c = 0;
#pragma unroll 1
        for (int i = tid; i < n; i += THREADS) {
            const uint32_t u = order_of(load_one<DT>(x + (int64_t)i * SIZE));
            c += u >= from && u <= to && i < below ? 1 : 0;
        }
        return block_count(sh, (int)wave_sum_dpp((float)c));  // at most 2^16 a wave: exact
    };
    uint32_t v = 0;
#pragma unroll 1
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t t = v | 1u << bit;
        if (count(t, 0xffffffffu, n) >= want) v = t;
    }
    const int above = v == 0xffffffffu ? 0 : count(v + 1, 0xffffffffu, n);
    int last = 0;  // the largest number of first ids that do not hold enough of the equals
#pragma unroll 1
    for (int bit = 16; bit >= 0; --bit)
        if (above + count(v, v, last + (1 << bit)) < want) last += 1 << bit;
    __syncthreads();
    if (tid == 0) sh.count[0] = 0;
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < n; i += THREADS) {
        const uint32_t u = order_of(load_one<DT>(x + (int64_t)i * SIZE));
        if (u > v || (u == v && i <= last)) sh.cand[atomicAdd(&sh.count[0], 1)] = key_of(u, first + i);
    }
    __syncthreads();
    return want;
}

// Renews sh.top with a round's n logits (at x, ids from `first` on), of which
// thread t holds ids (j / N * THREADS + t) * N + j % N of the round and, of the
// n % N behind the last whole load, the t-th (`rest`, else -inf); `own`: its
// largest; `odd`: some thread's are NaN.
template <int DT, int THREADS>
__device__ __forceinline__ void renew_top(Shared<THREADS>& sh, uint32_t (&r)[Logits<DT>::REGS], float rest, float own,
                                          bool odd,
                                          const uint8_t* x, int first, int n, int topn) {
    using L = Logits<DT>;
    constexpr int WAVES = THREADS / 64;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // A lower limit of the result: what `most` lanes of each of `waves` waves
    // reach, most * waves >= topn (a list of 20 from 16 waves gets some 45
    // candidates from the fifth of the waves' fourth), or the list's last so
    // far.  Above -inf: where there are not topn finite logits,
    // those of -inf that fill the list are among the round's first topn ids.
    const uint32_t low = order_of(-INFINITY);
    int most = (topn + WAVES - 1) / WAVES;
    while (most * most < topn) ++most;
    const int waves = (topn + most - 1) / most;
    uint32_t limit = nth_of_wave(order_of(own), most);
    if (lane == 0) sh.limit[wave] = limit;
    if (tid == 0) sh.found = 0;
    if (odd) sh.odd = first + 1;
    __syncthreads();
    limit = nth_of_wave(lane < WAVES ? sh.limit[lane] : 0u, waves);
    limit = max(max(low + 1, limit), (uint32_t)(sh.top[topn - 1] >> 32));
    // every logit that reaches it is a candidate: one bit each, the first
    // logit's the highest (read again by those few threads that have any)
    const float f = logit_of(limit);
    if (own >= f) {
        uint32_t bits = 0;
        fresh(r);
#pragma unroll
        for (int j = 0; j < PER; ++j) bits = bits + bits + (logit_at<DT>(r, j) >= f ? 1u : 0u);
        const int mine = __popc(bits) + (rest >= f ? 1 : 0);
        int at = atomicAdd(&sh.found, mine);
        if (at + mine <= CAND_MAX - 2 * TOP_MAX) {
            if (rest >= f) sh.cand[at++] = key_of(order_of(rest), first + n / L::N * L::N + tid);
            while (bits) {
                const int j = __clz(bits), id = (j / L::N * THREADS + tid) * L::N + j % L::N;
                bits &= ~(0x80000000u >> j);
                sh.cand[at++] = key_of(order_of(load_one<DT>(x + (uint32_t)(id * L::SIZE))), first + id);
            }
        }
    }
    __syncthreads();
    int total = sh.found;
    if (sh.odd == first + 1 || total > CAND_MAX - 2 * TOP_MAX) {
        total = exact_top<DT, THREADS>(sh, x, first, n, topn);
    } else if (total < topn) {
        if (total == 0 && sh.top[topn - 1] != 0) {  // nothing for a full list
            __syncthreads();
            return;
        }
        if (tid < topn) {
            // 0: a candidate already, or not a logit
            const float v = tid < n ? load_one<DT>(x + (int64_t)tid * L::SIZE) : 0.0f;
            sh.cand[total + tid] = tid < n && v == -INFINITY ? key_of(low, first + tid) : 0;
        }
        total += topn;
    }
    // the list so far is among the candidates too
    if (tid < topn) sh.cand[total + tid] = sh.top[tid];
    total += topn;
    __syncthreads();
    // A candidate's rank: the number of larger ones, counted by PARTS threads,
    // every PARTS-th candidate each.
    int parts = THREADS / 64;
    while (parts > 1 && THREADS / parts < total) parts >>= 1;
    for (int c0 = 0; c0 < total; c0 += THREADS / parts) {
        const int c = c0 + tid / parts;
        const uint64_t one = c < total ? sh.cand[c] : 0;
        int rank = 0;
        for (int i = tid % parts; i < total; i += parts) rank += sh.cand[i] > one ? 1 : 0;
        for (int off = parts >> 1; off > 0; off >>= 1) rank += __shfl_xor(rank, off, WAVE);
        if (tid % parts == 0 && one != 0 && rank < topn) sh.top[rank] = one;
    }
    __syncthreads();
}

// One logit, d below the maximum m: z = sum e^d, e = sum e^d d.  (0 * -inf of
// one that is -inf is kept from the second sum; a NaN stays one in both.)
__device__ __forceinline__ void add_logit(float d, float& z, float& e) {
    const float p = __builtin_amdgcn_exp2f(d * LOG2E);
    z += p;
    e = __builtin_fmaf(p, fmaxf(d, -1e4f), e);
}
// Sums about a maximum as sums about a larger one, d = the first minus the second.
__device__ __forceinline__ void shift_sums(float d, float& z, float& e) {
    const float f = __builtin_amdgcn_exp2f(d * LOG2E);
    e = f * (e + fmaxf(d, -1e4f) * z);
    z *= f;
}
// The lanes' parts as one, in every lane.
__device__ __forceinline__ Sums wave_join(Sums s) {
    Sums t;
    float m = s.m;
#pragma unroll
    for (int k = 0; k < 4; ++k) m = fmaxf(m, dpp_f(m, k));
    m = fmaxf(m, __shfl_xor(m, 16, WAVE));
    t.m = fmaxf(m, __shfl_xor(m, 32, WAVE));
    if (s.m != -INFINITY) shift_sums(s.m - t.m, s.z, s.e);
    t.z = wave_sum_dpp(s.z);
    t.e = wave_sum_dpp(s.e);
    return t;
}
// What a row's sums say.
struct Row {
    float lse, entropy;
    bool empty;  // every logit is -inf
};
__device__ __forceinline__ Row row_of(const Sums& s) {
    Row r;
    r.empty = s.z == 0.0f;
    const float lz = logf(s.z);
    r.lse = r.empty ? -INFINITY : s.m + lz;
    r.entropy = r.empty ? 0.0f : lz - s.e / s.z;
    return r;
}
// The target's logit (NaN: none), read before anything waits for it.
template <int DT>
__device__ __forceinline__ float target_logit(const LogProbs& a, int64_t row) {
    const int t = a.logprob ? a.targets[row] : -1;
    return t >= 0 && t < a.V ? load_one<DT>(static_cast<const uint8_t*>(a.x) + (row * a.stride + t) * Logits<DT>::SIZE)
                             : __builtin_nanf("");
}
__device__ __forceinline__ void store_row(const LogProbs& a, int64_t row, const Row& r, float target) {
    if (a.logprob) a.logprob[row] = r.empty && target == target ? -INFINITY : target - r.lse;
    if (a.entropy) a.entropy[row] = r.entropy;
    if (a.lse) a.lse[row] = r.lse;
}
__device__ __forceinline__ void store_top(const LogProbs& a, int64_t row, const Row& r, int i, uint64_t k) {
    a.top_ids[row * a.topn + i] = id_of(k);
    a.top_logprob[row * a.topn + i] = r.empty ? -INFINITY : logit_of((uint32_t)(k >> 32)) - r.lse;
}

// Parts of rows in the workspace: Sums [T][parts], then keys [T][parts][topn].
struct Parts {
    Sums* sums;
    uint64_t* keys;
    int parts, length;  // a part's logits, a multiple of 16
};

// One workgroup a row, or (SPLIT) a row's part.
template <int DT, int THREADS, bool SPLIT>
__global__ __launch_bounds__(THREADS, 8) void logprobs_kernel(LogProbs a, Parts parts) {
    using L = Logits<DT>;
    constexpr int WAVES = THREADS / 64, ROUND = THREADS * PER;
    __shared__ Shared<THREADS> sh;
    const int64_t row = SPLIT ? blockIdx.x / parts.parts : blockIdx.x;
    const int part = SPLIT ? (int)(blockIdx.x % parts.parts) : 0;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int from = SPLIT ? part * parts.length : 0;
    const int to = SPLIT && from + parts.length < a.V ? from + parts.length : (int)a.V;
    const uint8_t* x = static_cast<const uint8_t*>(a.x) + row * a.stride * L::SIZE;
    if (tid < TOP_MAX) sh.top[tid] = 0;
    if (tid == 0) sh.odd = 0;
    float target = 0.0f;
    // a thread's own maximum, and its sums about it
    float m = -INFINITY, z = 0.0f, e = 0.0f;
    for (int first = from; first < to; first += ROUND) {
        const int n = to - first < ROUND ? to - first : ROUND;
        uint32_t r[L::REGS];
#pragma unroll
        for (int k = 0; k < L::REGS / 4; ++k) {
            const int i = (k * THREADS + tid) * L::N;
            if (i + L::N <= n) {
                const u4_t w = __builtin_nontemporal_load(
                    reinterpret_cast<const u4_any*>(x + (uint32_t)((first + i) * L::SIZE)));
                r[4 * k] = w[0], r[4 * k + 1] = w[1], r[4 * k + 2] = w[2], r[4 * k + 3] = w[3];
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) r[4 * k + j] = low_bits<DT>();
            }
        }
        const int whole = n / L::N * L::N;
        const float rest = whole + tid < n ? load_one<DT>(x + (uint32_t)((first + whole + tid) * L::SIZE)) : -INFINITY;
        float own = rest;
#pragma unroll
        for (int j = 0; j < PER; ++j) own = fmaxf(own, logit_at<DT>(r, j));
        fresh(r);
        if (own > m) {
            if (m != -INFINITY) shift_sums(m - own, z, e);
            m = own;
        }
        const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            add_logit(logit_at<DT>(r, j) - base, z, e);
            if (j % 4 == 3) asm volatile("" : "+v"(z), "+v"(e));  // four at a time in registers
        }
        add_logit(rest - base, z, e);
        if (first + ROUND >= to) {  // the wave's sums; the target's logit, on its way over the selection
            if (!SPLIT && wave == 0) target = target_logit<DT>(a, row);
            const Sums w = wave_join(Sums{m, z, e});
            if (lane == 0) sh.sums[wave] = w;
        }
        __syncthreads();
        if (a.topn > 0) {
            renew_top<DT, THREADS>(sh, r, rest, own, z != z, x + (int64_t)first * L::SIZE, first, n, a.topn);
        }
    }
    if (wave != 0) return;
    const Sums w = lane < WAVES ? sh.sums[lane] : Sums{-INFINITY, 0.0f, 0.0f};
    const Sums t = wave_join(w);
    if (SPLIT) {
        const int64_t at = row * parts.parts + part;
        if (tid == 0) parts.sums[at] = t;
        if (tid < a.topn) parts.keys[at * a.topn + tid] = sh.top[tid];
    } else {
        const Row r = row_of(t);
        if (tid == 0) store_row(a, row, r, target);
        if (tid < a.topn) store_top(a, row, r, tid, sh.top[tid]);
    }
}

// A row's parts, one wave a row.  Lane p holds part p's sums; of the parts'
// lists, those that reach what `most` of each of `some` lists reach.
constexpr int PARTS_MAX = 16;
template <int DT>
__global__ __launch_bounds__(64) void logprobs_join_kernel(LogProbs a, Parts parts) {
    __shared__ uint64_t cand[PARTS_MAX * TOP_MAX];
    __shared__ int found;
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x, P = parts.parts, n = a.topn;
    Sums s{-INFINITY, 0.0f, 0.0f};
    if (lane < P) s = parts.sums[row * P + lane];
    const float target = target_logit<DT>(a, row);
    const uint64_t* keys = parts.keys + row * P * n;
    int most = 1;
    while (most * most < n || most * P < n) ++most;
    const int some = (n + most - 1) / most;
    uint64_t own[PARTS_MAX * TOP_MAX / 64];
    uint64_t mark = 0;
    if (n > 0) {
        if (lane < P) mark = keys[lane * n + most - 1];
#pragma unroll
        for (int i = 0; i < PARTS_MAX * TOP_MAX / 64; ++i) own[i] = i * 64 + lane < P * n ? keys[i * 64 + lane] : 0;
    }
    if (lane == 0) found = 0;
    const Row r = row_of(wave_join(s));
    if (lane == 0) store_row(a, row, r, target);
    if (n == 0) return;
    const uint32_t limit = nth_of_wave((uint32_t)(mark >> 32), some);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PARTS_MAX * TOP_MAX / 64; ++i)
        if (own[i] != 0 && (uint32_t)(own[i] >> 32) >= limit) cand[atomicAdd(&found, 1)] = own[i];
    __syncthreads();
    const int total = found;
    for (int c = lane; c < total; c += 64) {
        const uint64_t one = cand[c];
        int rank = 0;
        for (int i = 0; i < total; ++i) rank += cand[i] > one ? 1 : 0;
        if (rank < n) store_top(a, row, r, rank, one);
    }
}

// Parts of a row: none where a workgroup holds it in one round (the join's
// launch costs more than it saves: 1 x 32000 logits, 8 us whole), else enough
// for a workgroup a compute unit, of a quarter of a round at least.  Of 128257 bf16
// logits, top 20: 64 rows take 15.9 us (with parts for two workgroups a compute unit
// 20.6), 100 23.3 (20.3), 128 23.7 (21.2), and from 129 on, whole, 34.2 (30.9), 256
// 35.3 (33.1): a step at 129 rows, where half of the units have no row.
Parts parts_of(void* ws, int64_t T, int64_t V) {
    constexpr int64_t ROUND = 1024 * PER;
    Parts p{nullptr, nullptr, 1, 0};
    if (T < 1 || V <= ROUND) return p;
    int64_t n = 256 / T, most = (V + ROUND / 4 - 1) / (ROUND / 4);
    n = n < most ? n : most;
    p.parts = (int)(n < 1 ? 1 : n < PARTS_MAX ? n : PARTS_MAX);
    p.length = (int)((V + p.parts - 1) / p.parts + 15) / 16 * 16;
    p.sums = static_cast<Sums*>(ws);
    p.keys = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(ws) + align256((int64_t)sizeof(Sums) * T * p.parts));
    return p;
}

// Threads that hold a row of V logits in one round, if 256 do, else 1024.
int threads_of(int64_t V) { return V <= 256 * PER ? 256 : 1024; }

template <int DT>
hipError_t logprobs_dt(const LogProbs& a, void* ws, hipStream_t s) {
    const Parts p = parts_of(ws, a.T, a.V);
    if (p.parts > 1) {
        Q8K_LAUNCH((logprobs_kernel<DT, 1024, true>), dim3((unsigned)(a.T * p.parts)), dim3(1024), 0, s, a, p);
        Q8K_LAUNCH(logprobs_join_kernel<DT>, dim3((unsigned)a.T), dim3(64), 0, s, a, p);
    } else if (threads_of(a.V) == 256) {
        Q8K_LAUNCH((logprobs_kernel<DT, 256, false>), dim3((unsigned)a.T), dim3(256), 0, s, a, p);
    } else {
        Q8K_LAUNCH((logprobs_kernel<DT, 1024, false>), dim3((unsigned)a.T), dim3(1024), 0, s, a, p);
    }
    return hipGetLastError();
}

}  // namespace

int64_t logprobs_ws_bytes(int64_t T, int64_t V, int topn) {
    const Parts p = parts_of(nullptr, T, V);
    return p.parts > 1 ? align256((int64_t)sizeof(Sums) * T * p.parts) + 8 * T * p.parts * topn : 0;
}

int64_t logprobs_threads(int64_t T, int64_t V) { return (int64_t)parts_of(nullptr, T, V).parts * threads_of(V); }

hipError_t launch_logprobs(const LogProbs& a, void* ws, hipStream_t s) {
    return a.dtype == DT_F32   ? logprobs_dt<DT_F32>(a, ws, s)
           : a.dtype == DT_F16 ? logprobs_dt<DT_F16>(a, ws, s)
                               : logprobs_dt<DT_BF16>(a, ws, s);
}

}  // namespace q8k
