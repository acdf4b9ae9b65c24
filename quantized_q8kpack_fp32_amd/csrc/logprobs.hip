// Log probabilities of given tokens, the entropy of each row of logits and its
// top alternatives, in one pass over the logits.
//
//   m = max x, Z = sum e^(x - m), lse = m + log Z
//   logprob = x[target] - lse,  entropy = log Z - sum e^(x - m) (x - m) / Z
//   top: the topn largest, by (logit descending, id ascending)
//
// Bound by reading the logits once.  A row is cut into chunks of CHUNK logits,
// one workgroup each, which holds its chunk in registers: the maximum, the two
// sums and the chunk's own top list come from there.  A second launch joins a
// row's chunks.
#include "kv_cache.h"
#include "q8k_launch.h"

namespace q8k {

namespace {

constexpr int THREADS = 256;
constexpr int PER = 32;                // logits a thread
constexpr int CHUNK = THREADS * PER;   // logits a workgroup
constexpr int TOP_MAX = 32;

// A logit and its id as one integer that orders as (logit, -id) does: distinct
// for every id, so that "larger" leaves no ties.  -0 counts as 0; a NaN is
// below every number.  0 is no logit's key.
__device__ __forceinline__ uint64_t key_of(float x, int id) {
    uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);
    u = (u & 0x80000000u) ? ~u : u | 0x80000000u;
    if (x != x) u = 0;
    return (uint64_t)u << 32 | (uint32_t)~(uint32_t)id;
}
__device__ __forceinline__ int id_of(uint64_t k) { return (int)~(uint32_t)k; }
__device__ __forceinline__ float logit_of(uint64_t k) {
    const uint32_t u = (uint32_t)(k >> 32);
    if (u == 0) return __builtin_nanf("");
    return __builtin_bit_cast(float, (u & 0x80000000u) ? u & 0x7fffffffu : ~u);
}

struct Sums {
    float m, z, e;  // maximum, sum of e^(x - m), sum of e^(x - m) (x - m)
};

// Chunk results in the workspace: Sums [T][C], then keys [T][C][topn].
struct Ws {
    Sums* sums;
    uint64_t* keys;
    int chunks;
};
__host__ __device__ inline int64_t chunks_of(int64_t V) { return (V + CHUNK - 1) / CHUNK; }

// Loads 16 bytes of logits at any element's address.
template <int DT>
struct Vec {
    static constexpr int N = DT == DT_F32 ? 4 : 8;
};
struct __attribute__((packed, aligned(2))) Bytes16 {
    uint32_t w[4];
};
template <int DT>
__device__ __forceinline__ void load_vec(const uint8_t* p, float (&v)[Vec<DT>::N]) {
    const Bytes16 b = *reinterpret_cast<const Bytes16*>(p);
    if constexpr (DT == DT_F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = b.w[i];
            v[i] = __builtin_bit_cast(float, w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = b.w[i];
            v[2 * i] = DT == DT_BF16 ? __builtin_bit_cast(float, w << 16) : half_bits_to_float(w & 0xffffu);
            v[2 * i + 1] = DT == DT_BF16 ? __builtin_bit_cast(float, w & 0xffff0000u) : half_bits_to_float(w >> 16);
        }
    }
}
template <int DT>
__device__ __forceinline__ float load_one(const uint8_t* p) {
    if constexpr (DT == DT_F32) return *reinterpret_cast<const float*>(p);
    const uint32_t w = *reinterpret_cast<const uint16_t*>(p);
    return DT == DT_BF16 ? __builtin_bit_cast(float, w << 16) : half_bits_to_float(w);
}

__device__ __forceinline__ uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }

// The topn largest of the keys that the workgroup's threads hold in their
// registers (0: none), sorted, to out(rank, key); ranks beyond the keys there
// are get key 0.  The topn-th largest of the threads' own largest keys is a
// lower limit of the result, and only topn threads hold keys that reach it:
// these are counted out against each other.  `holders`: threads before it hold
// every key.
struct TopShared {
    uint64_t best[THREADS];
    uint64_t cand[TOP_MAX * PER];
    uint64_t limit;
    int count;
};
template <int M, class Out>
__device__ __forceinline__ void select_top(TopShared& sh, const uint64_t (&key)[M], int holders, int topn, Out out) {
    const int tid = threadIdx.x;
    uint64_t best = key[0];
#pragma unroll
    for (int k = 1; k < M; ++k) best = max_u64(best, key[k]);
    sh.best[tid] = best;
    if (tid == 0) {
        sh.count = 0;
        sh.limit = 1;  // fewer holders than topn: every key is a candidate
    }
    __syncthreads();
    int rank = 0;
    for (int i = 0; i < holders; ++i) rank += sh.best[i] > best;
    if (tid < holders && best != 0 && rank == topn - 1) sh.limit = best;
    __syncthreads();
    const uint64_t limit = sh.limit;
    if (best >= limit) {
#pragma unroll
        for (int k = 0; k < M; ++k)
            if (key[k] >= limit) sh.cand[atomicAdd(&sh.count, 1)] = key[k];
    }
    __syncthreads();
    const int n = sh.count;
    for (int c = tid; c < n; c += THREADS) {
        const uint64_t mine = sh.cand[c];
        int r = 0;
        for (int i = 0; i < n; ++i) r += sh.cand[i] > mine;
        if (r < topn) out(r, mine);
    }
    for (int r = n + tid; r < topn; r += THREADS) out(r, (uint64_t)0);
}

template <int DT>
__global__ __launch_bounds__(THREADS) void logprobs_chunk_kernel(LogProbs a, Ws ws) {
    constexpr int N = Vec<DT>::N, SIZE = DT == DT_F32 ? 4 : 2;
    __shared__ float red[3][THREADS / 64];
    __shared__ TopShared top;
    const int64_t row = blockIdx.x / ws.chunks;
    const int chunk = (int)(blockIdx.x % ws.chunks), tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t first = (int64_t)chunk * CHUNK;
    const int n = (int)(a.V - first < CHUNK ? a.V - first : CHUNK);
    const uint8_t* src = static_cast<const uint8_t*>(a.x) + (row * a.stride + first) * SIZE;
    // thread t's k-th vector starts at logit (k * THREADS + t) * N of the chunk
    float v[PER];
#pragma unroll
    for (int k = 0; k < PER / N; ++k) {
        const int i = (k * THREADS + tid) * N;
        float t[N];
        if (i + N <= n) {
            load_vec<DT>(src + (int64_t)i * SIZE, t);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) t[j] = i + j < n ? load_one<DT>(src + (int64_t)(i + j) * SIZE) : -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < N; ++j) v[k * N + j] = t[j];
    }
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < PER; ++k) m = fmaxf(m, v[k]);
    m = wave_max(m);
    if (lane == 0) red[0][wave] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    const float base = m == -INFINITY ? 0.0f : m;
    float z = 0.0f, e = 0.0f;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const float d = v[k] - base, x = __expf(d);
        z += x;
        e += v[k] == -INFINITY ? 0.0f : x * d;
    }
    z = wave_sum_dpp(z);
    e = wave_sum_dpp(e);
    if (lane == 0) red[1][wave] = z, red[2][wave] = e;
    if (a.topn > 0) {
        uint64_t key[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = ((k / N) * THREADS + tid) * N + k % N;
            key[k] = i < n ? key_of(v[k], (int)(first + i)) : 0;
        }
        uint64_t* out = ws.keys + (row * ws.chunks + chunk) * a.topn;
        const int holders = (n + N - 1) / N < THREADS ? (n + N - 1) / N : THREADS;
        select_top(top, key, holders, a.topn, [&](int r, uint64_t k) { out[r] = k; });
    }
    __syncthreads();
    if (tid == 0) {
        Sums s;
        s.m = m;
        s.z = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
        s.e = (red[2][0] + red[2][1]) + (red[2][2] + red[2][3]);
        ws.sums[row * ws.chunks + chunk] = s;
    }
}

// One workgroup a row: every wave joins the chunks' sums (at most CHUNKS_MAX,
// in an order that does not change), then all select from the chunks' lists.
constexpr int CHUNKS_MAX = 128;
template <int DT>
__global__ __launch_bounds__(THREADS) void logprobs_join_kernel(LogProbs a, Ws ws) {
    constexpr int SIZE = DT == DT_F32 ? 4 : 2, HELD = CHUNKS_MAX * TOP_MAX / THREADS;
    static_assert(HELD <= PER, "candidates fit");
    __shared__ TopShared top;
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63;
    const Sums* sums = ws.sums + row * ws.chunks;
    const Sums none{-INFINITY, 0.0f, 0.0f};
    const Sums s0 = lane < ws.chunks ? sums[lane] : none, s1 = lane + 64 < ws.chunks ? sums[lane + 64] : none;
    const float m = wave_max(fmaxf(s0.m, s1.m));
    const float base = m == -INFINITY ? 0.0f : m;
    const float d0 = s0.m == -INFINITY ? 0.0f : s0.m - base, d1 = s1.m == -INFINITY ? 0.0f : s1.m - base;
    const float f0 = __expf(d0), f1 = __expf(d1);
    const float z = wave_sum_dpp(f0 * s0.z + f1 * s1.z);
    const float e = wave_sum_dpp(f0 * (s0.e + d0 * s0.z) + f1 * (s1.e + d1 * s1.z));
    const bool empty = z == 0.0f;  // every logit is -inf
    const float logz = logf(z), lse = empty ? -INFINITY : base + logz;
    if (tid == 0) {
        if (a.logprob) {
            const int t = a.targets[row];
            float lp = __builtin_nanf("");
            if (t >= 0 && t < a.V) {
                const float xt =
                    load_one<DT>(static_cast<const uint8_t*>(a.x) + (row * a.stride + t) * SIZE);
                lp = empty ? -INFINITY : xt - lse;
            }
            a.logprob[row] = lp;
        }
        if (a.entropy) a.entropy[row] = empty ? 0.0f : logz - e / z;
        if (a.lse) a.lse[row] = lse;
    }
    if (a.topn > 0) {
        const int n = ws.chunks * a.topn;
        const uint64_t* keys = ws.keys + row * n;
        uint64_t key[HELD];
#pragma unroll
        for (int k = 0; k < HELD; ++k) key[k] = k * THREADS + tid < n ? keys[k * THREADS + tid] : 0;
        select_top(top, key, n < THREADS ? n : THREADS, a.topn, [&](int r, uint64_t k) {
            a.top_ids[row * a.topn + r] = id_of(k);
            a.top_logprob[row * a.topn + r] = empty ? -INFINITY : logit_of(k) - lse;
        });
    }
}

Ws ws_of(void* ws, int64_t T, int64_t V) {
    Ws w;
    w.chunks = (int)chunks_of(V);
    w.sums = static_cast<Sums*>(ws);
    w.keys = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(ws) + align256(sizeof(Sums) * T * w.chunks));
    return w;
}

template <int DT>
hipError_t logprobs_dt(const LogProbs& a, void* p, hipStream_t s) {
    const Ws ws = ws_of(p, a.T, a.V);
    Q8K_LAUNCH(logprobs_chunk_kernel<DT>, dim3((unsigned)(a.T * ws.chunks)), dim3(THREADS), 0, s, a, ws);
    Q8K_LAUNCH(logprobs_join_kernel<DT>, dim3((unsigned)a.T), dim3(THREADS), 0, s, a, ws);
    return hipGetLastError();
}

}  // namespace

int64_t logprobs_ws_bytes(int64_t T, int64_t V, int topn) {
    const int64_t c = chunks_of(V);
    return align256(sizeof(Sums) * T * c) + 8 * T * c * topn;
}

hipError_t launch_logprobs(const LogProbs& a, void* ws, hipStream_t s) {
    return a.dtype == DT_F32   ? logprobs_dt<DT_F32>(a, ws, s)
           : a.dtype == DT_F16 ? logprobs_dt<DT_F16>(a, ws, s)
                               : logprobs_dt<DT_BF16>(a, ws, s);
}

}  // namespace q8k
