// C ABI of libq8k: argument validation, sizing helpers and dispatch to the
// gfx950 kernels.  Every refusal is named and enqueues nothing (the launch
// checks with named reasons of "One kernel, any device", section 1; the
// 256-multiple width rule of "Language models on the device: the cajeta-llm
// kernels", section 3.2).  Validation touches no HIP API, so refusals work on
// a machine without a GPU.
#include <stdarg.h>
#include <stdio.h>

#include "../../include/q8k.h"
#include "kv4_cache.h"
#include "q8k_launch.h"

using namespace q8k;

namespace {

thread_local char g_err[512] = "";

// The launch record of the calling thread's last operation (test support: the
// kernel census).  Every operation clears it first; each launch appends its
// kernel's host handle.
constexpr int LAUNCH_RECORD_MAX = 16;
thread_local const void* g_launched[LAUNCH_RECORD_MAX];
thread_local int g_nlaunched = 0;
void begin_call() { g_nlaunched = 0; }

int fail(int status, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof(g_err), fmt, ap);
    va_end(ap);
    return status;
}

// Sizes are kept well inside int32 block counts per row and 2^31 rows so that
// grid sizes and per-row indexing cannot overflow.
constexpr int64_t MAX_ROWS = (int64_t)1 << 30;
constexpr int64_t MAX_K = (int64_t)1 << 24;
constexpr int64_t MAX_TOKENS = (int64_t)1 << 24;
constexpr int64_t MAX_EXPERTS = 4096;
static_assert(MAX_EXPERTS <= MOE_GROUP_MAX_E, "the MoE prefill groups pairs of at most MOE_GROUP_MAX_E experts");

// Every launch uses a 1-D grid of at most 2^31 - 1 workgroups.
constexpr int64_t MAX_GRID = ((int64_t)1 << 31) - 1;

int check_grid(const char* fn, int64_t workgroups) {
    if (workgroups > MAX_GRID)
        return fail(Q8K_ERR_SHAPE, "%s: problem needs %lld workgroups (at most %lld)", fn, (long long)workgroups,
                    (long long)MAX_GRID);
    return Q8K_OK;
}

// A launch counts its threads in 32 bits.
int check_threads(const char* fn, int64_t workgroups, int64_t threads) {
    if (workgroups > (int64_t)0xffffffff / threads)
        return fail(Q8K_ERR_SHAPE, "%s: problem needs %lld workgroups of %lld threads (fewer than 2^32 threads in all)",
                    fn, (long long)workgroups, (long long)threads);
    return Q8K_OK;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int check_k(const char* fn, int64_t K) {
    if (K <= 0 || K % QK != 0 || K > MAX_K)
        return fail(Q8K_ERR_SHAPE, "%s: K=%lld must be a positive multiple of 256 (at most %lld)", fn, (long long)K,
                    (long long)MAX_K);
    return Q8K_OK;
}

int check_count(const char* fn, const char* what, int64_t v, int64_t maxv) {
    if (v < 0 || v > maxv)
        return fail(Q8K_ERR_SHAPE, "%s: %s=%lld out of range [0, %lld]", fn, what, (long long)v, (long long)maxv);
    return Q8K_OK;
}

int check_ptr(const char* fn, const char* what, const void* p, size_t align) {
    if (!p) return fail(Q8K_ERR_NULL, "%s: %s is NULL", fn, what);
    if (!aligned(p, align))
        return fail(Q8K_ERR_ALIGN, "%s: %s=%p is not %zu-byte aligned", fn, what, p, align);
    return Q8K_OK;
}

Acts acts_of(const void* xq, int64_t T, int64_t K) {
    const ActLayout l = act_layout(T, K);
    const uint8_t* base = static_cast<const uint8_t*>(xq);
    Acts a;
    a.qs = reinterpret_cast<const int8_t*>(base);
    a.d = reinterpret_cast<const float*>(base + l.off_d);
    a.bs = reinterpret_cast<const int16_t*>(base + l.off_bs);
    a.K = K;
    return a;
}

struct Q6View {
    const uint16_t* prefix;
    const uint8_t* bodies;
};
Q6View q6_view(const void* w, int64_t nblocks) {
    const uint8_t* base = static_cast<const uint8_t*>(w);
    return Q6View{reinterpret_cast<const uint16_t*>(base), base + align256(2 * (size_t)nblocks)};
}

int launched(const char* fn, hipError_t e) {
    if (e != hipSuccess) return fail(Q8K_ERR_LAUNCH, "%s: launch failed: %s", fn, hipGetErrorString(e));
    return Q8K_OK;
}

#define Q8K_TRY(x)                    \
    do {                              \
        int _st = (x);                \
        if (_st != Q8K_OK) return _st; \
    } while (0)

// Every operation serves Q4_K, Q5_K and relaid Q6_K weights.
int check_weight(const char* fn, int qtype, const void* w) {
    if (qtype == Q8K_Q4_K || qtype == Q8K_Q5_K || qtype == Q8K_Q6_K_RELAID) return check_ptr(fn, "w", w, 16);
    if (qtype == Q8K_Q6_K_GGUF)
        return fail(Q8K_ERR_QTYPE, "%s: raw GGUF Q6_K must be bound first (q8k_bind_q6k -> Q8K_Q6_K_RELAID)", fn);
    return fail(Q8K_ERR_QTYPE, "%s: qtype=%d not served here (use Q8K_Q4_K=1, Q8K_Q6_K_RELAID=2 or Q8K_Q5_K=4)", fn,
                qtype);
}

// The prefill tile's format index and weight streams (Q6_K: bodies and prefix).
struct PrefillWeights {
    int fmt;
    const uint8_t* w;
    const uint16_t* prefix;
};
PrefillWeights prefill_weights(int qtype, const void* w, int64_t nblocks) {
    if (qtype == Q8K_Q6_K_RELAID) {
        const Q6View v = q6_view(w, nblocks);
        return PrefillWeights{WFMT_Q6_K, v.bodies, v.prefix};
    }
    return PrefillWeights{qtype == Q8K_Q5_K ? WFMT_Q5_K : WFMT_Q4_K, static_cast<const uint8_t*>(w), nullptr};
}

}  // namespace

void q8k::note_launch(const void* kernel) {
    if (g_nlaunched < LAUNCH_RECORD_MAX) g_launched[g_nlaunched] = kernel;
    ++g_nlaunched;  // counts past the record's end too, so an overflow is visible
}

extern "C" {

size_t q8k_act_layout(int64_t T, int64_t K, size_t* off_d, size_t* off_bsums) {
    if (T < 0 || K <= 0 || K % QK != 0) return 0;
    const ActLayout l = act_layout(T, K);
    if (off_d) *off_d = l.off_d;
    if (off_bsums) *off_bsums = l.off_bs;
    return l.total;
}

size_t q8k_act_bytes(int64_t T, int64_t K) { return q8k_act_layout(T, K, nullptr, nullptr); }

size_t q8k_weight_bytes(int qtype, int64_t rows, int64_t K) {
    if (rows < 0 || K <= 0 || K % QK != 0) return 0;
    const size_t nblk = (size_t)rows * (size_t)(K / QK);
    switch (qtype) {
        case Q8K_Q4_K: return nblk * Q4K_BLOCK;
        case Q8K_Q5_K: return nblk * Q5K_BLOCK;
        case Q8K_Q6_K_GGUF: return nblk * Q6K_BLOCK;
        case Q8K_Q6_K_RELAID: return align256(2 * nblk) + nblk * Q6K_BODY;
        default: return 0;
    }
}

int q8k_pack(const float* x, int64_t T, int64_t K, void* xq, void* stream) {
    begin_call();
    const char* fn = "q8k_pack";
    Q8K_TRY(check_k(fn, K));
    Q8K_TRY(check_count(fn, "T", T, MAX_TOKENS));
    Q8K_TRY(check_ptr(fn, "x", x, 16));
    Q8K_TRY(check_ptr(fn, "xq", xq, 16));
    Q8K_TRY(check_grid(fn, (T * (K / QK) + 15) / 16));  // 16 blocks per workgroup
    if (T == 0) return Q8K_OK;
    const ActLayout l = act_layout(T, K);
    uint8_t* base = static_cast<uint8_t*>(xq);
    return launched(fn, launch_pack(x, T * (K / QK), reinterpret_cast<int8_t*>(base),
                                    reinterpret_cast<float*>(base + l.off_d),
                                    reinterpret_cast<int16_t*>(base + l.off_bs), (hipStream_t)stream));
}

int q8k_bind_q6k(const void* w_gguf, int64_t rows, int64_t K, void* w_relaid, void* stream) {
    begin_call();
    const char* fn = "q8k_bind_q6k";
    Q8K_TRY(check_k(fn, K));
    Q8K_TRY(check_count(fn, "rows", rows, MAX_ROWS));
    Q8K_TRY(check_ptr(fn, "w_gguf", w_gguf, 2));
    Q8K_TRY(check_ptr(fn, "w_relaid", w_relaid, 16));
    Q8K_TRY(check_grid(fn, (rows * (K / QK) + 3) / 4));
    if (rows == 0) return Q8K_OK;
    const int64_t nblk = rows * (K / QK);
    uint8_t* base = static_cast<uint8_t*>(w_relaid);
    return launched(fn, launch_bind_q6k(static_cast<const uint8_t*>(w_gguf), nblk, reinterpret_cast<uint16_t*>(base),
                                        base + align256(2 * (size_t)nblk), (hipStream_t)stream));
}

static int matvec_common(const char* fn, int qtype, const void* w, int64_t rows, int64_t K, const void* xq,
                         int64_t ncols, float* y, void* stream) {
    Q8K_TRY(check_k(fn, K));
    Q8K_TRY(check_count(fn, "rows", rows, MAX_ROWS));
    Q8K_TRY(check_weight(fn, qtype, w));
    Q8K_TRY(check_ptr(fn, "xq", xq, 16));
    Q8K_TRY(check_ptr(fn, "y", y, 4));
    if (rows == 0) return Q8K_OK;
    const int nb = (int)(K / QK);
    const Acts a = acts_of(xq, ncols, K);
    hipError_t e;
    if (qtype == Q8K_Q4_K) {
        e = launch_matvec_q4k(static_cast<const uint8_t*>(w), rows, nb, a, (int)ncols, y, (hipStream_t)stream);
    } else if (qtype == Q8K_Q5_K) {
        e = launch_matvec_q5k(static_cast<const uint8_t*>(w), rows, nb, a, (int)ncols, y, (hipStream_t)stream);
    } else {
        const Q6View v = q6_view(w, rows * nb);
        e = launch_matvec_q6k(v.prefix, v.bodies, rows, nb, a, (int)ncols, y, (hipStream_t)stream);
    }
    return launched(fn, e);
}

int qmatvec_f32(int qtype, const void* w, int64_t rows, int64_t K, const float* x, int64_t ncols, float* y,
                void* xq_out, void* stream) {
    begin_call();
    const char* fn = "qmatvec_f32";
    Q8K_TRY(check_k(fn, K));
    Q8K_TRY(check_count(fn, "rows", rows, MAX_ROWS));
    if (ncols < 1 || ncols > Q8K_COLS_MAX)
        return fail(Q8K_ERR_ARG, "%s: ncols=%lld must be in [1, %d]", fn, (long long)ncols, Q8K_COLS_MAX);
    if (fused_lds_bytes(ncols, K) > FUSED_LDS_MAX)
        return fail(Q8K_ERR_SHAPE,
                    "%s: ncols*K=%lld: the packed columns (%zu bytes) exceed one workgroup's %zu bytes of LDS "
                    "(use q8k_pack + qmatvec_batched)",
                    fn, (long long)(ncols * K), fused_lds_bytes(ncols, K), FUSED_LDS_MAX);
    Q8K_TRY(check_weight(fn, qtype, w));
    Q8K_TRY(check_ptr(fn, "x", x, 16));
    Q8K_TRY(check_ptr(fn, "y", y, 4));
    if (xq_out) Q8K_TRY(check_ptr(fn, "xq_out", xq_out, 16));
    if (rows == 0) return Q8K_OK;
    const int nb = (int)(K / QK);
    PackedOut o{nullptr, nullptr, nullptr};
    if (xq_out) {
        const Acts a = acts_of(xq_out, ncols, K);
        o = PackedOut{const_cast<int8_t*>(a.qs), const_cast<float*>(a.d), const_cast<int16_t*>(a.bs)};
    }
    const PrefillWeights pw = prefill_weights(qtype, w, rows * nb);
    return launched(fn, launch_matvec_f32(pw.fmt, pw.w, pw.prefix, rows, nb, x, K, (int)ncols, y, o,
                                          (hipStream_t)stream));
}

int qmatvec(int qtype, const void* w, int64_t rows, int64_t K, const void* xq, float* y, void* stream) {
    begin_call();
    return matvec_common("qmatvec", qtype, w, rows, K, xq, 1, y, stream);
}

int qmatvec_batched(int qtype, const void* w, int64_t rows, int64_t K, const void* xq, int64_t ncols, float* y,
                    void* stream) {
    begin_call();
    if (ncols < 1 || ncols > Q8K_COLS_MAX)
        return fail(Q8K_ERR_ARG, "qmatvec_batched: ncols=%lld must be in [1, %d]", (long long)ncols, Q8K_COLS_MAX);
    return matvec_common("qmatvec_batched", qtype, w, rows, K, xq, ncols, y, stream);
}

int qmatvec_moe(int qtype, const void* w, int64_t E, int64_t rows, int64_t K, const void* xq, int64_t T,
                const int32_t* ids, const float* rw, int32_t topk, float* y, void* stream) {
    begin_call();
    const char* fn = "qmatvec_moe";
    Q8K_TRY(check_k(fn, K));
    Q8K_TRY(check_count(fn, "rows", rows, MAX_ROWS));
    if (E < 1 || E > MAX_EXPERTS)
        return fail(Q8K_ERR_ARG, "%s: E=%lld must be in [1, %lld]", fn, (long long)E, (long long)MAX_EXPERTS);
    if (E * rows > MAX_ROWS)
        return fail(Q8K_ERR_SHAPE, "%s: E*rows=%lld exceeds %lld", fn, (long long)(E * rows), (long long)MAX_ROWS);
    if (T < 0 || T > Q8K_MOE_MAX_TOKENS)
        return fail(Q8K_ERR_ARG, "%s: T=%lld must be in [0, %d]", fn, (long long)T, Q8K_MOE_MAX_TOKENS);
    if (topk < 1 || topk > E || topk > Q8K_MOE_MAX_TOPK)
        return fail(Q8K_ERR_ARG, "%s: topk=%d must be in [1, min(E=%lld, %d)]", fn, topk, (long long)E,
                    Q8K_MOE_MAX_TOPK);
    Q8K_TRY(check_weight(fn, qtype, w));
    Q8K_TRY(check_ptr(fn, "xq", xq, 16));
    Q8K_TRY(check_ptr(fn, "ids", ids, 4));
    Q8K_TRY(check_ptr(fn, "rw", rw, 4));
    Q8K_TRY(check_ptr(fn, "y", y, 4));
    if (rows == 0 || T == 0) return Q8K_OK;
    const int nb = (int)(K / QK);
    const Acts a = acts_of(xq, T, K);
    hipError_t e;
    if (qtype == Q8K_Q4_K) {
        // matrix-core kernel while a packed token fits its LDS stage (K up to
        // about 89k), the one-lane-per-row kernel beyond
        if (moe_mfma_q4k_fits(K))
            e = launch_moe_mfma_q4k(static_cast<const uint8_t*>(w), E, rows, nb, a, T, ids, rw, topk, y,
                                    (hipStream_t)stream);
        else
            e = launch_moe_q4k(static_cast<const uint8_t*>(w), E, rows, nb, a, T, ids, rw, topk, y,
                               (hipStream_t)stream);
    } else if (qtype == Q8K_Q5_K) {
        if (moe_mfma_q4k_fits(K))
            e = launch_moe_mfma_q5k(static_cast<const uint8_t*>(w), E, rows, nb, a, T, ids, rw, topk, y,
                                    (hipStream_t)stream);
        else
            e = launch_moe_q5k(static_cast<const uint8_t*>(w), E, rows, nb, a, T, ids, rw, topk, y,
                               (hipStream_t)stream);
    } else {
        // relaid Q6_K: the matrix-core kernel while a packed token fits its
        // stage (K up to about 84k), the per-chunk kernel beyond
        const Q6View v = q6_view(w, E * rows * nb);
        if (moe_mfma_q6k_fits(K))
            e = launch_moe_mfma_q6k(v.prefix, v.bodies, E, rows, nb, a, T, ids, rw, topk, y, (hipStream_t)stream);
        else
            e = launch_moe_q6k(v.prefix, v.bodies, E, rows, nb, a, T, ids, rw, topk, y, (hipStream_t)stream);
    }
    return launched(fn, e);
}

size_t qmatmul_prefill_workspace_bytes(int qtype, int64_t rows, int64_t K, int64_t M) {
    (void)qtype;
    if (rows <= 0 || M <= 0 || K <= 0 || K % QK != 0) return 0;
    const int ks = prefill_ksplit(rows, K / QK, M);
    return ks > 1 ? (size_t)ks * (size_t)M * (size_t)rows * 4 : 0;
}

int qmatmul_prefill(int qtype, const void* w, int64_t rows, int64_t K, const void* xq, int64_t M, float* y, void* ws,
                    size_t ws_bytes, void* stream) {
    begin_call();
    const char* fn = "qmatmul_prefill";
    Q8K_TRY(check_k(fn, K));
    Q8K_TRY(check_count(fn, "rows", rows, MAX_ROWS));
    Q8K_TRY(check_count(fn, "M", M, MAX_TOKENS));
    Q8K_TRY(check_weight(fn, qtype, w));
    Q8K_TRY(check_ptr(fn, "xq", xq, 16));
    Q8K_TRY(check_ptr(fn, "y", y, 4));
    const size_t need = qmatmul_prefill_workspace_bytes(qtype, rows, K, M);
    if (ws_bytes < need)
        return fail(Q8K_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes, need);
    if (need > 0) Q8K_TRY(check_ptr(fn, "ws", ws, 16));
    Q8K_TRY(check_grid(fn, ((rows + 31) / 32) * ((M + 63) / 64)));  // bound for every tile shape
    if (rows == 0 || M == 0) return Q8K_OK;
    const int nb = (int)(K / QK);
    const PrefillWeights pw = prefill_weights(qtype, w, rows * nb);
    return launched(fn, launch_prefill(pw.fmt, pw.w, pw.prefix, rows, nb, acts_of(xq, M, K), M, y,
                                       static_cast<float*>(ws), (hipStream_t)stream));
}

size_t qmatmul_prefill_f32_workspace_bytes(int qtype, int64_t rows, int64_t K, int64_t M) {
    (void)qtype;
    if (rows <= 0 || M <= 0 || K <= 0 || K % QK != 0) return 0;
    const int ks = prefill_ksplit(rows, K / QK, M);
    return (size_t)prefill_sync_bytes(M, ks) + (ks > 1 ? (size_t)ks * (size_t)M * (size_t)rows * 4 : 0);
}

int qmatmul_prefill_f32(int qtype, const void* w, int64_t rows, int64_t K, const float* x, int64_t M, void* xq,
                        float* y, void* ws, size_t ws_bytes, void* stream) {
    begin_call();
    const char* fn = "qmatmul_prefill_f32";
    Q8K_TRY(check_k(fn, K));
    Q8K_TRY(check_count(fn, "rows", rows, MAX_ROWS));
    Q8K_TRY(check_count(fn, "M", M, MAX_TOKENS));
    Q8K_TRY(check_weight(fn, qtype, w));
    Q8K_TRY(check_ptr(fn, "x", x, 16));
    Q8K_TRY(check_ptr(fn, "xq", xq, 16));
    Q8K_TRY(check_ptr(fn, "y", y, 4));
    const size_t need = qmatmul_prefill_f32_workspace_bytes(qtype, rows, K, M);
    if (ws_bytes < need)
        return fail(Q8K_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes, need);
    if (need > 0) Q8K_TRY(check_ptr(fn, "ws", ws, 16));
    Q8K_TRY(check_grid(fn, ((rows + 31) / 32) * ((M + 63) / 64)));
    if (rows == 0 || M == 0) return Q8K_OK;
    // the row tiles of a token tile wait for each other: they must fit on the
    // device together (one workgroup per compute unit)
    const int64_t tiles = (rows + 63) / 64, cus = device_cu_count();
    if (tiles > cus)
        return fail(Q8K_ERR_SHAPE,
                    "%s: rows=%lld make %lld row tiles that wait for each other, more than the device's %lld compute "
                    "units (rows <= %lld; use q8k_pack + qmatmul_prefill)",
                    fn, (long long)rows, (long long)tiles, (long long)cus, (long long)(64 * cus));
    const int nb = (int)(K / QK);
    const int ks = prefill_ksplit(rows, nb, M);
    const Acts a = acts_of(xq, M, K);
    PackDst pk{x, const_cast<int8_t*>(a.qs), const_cast<float*>(a.d), const_cast<int16_t*>(a.bs),
               static_cast<int32_t*>(ws)};
    float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + prefill_sync_bytes(M, ks));
    const PrefillWeights pw = prefill_weights(qtype, w, rows * nb);
    return launched(fn, launch_prefill_f32(pw.fmt, pw.w, pw.prefix, rows, nb, a, M, y, part, pk,
                                           (hipStream_t)stream));
}

size_t qmatmul_prefill_moe_workspace_bytes(int qtype, int64_t E, int64_t rows, int64_t K, int64_t T, int32_t topk) {
    if ((qtype != Q8K_Q4_K && qtype != Q8K_Q5_K && qtype != Q8K_Q6_K_RELAID) || E < 1 || rows < 0 || K <= 0 ||
        K % QK != 0 || T < 0 || topk < 1)
        return 0;
    return (size_t)moe_prefill_ws(E, rows, T, topk).total;
}

static int prefill_moe_common(const char* fn, int qtype, const void* w, int64_t E, int64_t rows, int64_t K,
                              const void* xq, int64_t T, const int32_t* ids, const float* rw, int32_t topk, float* y,
                              void* ws, size_t ws_bytes, bool noalloc, void* stream);

int qmatmul_prefill_moe(int qtype, const void* w, int64_t E, int64_t rows, int64_t K, const void* xq, int64_t T,
                        const int32_t* ids, const float* rw, int32_t topk, float* y, void* ws, size_t ws_bytes,
                        void* stream) {
    begin_call();
    return prefill_moe_common("qmatmul_prefill_moe", qtype, w, E, rows, K, xq, T, ids, rw, topk, y, ws, ws_bytes,
                              false, stream);
}

int qmatmul_prefill_moe_noalloc(int qtype, const void* w, int64_t E, int64_t rows, int64_t K, const void* xq,
                                int64_t T, const int32_t* ids, const float* rw, int32_t topk, float* y,
                                void* stream) {
    begin_call();
    return prefill_moe_common("qmatmul_prefill_moe_noalloc", qtype, w, E, rows, K, xq, T, ids, rw, topk, y, nullptr,
                              0, true, stream);
}

static int prefill_moe_common(const char* fn, int qtype, const void* w, int64_t E, int64_t rows, int64_t K,
                              const void* xq, int64_t T, const int32_t* ids, const float* rw, int32_t topk, float* y,
                              void* ws, size_t ws_bytes, bool noalloc, void* stream) {
    Q8K_TRY(check_k(fn, K));
    Q8K_TRY(check_count(fn, "rows", rows, MAX_ROWS));
    if (E < 1 || E > MAX_EXPERTS)
        return fail(Q8K_ERR_ARG, "%s: E=%lld must be in [1, %lld]", fn, (long long)E, (long long)MAX_EXPERTS);
    if (E * rows > MAX_ROWS)
        return fail(Q8K_ERR_SHAPE, "%s: E*rows=%lld exceeds %lld", fn, (long long)(E * rows), (long long)MAX_ROWS);
    Q8K_TRY(check_count(fn, "T", T, MAX_TOKENS));
    if (T * K >= ((int64_t)1 << 30))
        return fail(Q8K_ERR_SHAPE, "%s: T*K=%lld must be below 2^30 (32-bit gather offsets)", fn,
                    (long long)(T * K));
    if (topk < 1 || topk > E || topk > Q8K_MOE_MAX_TOPK)
        return fail(Q8K_ERR_ARG, "%s: topk=%d must be in [1, min(E=%lld, %d)]", fn, topk, (long long)E,
                    Q8K_MOE_MAX_TOPK);
    Q8K_TRY(check_weight(fn, qtype, w));
    Q8K_TRY(check_ptr(fn, "xq", xq, 16));
    Q8K_TRY(check_ptr(fn, "ids", ids, 4));
    Q8K_TRY(check_ptr(fn, "rw", rw, 4));
    Q8K_TRY(check_ptr(fn, "y", y, 4));
    const size_t need = qmatmul_prefill_moe_workspace_bytes(qtype, E, rows, K, T, topk);
    if (noalloc) {
        if (need > NOALLOC_SCRATCH_BYTES)
            return fail(Q8K_ERR_WORKSPACE,
                        "%s: the call needs %zu bytes of workspace, more than the library's %zu-byte scratch "
                        "(use qmatmul_prefill_moe with a caller workspace)",
                        fn, need, NOALLOC_SCRATCH_BYTES);
    } else {
        if (ws_bytes < need)
            return fail(Q8K_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes, need);
        if (need > 0) Q8K_TRY(check_ptr(fn, "ws", ws, 16));
    }
    Q8K_TRY(check_grid(fn, moe_prefill_ws(E, rows, T, topk).max_chunks * ((rows + 63) / 64)));
    Q8K_TRY(check_grid(fn, T * ((rows + 255) / 256)));  // the combine's workgroups, at most
    if (rows == 0 || T == 0) return Q8K_OK;
    if (noalloc) {
        const hipError_t e = noalloc_scratch(&ws);
        if (e != hipSuccess)
            return fail(Q8K_ERR_LAUNCH, "%s: the library's scratch is not available: %s", fn, hipGetErrorString(e));
    }
    const int nb = (int)(K / QK);
    const PrefillWeights pw = prefill_weights(qtype, w, E * rows * nb);
    return launched(fn, launch_prefill_moe(pw.fmt, pw.w, pw.prefix, E, rows, nb, acts_of(xq, T, K), T, ids, rw, topk,
                                           y, ws, (hipStream_t)stream));
}

// ---- the paged key/value cache and the operators behind the projections
constexpr int64_t MAX_PAGES = (int64_t)1 << 24;
constexpr int64_t MAX_HEADS = (int64_t)1 << 12;
constexpr int64_t MAX_LEN = (int64_t)1 << 30;
constexpr int64_t MAX_BATCH = (int64_t)1 << 20;
constexpr int64_t MAX_VOCAB = (int64_t)1 << 20;  // a row's byte offsets stay in 32 bits

static int check_dtype(const char* fn, int dtype) {
    if (dtype != Q8K_F32 && dtype != Q8K_F16 && dtype != Q8K_BF16)
        return fail(Q8K_ERR_ARG, "%s: dtype=%d must be Q8K_F32=0, Q8K_F16=1 or Q8K_BF16=2", fn, dtype);
    return Q8K_OK;
}

static bool kv_dim(int32_t D) { return D == 64 || D == 128 || D == 256; }

static int check_kv(const char* fn, const q8k_kv_cache* kv) {
    if (!kv) return fail(Q8K_ERR_NULL, "%s: kv is NULL", fn);
    if (!kv_dim(kv->head_dim))
        return fail(Q8K_ERR_SHAPE, "%s: head_dim=%d not served (64, 128 or 256)", fn, (int)kv->head_dim);
    if (kv->kv_heads < 1 || kv->kv_heads > MAX_HEADS)
        return fail(Q8K_ERR_SHAPE, "%s: kv_heads=%d out of range [1, %lld]", fn, (int)kv->kv_heads,
                    (long long)MAX_HEADS);
    Q8K_TRY(check_count(fn, "pages", kv->pages, MAX_PAGES));
    return check_ptr(fn, "kv->data", kv->data, 16);
}

// The rotation's description and its positions; view.table is NULL without one.
static int check_rope(const char* fn, const q8k_rope* rope, const int32_t* pos, int32_t D, RopeView* view) {
    *view = RopeView{nullptr, 0, 0, 0};
    if (!rope) return Q8K_OK;
    Q8K_TRY(check_ptr(fn, "rope->table", rope->table, 16));
    Q8K_TRY(check_ptr(fn, "pos", pos, 4));
    if (rope->positions < 1 || rope->positions > MAX_LEN)
        return fail(Q8K_ERR_SHAPE, "%s: rope->positions=%lld out of range [1, %lld]", fn, (long long)rope->positions,
                    (long long)MAX_LEN);
    if (rope->dim < 8 || rope->dim % 8 != 0 || rope->dim > D)
        return fail(Q8K_ERR_SHAPE, "%s: rope->dim=%d must be a positive multiple of 8, at most head_dim=%d", fn,
                    (int)rope->dim, (int)D);
    if (rope->pairs != Q8K_ROPE_HALF && rope->pairs != Q8K_ROPE_ADJACENT)
        return fail(Q8K_ERR_ARG, "%s: rope->pairs=%d must be Q8K_ROPE_HALF=0 or Q8K_ROPE_ADJACENT=1", fn,
                    (int)rope->pairs);
    *view = RopeView{rope->table, (int)rope->positions, rope->dim, rope->pairs == Q8K_ROPE_ADJACENT};
    return Q8K_OK;
}

static int check_stride(const char* fn, const char* what, int64_t stride, int64_t least) {
    if (stride < least || stride % 8 != 0 || stride > ((int64_t)1 << 32))
        return fail(Q8K_ERR_SHAPE, "%s: %s=%lld must be a multiple of 8, at least the row's %lld values", fn, what,
                    (long long)stride, (long long)least);
    return Q8K_OK;
}

// The calls of the caches of 8 and of 4 bits differ in the record alone.
static size_t kv_bytes(int bits, int64_t pages, int64_t kv_heads, int64_t head_dim) {
    if (pages < 0 || pages > MAX_PAGES || kv_heads < 1 || kv_heads > MAX_HEADS ||
        (head_dim != 64 && head_dim != 128 && head_dim != 256))
        return 0;
    return (size_t)pages * (size_t)kv_heads * (size_t)kv_record_of(bits, (int)head_dim);
}

size_t q8k_kv_bytes(int64_t pages, int64_t kv_heads, int64_t head_dim) { return kv_bytes(8, pages, kv_heads, head_dim); }
size_t q8k_kv4_bytes(int64_t pages, int64_t kv_heads, int64_t head_dim) { return kv_bytes(4, pages, kv_heads, head_dim); }

static int kv_append(const char* fn, int bits, int dtype, const void* k, int64_t k_stride, const void* v,
                     int64_t v_stride, int64_t T, const int32_t* pos, const q8k_rope* rope, const int32_t* slots,
                     const q8k_kv_cache* kv, void* stream) {
    begin_call();
    Q8K_TRY(check_dtype(fn, dtype));
    Q8K_TRY(check_kv(fn, kv));
    Q8K_TRY(check_count(fn, "T", T, MAX_TOKENS));
    const int64_t row = (int64_t)kv->kv_heads * kv->head_dim;
    Q8K_TRY(check_stride(fn, "k_stride", k_stride, row));
    Q8K_TRY(check_stride(fn, "v_stride", v_stride, row));
    Q8K_TRY(check_ptr(fn, "k", k, 16));
    Q8K_TRY(check_ptr(fn, "v", v, 16));
    Q8K_TRY(check_ptr(fn, "slots", slots, 4));
    KvAppend a{k, v, k_stride, v_stride, T, pos, slots, {}, static_cast<uint8_t*>(kv->data), kv->pages,
               kv->kv_heads, dtype};
    Q8K_TRY(check_rope(fn, rope, pos, kv->head_dim, &a.rope));
    Q8K_TRY(check_grid(fn, (2 * T * row + 2047) / 2048));
    Q8K_TRY(check_threads(fn, kv_workgroups(T, kv->kv_heads), 256));
    if (T == 0 || kv->pages == 0) return Q8K_OK;
    return launched(fn, bits == 8 ? launch_kv_append(kv->head_dim, a, (hipStream_t)stream)
                                  : launch_kv4_append(kv->head_dim, a, (hipStream_t)stream));
}

int q8k_kv_append(int dtype, const void* k, int64_t k_stride, const void* v, int64_t v_stride, int64_t T,
                  const int32_t* pos, const q8k_rope* rope, const int32_t* slots, const q8k_kv_cache* kv,
                  void* stream) {
    return kv_append("q8k_kv_append", 8, dtype, k, k_stride, v, v_stride, T, pos, rope, slots, kv, stream);
}

int q8k_kv4_append(int dtype, const void* k, int64_t k_stride, const void* v, int64_t v_stride, int64_t T,
                   const int32_t* pos, const q8k_rope* rope, const int32_t* slots, const q8k_kv_cache* kv,
                   void* stream) {
    return kv_append("q8k_kv4_append", 4, dtype, k, k_stride, v, v_stride, T, pos, rope, slots, kv, stream);
}

static int kv_read(const char* fn, int bits, int dtype, const q8k_kv_cache* kv, const int32_t* slots, int64_t T,
                   void* k, void* v, void* stream) {
    begin_call();
    Q8K_TRY(check_dtype(fn, dtype));
    Q8K_TRY(check_kv(fn, kv));
    Q8K_TRY(check_count(fn, "T", T, MAX_TOKENS));
    Q8K_TRY(check_ptr(fn, "slots", slots, 4));
    Q8K_TRY(check_ptr(fn, "k", k, 16));
    Q8K_TRY(check_ptr(fn, "v", v, 16));
    Q8K_TRY(check_grid(fn, (T * kv->kv_heads * kv->head_dim + 2047) / 2048));
    Q8K_TRY(check_threads(fn, kv_workgroups(T, kv->kv_heads), 256));
    if (T == 0) return Q8K_OK;
    const KvRead a{static_cast<const uint8_t*>(kv->data), kv->pages, kv->kv_heads, dtype, slots, T, k, v};
    return launched(fn, bits == 8 ? launch_kv_read(kv->head_dim, a, (hipStream_t)stream)
                                  : launch_kv4_read(kv->head_dim, a, (hipStream_t)stream));
}

int q8k_kv_read(int dtype, const q8k_kv_cache* kv, const int32_t* slots, int64_t T, void* k, void* v, void* stream) {
    return kv_read("q8k_kv_read", 8, dtype, kv, slots, T, k, v, stream);
}

int q8k_kv4_read(int dtype, const q8k_kv_cache* kv, const int32_t* slots, int64_t T, void* k, void* v, void* stream) {
    return kv_read("q8k_kv4_read", 4, dtype, kv, slots, T, k, v, stream);
}

static int check_attend_sizes(const char* fn, const q8k_kv_cache* kv, int64_t q_heads, int64_t B, int64_t Tq,
                              int64_t max_q, int64_t max_len) {
    if (q_heads < 1 || q_heads > MAX_HEADS || q_heads % kv->kv_heads != 0)
        return fail(Q8K_ERR_SHAPE, "%s: q_heads=%lld must be a positive multiple of kv_heads=%d (at most %lld)", fn,
                    (long long)q_heads, (int)kv->kv_heads, (long long)MAX_HEADS);
    Q8K_TRY(check_count(fn, "B", B, MAX_BATCH));
    Q8K_TRY(check_count(fn, "Tq", Tq, MAX_TOKENS));
    Q8K_TRY(check_count(fn, "max_q", max_q, Tq));
    if (max_q * (q_heads / kv->kv_heads) > ((int64_t)1 << 30))
        return fail(Q8K_ERR_SHAPE, "%s: max_q=%lld new tokens of %lld query heads a key head are over 2^30 rows", fn,
                    (long long)max_q, (long long)(q_heads / kv->kv_heads));
    return check_count(fn, "max_len", max_len, MAX_LEN);
}

static size_t attend_workspace_bytes(const char* fn, int bits, const q8k_kv_cache* kv, int64_t q_heads, int64_t B, int64_t Tq,
                                     int64_t max_q, int64_t max_len) {
    if (!kv || !kv_dim(kv->head_dim) || kv->kv_heads < 1 || kv->kv_heads > MAX_HEADS ||
        check_attend_sizes(fn, kv, q_heads, B, Tq, max_q, max_len) != Q8K_OK || B == 0 || max_q == 0)
        return 0;
    return (size_t)attend_plan(bits, B, max_q, max_len, (int)q_heads, kv->kv_heads, kv->head_dim, 0).ws_bytes;
}

size_t qattend_workspace_bytes(const q8k_kv_cache* kv, int64_t q_heads, int64_t B, int64_t Tq, int64_t max_q,
                               int64_t max_len) {
    return attend_workspace_bytes("qattend_workspace_bytes", 8, kv, q_heads, B, Tq, max_q, max_len);
}

size_t qattend_kv4_workspace_bytes(const q8k_kv_cache* kv, int64_t q_heads, int64_t B, int64_t Tq, int64_t max_q,
                                   int64_t max_len) {
    return attend_workspace_bytes("qattend_kv4_workspace_bytes", 4, kv, q_heads, B, Tq, max_q, max_len);
}

// What attention and its weights are asked of queries, pages and lengths: the
// checks, and these in *a.
static int check_attend(const char* fn, int dtype, const void* q, int64_t q_stride, int64_t q_heads,
                        const q8k_kv_cache* kv, int64_t B, const int32_t* cu_q, int64_t Tq, int64_t max_q,
                        const int32_t* page_table, int64_t max_pages, const int32_t* kv_len, int64_t max_len,
                        float scale, int64_t window, const int32_t* pos, const q8k_rope* rope, Attend* a) {
    Q8K_TRY(check_dtype(fn, dtype));
    Q8K_TRY(check_kv(fn, kv));
    Q8K_TRY(check_attend_sizes(fn, kv, q_heads, B, Tq, max_q, max_len));
    Q8K_TRY(check_count(fn, "max_pages", max_pages, MAX_PAGES));
    if (max_len > max_pages * KV_PAGE)
        return fail(Q8K_ERR_SHAPE, "%s: max_len=%lld exceeds the page table's %lld pages of %d tokens", fn,
                    (long long)max_len, (long long)max_pages, KV_PAGE);
    Q8K_TRY(check_count(fn, "window", window, MAX_LEN));
    if (!(scale - scale == 0.0f)) return fail(Q8K_ERR_ARG, "%s: scale=%g must be finite", fn, (double)scale);
    Q8K_TRY(check_stride(fn, "q_stride", q_stride, q_heads * kv->head_dim));
    Q8K_TRY(check_ptr(fn, "q", q, 16));
    Q8K_TRY(check_ptr(fn, "cu_q", cu_q, 4));
    Q8K_TRY(check_ptr(fn, "page_table", page_table, 4));
    Q8K_TRY(check_ptr(fn, "kv_len", kv_len, 4));
    Q8K_TRY(check_rope(fn, rope, pos, kv->head_dim, &a->rope));
    a->q = q;
    a->q_stride = q_stride;
    a->q_heads = (int)q_heads;
    a->heads = kv->kv_heads;
    a->group = (int)(q_heads / kv->kv_heads);
    a->dtype = dtype;
    a->cache = static_cast<const uint8_t*>(kv->data);
    a->pages = kv->pages;
    a->B = B;
    a->cu_q = cu_q;
    a->Tq = Tq;
    a->max_q = max_q;
    a->table = page_table;
    a->max_pages = max_pages;
    a->kv_len = kv_len;
    a->max_len = max_len;
    a->scale = scale;
    a->window = window;
    a->pos = pos;
    return Q8K_OK;
}

static int attend(const char* fn, int bits, int dtype, const void* q, int64_t q_stride, int64_t q_heads,
                  const q8k_kv_cache* kv, int64_t B, const int32_t* cu_q, int64_t Tq, int64_t max_q,
                  const int32_t* page_table, int64_t max_pages, const int32_t* kv_len, int64_t max_len, float scale,
                  int64_t window, const int32_t* pos, const q8k_rope* rope, void* out, float* lse, void* ws,
                  size_t ws_bytes, void* stream) {
    begin_call();
    Attend a{};
    Q8K_TRY(check_attend(fn, dtype, q, q_stride, q_heads, kv, B, cu_q, Tq, max_q, page_table, max_pages, kv_len,
                         max_len, scale, window, pos, rope, &a));
    Q8K_TRY(check_ptr(fn, "out", out, 16));
    if (lse) Q8K_TRY(check_ptr(fn, "lse", lse, 4));
    const size_t need = attend_workspace_bytes(fn, bits, kv, q_heads, B, Tq, max_q, max_len);
    if (ws_bytes < need)
        return fail(Q8K_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes, need);
    if (need > 0) Q8K_TRY(check_ptr(fn, "ws", ws, 16));
    if (B == 0 || max_q == 0) return Q8K_OK;
    const AttendPlan p = attend_plan(bits, B, max_q, max_len, (int)q_heads, kv->kv_heads, kv->head_dim, window);
    Q8K_TRY(check_grid(fn, p.items * kv->kv_heads));
    Q8K_TRY(check_threads(fn, p.items * kv->kv_heads * p.slices, p.threads));
    a.out = out;
    a.lse = lse;
    return launched(fn, launch_attend(bits, kv->head_dim, p, a, ws, (hipStream_t)stream));
}

int qattend(int dtype, const void* q, int64_t q_stride, int64_t q_heads, const q8k_kv_cache* kv, int64_t B,
            const int32_t* cu_q, int64_t Tq, int64_t max_q, const int32_t* page_table, int64_t max_pages,
            const int32_t* kv_len, int64_t max_len, float scale, int64_t window, const int32_t* pos,
            const q8k_rope* rope, void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    return attend("qattend", 8, dtype, q, q_stride, q_heads, kv, B, cu_q, Tq, max_q, page_table, max_pages, kv_len,
                  max_len, scale, window, pos, rope, out, lse, ws, ws_bytes, stream);
}

int qattend_kv4(int dtype, const void* q, int64_t q_stride, int64_t q_heads, const q8k_kv_cache* kv, int64_t B,
                const int32_t* cu_q, int64_t Tq, int64_t max_q, const int32_t* page_table, int64_t max_pages,
                const int32_t* kv_len, int64_t max_len, float scale, int64_t window, const int32_t* pos,
                const q8k_rope* rope, void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    return attend("qattend_kv4", 4, dtype, q, q_stride, q_heads, kv, B, cu_q, Tq, max_q, page_table, max_pages,
                  kv_len, max_len, scale, window, pos, rope, out, lse, ws, ws_bytes, stream);
}

static int check_bits(const char* fn, int bits) {
    if (bits != 8 && bits != 4) return fail(Q8K_ERR_ARG, "%s: bits=%d: a cache is held in 8 or 4", fn, bits);
    return Q8K_OK;
}

size_t qattend_weights_workspace_bytes(const q8k_kv_cache* kv, int64_t q_heads, int64_t B, int64_t Tq, int64_t max_q,
                                       int64_t max_len) {
    const char* fn = "qattend_weights_workspace_bytes";
    if (!kv || !kv_dim(kv->head_dim) || kv->kv_heads < 1 || kv->kv_heads > MAX_HEADS ||
        check_attend_sizes(fn, kv, q_heads, B, Tq, max_q, max_len) != Q8K_OK || B == 0 || max_len == 0)
        return 0;
    return (size_t)weights_plan(B, Tq, max_q, max_len, (int)q_heads, kv->kv_heads, kv->head_dim).ws_bytes;
}

int qattend_weights(int dtype, int bits, const void* q, int64_t q_stride, int64_t q_heads, const q8k_kv_cache* kv,
                    int64_t B, const int32_t* cu_q, int64_t Tq, int64_t max_q, const int32_t* page_table,
                    int64_t max_pages, const int32_t* kv_len, int64_t max_len, float scale, int64_t window,
                    const int32_t* pos, const q8k_rope* rope, const float* lse, const float* old, float keep,
                    float* weights, int64_t w_stride, void* ws, size_t ws_bytes, void* stream) {
    begin_call();
    const char* fn = "qattend_weights";
    AttendWeights w{};
    Q8K_TRY(check_bits(fn, bits));
    Q8K_TRY(check_attend(fn, dtype, q, q_stride, q_heads, kv, B, cu_q, Tq, max_q, page_table, max_pages, kv_len,
                         max_len, scale, window, pos, rope, &w.a));
    Q8K_TRY(check_ptr(fn, "lse", lse, 4));
    if (old) Q8K_TRY(check_ptr(fn, "old", old, 4));
    Q8K_TRY(check_ptr(fn, "weights", weights, 4));
    if (!(keep - keep == 0.0f)) return fail(Q8K_ERR_ARG, "%s: keep=%g must be finite", fn, (double)keep);
    if (w_stride < max_len || w_stride > ((int64_t)1 << 32))
        return fail(Q8K_ERR_SHAPE, "%s: w_stride=%lld must be at least max_len=%lld", fn, (long long)w_stride,
                    (long long)max_len);
    const size_t need = qattend_weights_workspace_bytes(kv, q_heads, B, Tq, max_q, max_len);
    if (ws_bytes < need)
        return fail(Q8K_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes, need);
    if (need > 0) Q8K_TRY(check_ptr(fn, "ws", ws, 16));
    if (B == 0 || max_len == 0) return Q8K_OK;
    const WeightsPlan p = weights_plan(B, Tq, max_q, max_len, (int)q_heads, kv->kv_heads, kv->head_dim);
    Q8K_TRY(check_grid(fn, p.workgroups));
    Q8K_TRY(check_threads(fn, p.workgroups, p.threads));
    if (p.split) Q8K_TRY(check_threads(fn, p.join_workgroups, p.threads));
    Q8K_TRY(check_threads(fn, B * kv->kv_heads * p.tiles_max, 64));
    w.lse = lse;
    w.old = old;
    w.keep = keep;
    w.weights = weights;
    w.stride = w_stride;
    return launched(fn, launch_attend_weights(bits, kv->head_dim, p, w, ws, (hipStream_t)stream));
}

int q8k_kv_evict(int bits, const q8k_kv_cache* kv, int64_t B, const int32_t* page_table, int64_t max_pages,
                 const int32_t* kv_len, int64_t max_len, const float* weights, int64_t w_stride, int64_t budget,
                 int64_t first, int64_t last, const int32_t* out_table, int64_t out_pages, float* out_weights,
                 int64_t out_stride, int32_t* kept, int32_t* new_len, void* stream) {
    begin_call();
    const char* fn = "q8k_kv_evict";
    Q8K_TRY(check_bits(fn, bits));
    Q8K_TRY(check_kv(fn, kv));
    Q8K_TRY(check_count(fn, "B", B, MAX_BATCH));
    Q8K_TRY(check_count(fn, "max_pages", max_pages, MAX_PAGES));
    Q8K_TRY(check_count(fn, "max_len", max_len, MAX_LEN));
    Q8K_TRY(check_count(fn, "out_pages", out_pages, MAX_PAGES));
    if (max_len > max_pages * KV_PAGE)
        return fail(Q8K_ERR_SHAPE, "%s: max_len=%lld exceeds the page table's %lld pages of %d tokens", fn,
                    (long long)max_len, (long long)max_pages, KV_PAGE);
    if (budget < 1 || budget > MAX_LEN || budget > out_pages * KV_PAGE)
        return fail(Q8K_ERR_SHAPE, "%s: budget=%lld must be at least 1 and fit the new page table's %lld pages of %d tokens",
                    fn, (long long)budget, (long long)out_pages, KV_PAGE);
    if (first < 0 || last < 0 || first > budget || last > budget - first)
        return fail(Q8K_ERR_ARG, "%s: first=%lld and last=%lld tokens exceed budget=%lld", fn, (long long)first,
                    (long long)last, (long long)budget);
    if (w_stride < max_len || w_stride > ((int64_t)1 << 32))
        return fail(Q8K_ERR_SHAPE, "%s: w_stride=%lld must be at least max_len=%lld", fn, (long long)w_stride,
                    (long long)max_len);
    Q8K_TRY(check_ptr(fn, "page_table", page_table, 4));
    Q8K_TRY(check_ptr(fn, "kv_len", kv_len, 4));
    Q8K_TRY(check_ptr(fn, "weights", weights, 4));
    Q8K_TRY(check_ptr(fn, "out_table", out_table, 4));
    if (out_weights) {
        Q8K_TRY(check_ptr(fn, "out_weights", out_weights, 4));
        if (out_stride < budget || out_stride > ((int64_t)1 << 32))
            return fail(Q8K_ERR_SHAPE, "%s: out_stride=%lld must be at least budget=%lld", fn, (long long)out_stride,
                        (long long)budget);
        if (out_weights == weights && out_stride != w_stride)
            return fail(Q8K_ERR_ARG, "%s: weights kept in place need out_stride=%lld to be w_stride=%lld", fn,
                        (long long)out_stride, (long long)w_stride);
    }
    Q8K_TRY(check_ptr(fn, "kept", kept, 4));
    Q8K_TRY(check_ptr(fn, "new_len", new_len, 4));
    if (new_len == kv_len) return fail(Q8K_ERR_ARG, "%s: new_len must not be kv_len, which the call reads to its end", fn);
    const bool in_place = out_table == page_table;
    if (in_place && out_pages != max_pages)
        return fail(Q8K_ERR_ARG, "%s: a move in place needs out_pages=%lld to be max_pages=%lld", fn,
                    (long long)out_pages, (long long)max_pages);
    Q8K_TRY(check_threads(fn, B * kv->kv_heads, evict_threads()));
    Q8K_TRY(check_threads(fn, evict_workgroups(bits, kv->head_dim, B, kv->kv_heads, budget, in_place), 64));
    if (B == 0) return Q8K_OK;
    const KvEvict a{static_cast<uint8_t*>(kv->data), kv->pages, kv->kv_heads, B, page_table, max_pages, kv_len, max_len,
                    weights, w_stride, budget, first, last, out_table, out_pages, out_weights, out_stride, kept, new_len};
    return launched(fn, launch_kv_evict(bits, kv->head_dim, a, in_place, (hipStream_t)stream));
}

size_t qlogprobs_workspace_bytes(int64_t T, int64_t V, int32_t topn) {
    if (T <= 0 || T > MAX_TOKENS || V < 1 || V > MAX_VOCAB || topn < 0 || topn > Q8K_TOP_MAX || topn > V) return 0;
    return (size_t)logprobs_ws_bytes(T, V, topn);
}

int qlogprobs(int dtype, const void* logits, int64_t stride, int64_t T, int64_t V, const int32_t* targets,
              float* logprob, float* entropy, float* lse, int32_t topn, int32_t* top_ids, float* top_logprob,
              void* ws, size_t ws_bytes, void* stream) {
    begin_call();
    const char* fn = "qlogprobs";
    Q8K_TRY(check_dtype(fn, dtype));
    Q8K_TRY(check_count(fn, "T", T, MAX_TOKENS));
    if (V < 1 || V > MAX_VOCAB)
        return fail(Q8K_ERR_SHAPE, "%s: V=%lld out of range [1, %lld]", fn, (long long)V, (long long)MAX_VOCAB);
    if (stride < V || stride > ((int64_t)1 << 32))
        return fail(Q8K_ERR_SHAPE, "%s: stride=%lld must be at least V=%lld", fn, (long long)stride, (long long)V);
    if (topn < 0 || topn > Q8K_TOP_MAX || topn > V)
        return fail(Q8K_ERR_ARG, "%s: topn=%d must be in [0, min(V=%lld, %d)]", fn, topn, (long long)V, Q8K_TOP_MAX);
    Q8K_TRY(check_ptr(fn, "logits", logits, dtype == Q8K_F32 ? 4 : 2));
    if (targets || logprob) {  // both or neither
        Q8K_TRY(check_ptr(fn, "targets", targets, 4));
        Q8K_TRY(check_ptr(fn, "logprob", logprob, 4));
    }
    if (entropy) Q8K_TRY(check_ptr(fn, "entropy", entropy, 4));
    if (lse) Q8K_TRY(check_ptr(fn, "lse", lse, 4));
    if (topn > 0) {
        Q8K_TRY(check_ptr(fn, "top_ids", top_ids, 4));
        Q8K_TRY(check_ptr(fn, "top_logprob", top_logprob, 4));
    }
    const size_t need = qlogprobs_workspace_bytes(T, V, topn);
    if (ws_bytes < need)
        return fail(Q8K_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes, need);
    if (need > 0) Q8K_TRY(check_ptr(fn, "ws", ws, 16));
    Q8K_TRY(check_grid(fn, T * ((V + 1023) / 1024)));
    Q8K_TRY(check_threads(fn, T, logprobs_threads(T, V)));
    if (T == 0) return Q8K_OK;
    const LogProbs a{logits, stride, T, V, dtype, targets, logprob, entropy, lse, topn, top_ids, top_logprob};
    return launched(fn, launch_logprobs(a, ws, (hipStream_t)stream));
}

int q8k_debug_subblock_sums(int qtype, const void* w, int64_t rows, int64_t K, const void* xq, float* y, int32_t* S,
                            void* stream) {
    begin_call();
    const char* fn = "q8k_debug_subblock_sums";
    Q8K_TRY(check_k(fn, K));
    Q8K_TRY(check_count(fn, "rows", rows, MAX_ROWS));
    Q8K_TRY(check_weight(fn, qtype, w));
    Q8K_TRY(check_ptr(fn, "xq", xq, 16));
    Q8K_TRY(check_ptr(fn, "y", y, 4));
    Q8K_TRY(check_ptr(fn, "S", S, 4));
    if (rows == 0) return Q8K_OK;
    const int nb = (int)(K / QK);
    const PrefillWeights pw = prefill_weights(qtype, w, rows * nb);
    return launched(fn, launch_matvec_sums(pw.fmt, pw.w, pw.prefix, rows, nb, acts_of(xq, 1, K), y, S,
                                           (hipStream_t)stream));
}

int q8k_debug_prefill_block_sums(int qtype, const void* w, int64_t rows, int64_t K, const void* xq, int64_t M,
                                 float* y, int32_t* I, void* stream) {
    begin_call();
    const char* fn = "q8k_debug_prefill_block_sums";
    Q8K_TRY(check_k(fn, K));
    Q8K_TRY(check_count(fn, "rows", rows, MAX_ROWS));
    Q8K_TRY(check_count(fn, "M", M, MAX_TOKENS));
    Q8K_TRY(check_weight(fn, qtype, w));
    Q8K_TRY(check_ptr(fn, "xq", xq, 16));
    Q8K_TRY(check_ptr(fn, "y", y, 4));
    Q8K_TRY(check_ptr(fn, "I", I, 4));
    Q8K_TRY(check_grid(fn, ((rows + 31) / 32) * ((M + 63) / 64)));
    if (rows == 0 || M == 0) return Q8K_OK;
    const int nb = (int)(K / QK);
    const PrefillWeights pw = prefill_weights(qtype, w, rows * nb);
    return launched(fn, launch_prefill_sums(pw.fmt, pw.w, pw.prefix, rows, nb, acts_of(xq, M, K), M, y, I,
                                            (hipStream_t)stream));
}

int q8k_debug_moe_subblock_sums(int qtype, const void* w, int64_t E, int64_t rows, int64_t K, const void* xq,
                                int64_t T, const int32_t* ids, const float* rw, int32_t topk, float* y, int32_t* S,
                                void* stream) {
    begin_call();
    const char* fn = "q8k_debug_moe_subblock_sums";
    Q8K_TRY(check_k(fn, K));
    Q8K_TRY(check_count(fn, "rows", rows, MAX_ROWS));
    if (qtype != Q8K_Q4_K && qtype != Q8K_Q5_K && qtype != Q8K_Q6_K_RELAID)
        return fail(Q8K_ERR_QTYPE,
                    "%s: qtype=%d: the matrix-core MoE kernels serve Q8K_Q4_K, Q8K_Q5_K and Q8K_Q6_K_RELAID", fn, qtype);
    if (qtype == Q8K_Q6_K_RELAID ? !moe_mfma_q6k_fits(K) : !moe_mfma_q4k_fits(K))
        return fail(Q8K_ERR_SHAPE, "%s: K=%lld: a packed token exceeds the matrix-core MoE kernel's LDS stage", fn,
                    (long long)K);
    if (E < 1 || E > MAX_EXPERTS)
        return fail(Q8K_ERR_ARG, "%s: E=%lld must be in [1, %lld]", fn, (long long)E, (long long)MAX_EXPERTS);
    if (E * rows > MAX_ROWS)
        return fail(Q8K_ERR_SHAPE, "%s: E*rows=%lld exceeds %lld", fn, (long long)(E * rows), (long long)MAX_ROWS);
    if (T < 0 || T > Q8K_MOE_MAX_TOKENS)
        return fail(Q8K_ERR_ARG, "%s: T=%lld must be in [0, %d]", fn, (long long)T, Q8K_MOE_MAX_TOKENS);
    if (topk < 1 || topk > E || topk > Q8K_MOE_MAX_TOPK)
        return fail(Q8K_ERR_ARG, "%s: topk=%d must be in [1, min(E=%lld, %d)]", fn, topk, (long long)E,
                    Q8K_MOE_MAX_TOPK);
    Q8K_TRY(check_ptr(fn, "w", w, 16));
    Q8K_TRY(check_ptr(fn, "xq", xq, 16));
    Q8K_TRY(check_ptr(fn, "ids", ids, 4));
    Q8K_TRY(check_ptr(fn, "rw", rw, 4));
    Q8K_TRY(check_ptr(fn, "y", y, 4));
    Q8K_TRY(check_ptr(fn, "S", S, 4));
    if (rows == 0 || T == 0) return Q8K_OK;
    if (qtype == Q8K_Q6_K_RELAID) {
        const Q6View v = q6_view(w, E * rows * (K / QK));
        return launched(fn, launch_moe_mfma6_sums(v.prefix, v.bodies, E, rows, (int)(K / QK), acts_of(xq, T, K), T, ids,
                                                  rw, topk, y, S, (hipStream_t)stream));
    }
    return launched(fn, launch_moe_mfma_sums(qtype == Q8K_Q5_K, static_cast<const uint8_t*>(w), E, rows, (int)(K / QK),
                                             acts_of(xq, T, K), T, ids, rw, topk, y, S, (hipStream_t)stream));
}

int q8k_debug_wave_sums(float* out, void* stream) {
    begin_call();
    Q8K_TRY(check_ptr("q8k_debug_wave_sums", "out", out, 4));
    return launched("q8k_debug_wave_sums", launch_wave_sums(out, (hipStream_t)stream));
}

int q8k_debug_last_launches(const void** handles, int max) {
    const int n = g_nlaunched < LAUNCH_RECORD_MAX ? g_nlaunched : LAUNCH_RECORD_MAX;
    for (int i = 0; i < n && i < max; ++i) handles[i] = g_launched[i];
    return g_nlaunched;
}

const char* q8k_status_str(int status) {
    switch (status) {
        case Q8K_OK: return "Q8K_OK";
        case Q8K_ERR_NULL: return "Q8K_ERR_NULL";
        case Q8K_ERR_SHAPE: return "Q8K_ERR_SHAPE";
        case Q8K_ERR_ALIGN: return "Q8K_ERR_ALIGN";
        case Q8K_ERR_QTYPE: return "Q8K_ERR_QTYPE";
        case Q8K_ERR_ARG: return "Q8K_ERR_ARG";
        case Q8K_ERR_WORKSPACE: return "Q8K_ERR_WORKSPACE";
        case Q8K_ERR_LAUNCH: return "Q8K_ERR_LAUNCH";
        default: return "Q8K_ERR_UNKNOWN";
    }
}

const char* q8k_last_error(void) { return g_err; }

}  // extern "C"
