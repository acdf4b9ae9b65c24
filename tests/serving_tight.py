"""Tolerances near what the serving kernels' own arithmetic can be off by, and
inputs on which one token or one logit more or less shows.

serving_helpers.py bounds the errors by the worst order of summation, which
grows with the length; here they follow the depth of the sums that the kernels
take, and inputs are such that a miscounted term exceeds them by far
(test_serving_bounds.py plants such mistakes in the plain forms).
"""
from __future__ import annotations

import numpy as np

import serving_helpers as sh

U = 2.0 ** -24  # half a step of fp32, relative

# ------------------------------------------------------------ log probabilities
ROUND = 32768  # logits that a row's workgroup takes at a time


def logprobs(x, targets, n):
    """sh.logprobs' wanted values of finite or -inf logits, with tolerances by the depth of the sums.

    Z = sum e^d, d = x - max.  A thread adds 32 logits and one of the row's rest a round, one after another, and the
    threads', waves' and parts' sums meet in trees of 64: a term passes at most 33 rounds + 18 additions, each off by
    half a step of a sum no larger than Z (all terms are positive).  A term's exponent is d log2(e): d, the product and
    the constant are off by half a step each, |d| 2.5 U; the exponential by a step, 2 U.  A sum that moves to a larger
    maximum is multiplied by such an exponential, at most rounds + 3 times; the distances add up to |d|.
    entropy = log Z - E / Z, E = sum e^d d (all of one sign): its terms as Z's, weighed by |d|, and half a step more
    for the product.  The logarithm is off by at most four half steps of its result.
    """
    want = sh.logprobs(x, targets, n)
    x = x.astype(np.float64)
    V = x.shape[1]
    rounds = -(-V // ROUND)
    m = x.max(-1, keepdims=True)
    base = np.where(np.isneginf(m), 0, m)
    d = np.where(np.isneginf(x), 0, x - base)
    e = np.exp(x - base)
    z = e.sum(-1)
    zz = np.where(z == 0, 1, z)
    spread, second = (e * np.abs(d)).sum(-1) / zz, (e * d * d).sum(-1) / zz
    adds = 33 * rounds + 18
    rel = adds * U + spread * 2.5 * U + (rounds + 4) * 3 * U
    lz = np.abs(np.log(zz))
    fin = lambda a: np.where(np.isfinite(a), np.abs(a), 0)  # noqa: E731
    bl = rel + lz * 4 * U + fin(want["lse"][0]) * U
    be = rel + lz * 4 * U + spread * (rel + (adds + (rounds + 4) * 3 + 3) * U) + second * 2.5 * U \
        + (fin(want["entropy"][0]) + spread) * U
    return dict(logprob=(want["logprob"][0], bl + fin(want["logprob"][0]) * U), lse=(want["lse"][0], bl),
                entropy=(want["entropy"][0], be), top_ids=want["top_ids"],
                top_logprob=(want["top_logprob"][0], bl[:, None] + fin(want["top_logprob"][0]) * U))


def even_rows(V, level):
    """Tolerance of lse and entropy of V equal logits: every sum is a whole number, so only the logarithm (four half
    steps) and the last addition round."""
    return np.log(V) * 4 * U + abs(level + np.log(V)) * U


def edges(V, length):
    """Places where a row's walk can go wrong: its ends, the rest behind the last whole load of 4 and of 8, the borders
    of rounds, of 256 and 1024 threads' loads, and of parts of `length`."""
    at = {0, 1, V - 1, V - 2, V // 4 * 4, V // 8 * 8, V // 4 * 4 - 1, V // 8 * 8 - 1}
    for step in (ROUND, length, 8192, 4096, 2048, 1024):
        for k in range(step, V, step):
            if step >= 8192 or k <= 2 * step or k + 2 * step > V:
                at |= {k - 1, k, k + 1}
    return sorted(a for a in at if 0 <= a < V)


def part_length(T, V):
    """Logits a part of a row that is cut (few long rows)."""
    parts = min(256 // T, -(-V // (ROUND // 4)), 16)
    return -(-(-(-V // parts)) // 16) * 16


# -------------------------------------------------------------------- attention
def counting_cache(g, D, heads, lens, spare=2):
    """Keys that are all alike, so that every token seen has the same probability, and values that count: token j has
    127 at value j % D and zeros elsewhere.  A row's result is then how many of its tokens fall on each value, over
    their number.  Places behind the sequences hold other codes and NaN scales."""
    per = [-(-n // 64) for n in lens]
    pages = sum(per) + spare
    raw = g.integers(0, 256, (pages, heads, sh.record(D)), dtype=np.uint8)
    sc = raw[..., 128 * D:].view(np.float32)
    sc[:] = np.nan
    table = np.full((len(lens), max(per + [1])), -1, np.int32)
    order = g.permutation(pages).astype(np.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at: at + n]
        at += n
        for j in range(lens[b]):
            r = raw[table[b, j // 64]]
            r[:, : 64 * D].reshape(heads, D // 64, 64, 64)[:, :, j % 64] = 1
            v = r[:, 64 * D: 128 * D].reshape(heads, D, 64)
            v[:, :, sh.place(j % 64)] = 0
            v[:, j % D, sh.place(j % 64)] = 127
            r[:, 128 * D:].view(np.float32)[:, j % 64] = 0.01
            r[:, 128 * D:].view(np.float32)[:, 64 + j % 64] = 1.0
    return raw, table


def counted(D, L, n, window):
    """[n][D] results of a sequence's new tokens over counting_cache, and each one's number of tokens."""
    out, number = np.zeros((n, D)), np.zeros(n)
    for i in range(n):
        p = L - n + i
        j = np.arange(max(0, p - window + 1) if window else 0, p + 1)
        number[i] = len(j)
        if len(j):
            out[i] = 127.0 * np.bincount(j % D, minlength=D) / len(j)
    return out, number


def lane_adds(L):
    """Probabilities that a lane adds one after another, and the trees behind: a fourth of a page's tokens, of a whole
    tile's pages (33 at most: longer ones are cut; a chunk of these tests' lengths has no more)."""
    return min(-(-L // 4), 33 * 16) + 32


def counting_bound(dtype, D, L):
    """Relative: all probabilities are one number.  It enters as two fp16 pieces (2^-21) or as one (2^-11, bf16
    results).  Sums of equal terms are rounded alike at every addition, so these count in full: a value's, one term a
    piece every D tokens, and those of the probabilities; then the division and the result's rounding."""
    return (2.0 ** -11 if dtype == "bf16" else 2.0 ** -21) + (2 * -(-L // D) + lane_adds(L) + 16) * U + sh.HALF_STEP[dtype]


def counting_lse_bound(qx, s, L, D):
    """The score's pieces and its sum's roundings, the probabilities' sum, and log2, its product and the sum, four
    half steps each.  qx: the queries, s: their scores, of keys of 0.01."""
    S = np.abs(qx.astype(np.float64)).sum(-1) * 0.01 * D ** -0.5
    return S * (2.0 ** -21 + 16 * U) + lane_adds(L) * U + (np.abs(s) + np.log(max(L, 1)) + 1) * 8 * U


def rms_limit(scores):
    """What the relative RMS error of fp32 results may be, with random values: a result's relative error is its
    probabilities' (those of the tokens are independent).  `scores`: the seen ones, natural.  A score of size s is off
    by its query's pieces, 2^-21 s, and at most 16 roundings of fp32 sums, 16 U s; a probability by its pieces (2^-21),
    the exponential and six more roundings (8 U)."""
    s = np.sqrt(np.mean(np.square(scores)))
    return s * (2.0 ** -21 + 16 * U) + 2.0 ** -21 + 8 * U


def rms(got, want):
    return float(np.sqrt(np.mean(np.square(got - want)) / np.mean(np.square(want))))


def rms_limit_lse(scores, lse):
    """The same of lse, absolute: a score's error, that of the sums and four half steps of log2, its product and the sum."""
    s = np.sqrt(np.mean(np.square(scores)))
    return s * (2.0 ** -21 + 16 * U) + 16 * U + np.sqrt(np.mean(np.square(lse))) * 8 * U
