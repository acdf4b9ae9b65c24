"""Plain numpy forms of the operators for long contexts (the paged 4-bit cache and
attention over it, accumulated attention weights, eviction), and their error bounds.

What is decided in fp32 (codes, factors, scales) or only moved is compared
exactly; attention and weights are computed in 64 bits.  Nothing here shares code
with the library.
"""
from __future__ import annotations

import numpy as np

import census
import serving_helpers as sh
from serving_helpers import HALF_STEP, PAGE

OPS = ("q8k_kv4_append", "q8k_kv4_read", "qattend_kv4", "qattend_weights", "q8k_kv_evict")


class _Tracked(sh._Tracked):
    """serving_helpers._Tracked with these operators noted too."""

    def __getattr__(self, name):
        if name not in OPS:
            return super().__getattr__(name)
        v = getattr(self._q, name)

        def call(*a, **k):
            try:
                return v(*a, **k)
            finally:
                census.CENSUS.note(self._q.q8k_debug_last_launches())

        return call


def tracked(q):
    return _Tracked(q)


# ------------------------------------------------------------------ the caches
def place(bits, t):
    if bits == 8:
        return sh.place(t)
    return ((t >> 2) & 3) << 4 | (t >> 5) << 3 | ((t >> 4) & 1) << 2 | (t & 1) << 1 | ((t >> 1) & 1)


def record(bits, D):
    return sh.record(D) if bits == 8 else 68 * D + 8 * PAGE


def factor_values():
    """The 256 factors: four bits of exponent, four of mantissa."""
    e, m = np.divmod(np.arange(256), 16)
    return np.where(e > 0, (16.0 + m) * 2.0 ** (e - 19), m * 2.0 ** -18)


FACTORS = factor_values()


def quantise4(x):
    """fp32 rows -> codes [-7, 7], factors' bytes [.., D/32], fp32 scales."""
    f32 = np.float32
    x = x.astype(f32)
    g = x.reshape(*x.shape[:-1], -1, 32)
    with np.errstate(all="ignore"):
        top = np.nan_to_num(np.fmax.reduce(np.abs(g), -1), nan=0.0, posinf=np.inf)
        amax = top.max(-1)
        scale = (amax / f32(7)).astype(f32)
        r = (top / amax[..., None]).astype(f32)
        r = np.where(r > 0, r, 0)  # NaN too
        byte = np.searchsorted(FACTORS[:241], r.astype(np.float64))  # the least that is not below
        step = (FACTORS.astype(f32)[byte] * scale[..., None]).astype(f32)
        inverse = (f32(1) / step).astype(f32)
        none = (byte == 0) | ~np.isfinite(scale)[..., None]
        c = np.rint((g * inverse[..., None]).astype(f32))
        c = np.where(np.isinf(inverse)[..., None], np.sign(g) * 7, c)
        c = np.where(none[..., None] | np.isnan(g) | np.isnan(c), 0, c)
    return c.astype(np.int8).reshape(x.shape), byte.astype(np.uint8), scale


def key_bits(D, t, i):
    """(byte of the word, bit of it) of value i of token t's key, byte counted in the record."""
    s, h, w, j = i // 64, i % 64 // 16, i % 16 // 8, i % 8
    p = t // 16 * (D // 64) + s
    return p // 2 * 1024 + t % 16 * 64 + h * 16 + p % 2 * 8 + w * 4, (4 * (j // 2 + 4 * (j % 2)) + 2) % 32


def put_token(bits, r, D, t, kc, kf, ks, vc, vf, vs):
    """Writes one token into a record (uint8 [record])."""
    if bits == 8:
        r[: PAGE * D].reshape(D // 64, PAGE, 64)[:, t] = kc.view(np.uint8).reshape(D // 64, 64)
        r[PAGE * D: 2 * PAGE * D].reshape(D, PAGE)[:, place(8, t)] = vc.view(np.uint8)
    else:
        at, bit = key_bits(D, t, np.arange(D))
        u = (kc.astype(np.uint64) + np.uint64(8) & np.uint64(15)) << bit.astype(np.uint64)
        word = np.bitwise_or.reduce((u | u >> np.uint64(32)).reshape(-1, 8), 1).astype(np.uint32)
        r[at[::8, None] + np.arange(4)] = word.view(np.uint8).reshape(-1, 4)
        u = (vc.astype(np.int64) + 8).reshape(D // 32, 2, 16)
        r[32 * D: 64 * D].reshape(D // 32, 16, PAGE)[:, :, place(4, t)] = u[:, 0] | u[:, 1] << 4
        for y in range(D // 32):
            r[64 * D: 66 * D].reshape(16, 2, 4, D // 64)[t % 16, y % 2, t // 16, y // 2] = kf[y]
            r[66 * D: 68 * D].reshape(D // 32, PAGE)[y, place(4, t)] = vf[y]
    r[record(bits, D) - 8 * PAGE:].view(np.float32)[[t, PAGE + t]] = ks, vs


def get_token(bits, r, D, t):
    """(key codes * factors, key scale, value codes * factors, value scale): 64 bits, exact."""
    s = r[record(bits, D) - 8 * PAGE:].view(np.float32)
    if bits == 8:
        k = r[: PAGE * D].reshape(D // 64, PAGE, 64)[:, t].reshape(-1).view(np.int8)
        v = r[PAGE * D: 2 * PAGE * D].reshape(D, PAGE)[:, place(8, t)].copy().view(np.int8)
        return k.astype(np.float64), s[t], v.astype(np.float64), s[PAGE + t]
    i = np.arange(D)
    at, bit = key_bits(D, t, i)
    w = r[(at[:, None] + np.arange(4))].astype(np.uint64)
    w = w[:, 0] | w[:, 1] << np.uint64(8) | w[:, 2] << np.uint64(16) | w[:, 3] << np.uint64(24)
    k = (((w | w << np.uint64(32)) >> bit.astype(np.uint64)) & np.uint64(15)).astype(np.float64) - 8
    b = r[32 * D: 64 * D].reshape(D // 32, 16, PAGE)[:, :, place(4, t)]
    v = np.stack([b & 15, b >> 4], 1).reshape(-1).astype(np.float64) - 8
    y = np.arange(D // 32)
    kf = FACTORS[r[64 * D: 66 * D].reshape(16, 2, 4, D // 64)[t % 16, y % 2, t // 16, y // 2]]
    vf = FACTORS[r[66 * D: 68 * D].reshape(D // 32, PAGE)[:, place(4, t)]]
    return k * np.repeat(kf, 32), s[t], v * np.repeat(vf, 32), s[PAGE + t]


def append4(cache, k, v, table, pos, pairs, slots, D):
    """Writes into `cache`, uint8 [pages][heads][record], what q8k_kv4_append should."""
    pages = cache.shape[0]
    some = np.clip(pos, 0, (len(table) if table is not None else 1) - 1)
    kc, kf, ks = quantise4(sh.rotate(k.astype(np.float32), table, some, pairs))
    vc, vf, vs = quantise4(v)
    for t, slot in enumerate(slots):
        if slot < 0 or slot >= pages * PAGE or (table is not None and not 0 <= pos[t] < len(table)):
            continue
        p, j = divmod(int(slot), PAGE)
        for h in range(cache.shape[1]):
            put_token(4, cache[p, h], D, j, kc[t, h], kf[t, h], ks[t, h], vc[t, h], vf[t, h], vs[t, h])


def held(bits, cache, slots, D):
    """(codes * factors in 64 bits, scales) of keys and values at slots: [T][heads][D], fp32 [T][heads], twice."""
    slots = np.asarray(slots, np.int64)
    good = (slots >= 0) & (slots < cache.shape[0] * PAGE)
    page, t = np.divmod(np.where(good, slots, 0), PAGE)
    if (bits, D) not in _BYTES:
        _BYTES[bits, D] = token_bytes(bits, D)
    raw = cache[page[:, None, None], np.arange(cache.shape[1])[None, :, None], _BYTES[bits, D][t][:, None]] if len(cache) \
        else np.zeros((len(slots), cache.shape[1], _BYTES[bits, D].shape[1]), np.uint8)
    raw = np.where(good[:, None, None], raw, 0)
    s = np.ascontiguousarray(raw[..., -8:]).view(np.float32)
    if bits == 8:
        k, v = (np.ascontiguousarray(x).view(np.int8).astype(np.float64) for x in (raw[..., :D], raw[..., D: 2 * D]))
        return k, s[..., 0], v, s[..., 1]
    n, G = D // 2, D // 32
    w = np.ascontiguousarray(raw[..., :n]).view(np.uint32).astype(np.uint64)[..., None]
    bit = np.array([(4 * (j // 2 + 4 * (j % 2)) + 2) % 32 for j in range(8)], np.uint64)
    k = ((w | w << np.uint64(32)) >> bit & np.uint64(15)).astype(np.float64).reshape(*raw.shape[:2], D) - 8
    b = raw[..., n: 2 * n].reshape(*raw.shape[:2], G, 1, 16)
    v = np.concatenate([b & 15, b >> 4], -2).reshape(*raw.shape[:2], D).astype(np.float64) - 8
    kf, vf = FACTORS[raw[..., 2 * n: 2 * n + G]], FACTORS[raw[..., 2 * n + G: 2 * n + 2 * G]]
    live = good[:, None, None]
    return np.where(live, k * np.repeat(kf, 32, -1), 0), s[..., 0], np.where(live, v * np.repeat(vf, 32, -1), 0), s[..., 1]


def random_cache(g, bits, pages, heads, D):
    """Random bytes whose scales are NaN (places that no sequence has); codes and factors any."""
    raw = g.integers(0, 256, (pages, heads, record(bits, D)), dtype=np.uint8)
    if bits == 8:
        codes = raw[..., : 2 * PAGE * D].view(np.int8)
        codes[codes == -128] = -127
    else:
        f = raw[..., 64 * D: 68 * D]
        f[f > 0xf0] = 0xf0
    raw[..., record(bits, D) - 8 * PAGE:].view(np.float32)[:] = np.nan
    return raw


def paged(g, bits, D, heads, lens, news, spare=3, spread=1.0):
    """A random cache, scales where the sequences' tokens are, its page table (places beyond a sequence's pages point
    outside the cache) and the new tokens' starts."""
    per = [-(-n // PAGE) for n in lens]
    pages = sum(per) + spare
    raw = random_cache(g, bits, pages, heads, D)
    if bits == 4:  # factors as they are: between 1/4 and 1 of the row's largest, and a few small ones
        f = raw[..., 64 * D: 68 * D]
        small = g.random(f.shape) < 0.05
        f[:] = np.where(small, f, 0xd0 + f % 33)
    sc = raw[..., record(bits, D) - 8 * PAGE:].view(np.float32)
    unit = 73 if bits == 8 else 4
    order = g.permutation(pages).astype(np.int32)
    table = np.full((len(lens), max(per + [1])), -1, np.int32)
    table[:, 1::2] = 2 ** 30
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at: at + n]
        at += n
        for i in range(lens[b]):
            r = sc[table[b, i // PAGE]]
            r[:, i % PAGE] = g.uniform(0.2, 2.0, heads) / unit * spread
            r[:, PAGE + i % PAGE] = 10.0 ** g.uniform(-3, 1, heads) / unit
    return raw, table, np.concatenate([[0], np.cumsum(news)]).astype(np.int32)


# -------------------------------------------------------------------- attention
def _sequences(q, cu_q, bits, cache, table_of_pages, kv_len, scale, window, rope, pos, pairs, D):
    """For each sequence with new tokens: (b, first row, rows, length, seen [n][L], keys, values [L][heads][D],
    queries [n][heads][D]), unseen places zeros."""
    for b in range(len(kv_len)):
        q0, n, L = cu_q[b], cu_q[b + 1] - cu_q[b], int(kv_len[b])
        if n == 0:
            continue
        j = np.arange(L)
        pages = table_of_pages[b][j // PAGE].astype(np.int64)
        good = (pages >= 0) & (pages < cache.shape[0])
        kc, ks, vc, vs = held(bits, cache, np.where(good, pages * PAGE + j % PAGE, -1), D)
        p = np.arange(L - n, L)[:, None]
        seen = good & (j <= p)
        if window:
            seen &= j > p - window
        x = sh.rotate(q[q0: q0 + n].astype(np.float64), rope, pos[q0: q0 + n] if pos is not None else None, pairs)
        any_row = seen.any(0)[:, None, None]
        with np.errstate(invalid="ignore"):
            k = np.where(any_row, kc * ks[..., None].astype(np.float64), 0)
            v = np.where(any_row, vc * vs[..., None].astype(np.float64), 0)
        yield b, q0, n, L, seen, k, v, x


def score_error(x, k, seen, scale, D):
    """What a score can be off by (serving_helpers.attend): [n][1], natural."""
    S = np.where(seen, np.abs(x) @ np.abs(k).T, 0).max(1, initial=0)[:, None] * abs(scale)
    return S * (2.0 ** -21 + (2 * D + 10) * 2.0 ** -24) + 2.0 ** -22


def attend(bits, q, cu_q, cache, table_of_pages, kv_len, scale, window, rope, pos, pairs, D, dtype):
    """-> (out, lse, bound of out, bound of lse), 64 bits; rows of no sequence are NaN in all four.

    The bounds are serving_helpers.attend's: the operand code * factor is exact in fp16 as a code is.  What fp16's
    smallest step loses of a probability is 2^-40 of the unit, at most twice the largest value scale seen, times the
    operand, at most 8: 2^-36 of that scale."""
    Tq, Hq, _ = q.shape
    G = Hq // cache.shape[1]
    out, lse = np.full((Tq, Hq, D), np.nan), np.full((Tq, Hq), np.nan)
    bo, bl = out.copy(), lse.copy()
    piece = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -21
    for b, q0, n, L, seen, k, v, x in _sequences(q, cu_q, bits, cache, table_of_pages, kv_len, scale, window, rope, pos,
                                                 pairs, D):
        some, count = seen.any(1), seen.sum(1)[:, None]
        for a in range(Hq):
            h, rows = a // G, slice(q0, q0 + n)
            kk, vv = k[:, h], v[:, h]
            s = np.where(seen, x[:, a] @ kk.T * scale, -np.inf)
            m = np.where(some, s.max(1, initial=-np.inf), 0)[:, None]
            w = np.exp(s - m)
            z = w.sum(1, keepdims=True)
            w = w / np.where(z == 0, 1, z)
            out[rows, a] = w @ vv
            with np.errstate(divide="ignore"):
                lse[rows, a] = (m + np.log(z))[:, 0]
            ds = score_error(x[:, a], kk, seen, scale, D)
            vmax = np.where(seen, np.abs(vv).max(1), 0).max(1, initial=0)[:, None]
            bo[rows, a] = (w @ np.abs(vv)) * (2 * ds + piece + (count + 64) * 2.0 ** -24) + 2.0 ** -36 * count * vmax
            bo[rows, a] += np.abs(out[rows, a]) * HALF_STEP[dtype] + (2.0 ** -25 if dtype == "f16" else 0)
            fin = np.where(some, lse[rows, a], 0)[:, None]
            bl[rows, a] = (ds + (count + 16) * 2.0 ** -24 + np.abs(fin) * 2.0 ** -22 + np.abs(m) * 2.0 ** -22)[:, 0]
            bo[rows, a][~some] = 0
    return out, lse, bo, bl


def weights(bits, q, cu_q, cache, table_of_pages, kv_len, scale, window, rope, pos, pairs, D, lse, old, keep, served=None):
    """-> (weights, bound) of q8k's [B][heads][L] for the tokens of each sequence, NaN behind them, with the fp32 lse
    that the kernel is given.  served: new tokens of a sequence that count at most.

    A term e^(s - lse) is relatively off by its score's error, by what the fused s log2 e unit - lse log2 e rounds (one
    step of the larger, one more of lse log2 e and of the unit each: 2^-23 (|s| + |lse|) at most) and by the
    exponential's 2^-22; the sum over R rows by R 2^-24 in any order; keep old by a rounding and the last sum by one."""
    B, H = len(kv_len), cache.shape[1]
    G = q.shape[1] // H
    longest = max([int(n) for n in kv_len] + [1])
    got, bound = np.full((B, H, longest), np.nan), np.zeros((B, H, longest))
    for b in range(B):
        L, n = int(kv_len[b]), int(cu_q[b + 1] - cu_q[b])
        got[b, :, :L] = 0
        if old is not None and L > n:
            # (keep is a float at the interface: 0.9 is 2.6e-8 of itself off, which no rounding of the kernel's is)
            got[b, :, : L - n] = np.float64(np.float32(keep)) * old[b, :, : L - n].astype(np.float64)
    for b, q0, n, L, seen, k, v, x in _sequences(q, cu_q, bits, cache, table_of_pages, kv_len, scale, window, rope, pos,
                                                 pairs, D):
        rows = min(n, served) if served is not None else n
        seen, x = seen[:rows], x[:rows]
        for a in range(q.shape[1]):
            h = a // G
            l = lse[q0: q0 + rows, a].astype(np.float64)[:, None]
            s = x[:, a] @ k[:, h].T * scale
            with np.errstate(invalid="ignore", over="ignore"):
                p = np.where(seen & ~np.isneginf(l), np.exp(s - np.where(np.isneginf(l), 0, l)), 0)
            rel = score_error(x[:, a], k[:, h], seen, scale, D) + 2.0 ** -23 * (np.abs(s) + np.where(np.isneginf(l), 0, np.abs(l))) + 2.0 ** -22
            got[b, h, :L] += p.sum(0)
            bound[b, h, :L] += (p * rel).sum(0) + p.sum(0) * (rows * G + 8) * 2.0 ** -24
    fin = np.where(np.isfinite(got), np.abs(got), 0)
    return got, bound + fin * 2.0 ** -23 + 2.0 ** -126


# --------------------------------------------------------------------- eviction
def choose(w, L, budget, first, last):
    """Old indices of the kept tokens of one row of weights."""
    if L <= budget:
        return np.arange(L)
    inner = np.arange(first, L - last)
    x = w[first: L - last].astype(np.float64)
    key = np.where(np.isnan(x), -np.inf, x)
    # largest first, NaN behind -inf, equal ones by ascending index
    order = np.lexsort((inner, np.isnan(x), -key))[: budget - first - last]
    return np.sort(np.concatenate([np.arange(first), inner[order], np.arange(L - last, L)]))


def evict(bits, cache, table, lens, w, budget, first, last, out_table, D):
    """-> (cache, kept [B][heads][budget], kept weights (NaN where none), new lengths)."""
    B, H = len(lens), cache.shape[1]
    new = cache.copy()
    kept = np.full((B, H, budget), -1, np.int32)
    out_w = np.full((B, H, budget), np.nan, np.float32)
    for b in range(B):
        for h in range(H):
            at = choose(w[b, h], int(lens[b]), budget, first, last)
            kept[b, h, : len(at)] = at
            out_w[b, h, : len(at)] = w[b, h, at]
            for i, j in enumerate(at):
                to, src = int(out_table[b, i // PAGE]), int(table[b, j // PAGE])
                if 0 <= to < cache.shape[0]:
                    r = cache[src, h] if 0 <= src < cache.shape[0] else np.zeros(cache.shape[2], np.uint8)
                    move_token(bits, D, r, int(j) % PAGE, new[to, h], i % PAGE)
    return new, kept, out_w, np.minimum(lens, budget).astype(np.int32)


def token_bytes(bits, D):
    """[64 tokens][bytes]: where each token's bytes of a record lie."""
    t = np.arange(PAGE)[:, None]
    i = np.arange(D)
    if bits == 8:
        k, v = i // 64 * 4096 + t * 64 + i % 64, PAGE * D + i * PAGE + place(8, t)
        parts = [k, v]
    else:
        word = np.array([[key_bits(D, a, b)[0] for b in range(0, D, 8)] for a in range(PAGE)])
        k = (word[:, :, None] + np.arange(4)).reshape(PAGE, -1)
        y, n = np.arange(D // 32), np.arange(D // 2)
        parts = [k, 32 * D + n * PAGE + place(4, t),
                 64 * D + ((t % 16 * 2 + y % 2) * 4 + t // 16) * (D // 64) + y // 2, 66 * D + y * PAGE + place(4, t)]
    end = record(bits, D) - 8 * PAGE
    four = np.arange(4)
    return np.concatenate(parts + [end + 4 * t + four, end + 256 + 4 * t + four], 1)


_BYTES = {}


def move_token(bits, D, src, j, dst, i):
    if (bits, D) not in _BYTES:
        _BYTES[bits, D] = token_bytes(bits, D)
    at = _BYTES[bits, D]
    dst[at[i]] = src[at[j]]
