"""Plain numpy forms of the operators between the projections (the paged 8-bit
key/value cache, attention over it, log probabilities), and their error bounds.

The cache's codes are decided in fp32 on both sides (one rounding an
operation), so they are compared exactly; attention and log probabilities are
computed in 64 bits.  Nothing here shares code with the library.
"""
from __future__ import annotations

import numpy as np

import census
import gpu_helpers
from gpu_helpers import host, to_dev  # noqa: F401

PAGE = 64
OPS = ("q8k_kv_append", "q8k_kv_read", "qattend", "qlogprobs")
DTYPES = ("f32", "f16", "bf16")
# half a step of each type, relative to the value
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


class _Tracked(census._Tracked):
    """census._Tracked with these operators noted too."""

    def __getattr__(self, name):
        v = getattr(self._q, name)
        if name not in OPS:
            return super().__getattr__(name)

        def call(*a, **k):
            try:
                return v(*a, **k)
            finally:
                census.CENSUS.note(self._q.q8k_debug_last_launches())

        return call


def tracked(q):
    return _Tracked(q)


def q_dtype(q, name):
    return {"f32": q.Q8K_F32, "f16": q.Q8K_F16, "bf16": q.Q8K_BF16}[name]


def torch_dtype(name):
    import torch

    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def round_to(x: np.ndarray, dtype: str) -> np.ndarray:
    """fp32 values rounded to the type (to nearest even), as fp32."""
    import torch

    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch_dtype(dtype)).float().numpy()


def to_dev_as(x: np.ndarray, dtype: str):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch_dtype(dtype)).cuda()


def back(t) -> np.ndarray:
    import torch

    torch.cuda.synchronize()
    return t.float().cpu().numpy()


# ------------------------------------------------------------------ the cache
def place(t):
    return ((t >> 2) & 3) << 4 | (t >> 5) << 3 | ((t >> 4) & 1) << 2 | (t & 3)


def record(D):
    return 2 * PAGE * D + 8 * PAGE


def rope_table(g, positions, dim):
    """Any angles will do: one row a position, cosines then sines."""
    a = g.uniform(-np.pi, np.pi, size=(positions, dim // 2))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def rotate(x, table, pos, pairs):
    """x [T][heads][D] turned by its positions, each product and sum rounded to x's own type."""
    if table is None:
        return x
    dim = table.shape[1]
    c = table[pos, : dim // 2].astype(x.dtype)[:, None]
    s = table[pos, dim // 2:].astype(x.dtype)[:, None]
    y = x.copy()
    i = np.arange(dim // 2)
    ia, ib = (i, i + dim // 2) if pairs == "half" else (2 * i, 2 * i + 1)
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = a * s + b * c
    return y


def quantise(x):
    """fp32 rows -> (int8 codes, fp32 scales), q8_K's rule."""
    x = x.astype(np.float32)
    amax = np.abs(x).max(-1)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        r = np.rint(x * (np.float32(127.0) / amax)[..., None])
    r = np.clip(np.nan_to_num(r, nan=0.0, posinf=127, neginf=-127), -127, 127)
    r[amax == 0] = 0
    return r.astype(np.int8), (amax / np.float32(127.0)).astype(np.float32)


def append(cache, k, v, table, pos, pairs, slots, D):
    """Writes into `cache`, uint8 [pages][heads][record(D)], what q8k_kv_append should."""
    pages = cache.shape[0]
    kq, ks = quantise(rotate(k.astype(np.float32), table, np.clip(pos, 0, (len(table) if table is not None else 1) - 1), pairs))
    vq, vs = quantise(v)
    for t, slot in enumerate(slots):
        if slot < 0 or slot >= pages * PAGE or (table is not None and not 0 <= pos[t] < len(table)):
            continue
        p, j = divmod(int(slot), PAGE)
        for h in range(cache.shape[1]):
            r = cache[p, h]
            r[: PAGE * D].reshape(D // 64, PAGE, 64)[:, j] = kq[t, h].view(np.uint8).reshape(D // 64, 64)
            r[PAGE * D: 2 * PAGE * D].reshape(D, PAGE)[:, place(j)] = vq[t, h].view(np.uint8)
            r[2 * PAGE * D:].view(np.float32)[j] = ks[t, h]
            r[2 * PAGE * D:].view(np.float32)[PAGE + j] = vs[t, h]


def held(cache, slots, D):
    """(codes, scales) of keys and values at slots: int8 [T][heads][D], fp32 [T][heads], twice."""
    T, H = len(slots), cache.shape[1]
    k, v = np.zeros((T, H, D), np.int8), np.zeros((T, H, D), np.int8)
    ks, vs = np.zeros((T, H), np.float32), np.zeros((T, H), np.float32)
    for t, slot in enumerate(slots):
        if slot < 0 or slot >= cache.shape[0] * PAGE:
            continue
        p, j = divmod(int(slot), PAGE)
        for h in range(H):
            r = cache[p, h]
            k[t, h] = r[: PAGE * D].reshape(D // 64, PAGE, 64)[:, j].reshape(-1).view(np.int8)
            v[t, h] = r[PAGE * D: 2 * PAGE * D].reshape(D, PAGE)[:, place(j)].view(np.int8)
            ks[t, h], vs[t, h] = r[2 * PAGE * D:].view(np.float32)[[j, PAGE + j]]
    return k, ks, v, vs


# -------------------------------------------------------------------- attention
def attend(q, cu_q, cache, table_of_pages, kv_len, scale, window, rope, pos, pairs, D, dtype):
    """-> (out, lse, bound of out, bound of lse), 64 bits; rows of no sequence are NaN in all four.

    Bounds.  fp16 has 11 significant bits, so rounding to nearest is off by at
    most 2^-11 of the value, truncating by 2^-10, and two pieces, the second the
    rounded rest of a truncated first, by 2^-10 * 2^-11 = 2^-21.  With S_j = scale * sum_d |q_d k_d|: a
    score's error is at most S_j times that of q's two pieces (2^-21), of the
    fp32 sum of 2 D products (2 D 2^-24) and of ten more fp32 roundings
    (rotation, scale, log2 e, key scale, the exponent's argument); a
    probability's relative error is twice the largest score error (numerator
    and sum), its pieces' (2^-21, or 2^-11 for the one piece of a bf16
    result) and a few roundings; the sums over `len` tokens, in any order, add
    len 2^-24.  exp's own error: 2^-22.
    """
    Tq, Hq, _ = q.shape
    H = cache.shape[1]
    G = Hq // H
    out = np.full((Tq, Hq, D), np.nan)
    lse = np.full((Tq, Hq), np.nan)
    bo, bl = out.copy(), lse.copy()
    piece = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -21
    for b in range(len(kv_len)):
        q0, n, L = cu_q[b], cu_q[b + 1] - cu_q[b], int(kv_len[b])
        if n == 0:
            continue
        j = np.arange(L)
        pages = table_of_pages[b][j // PAGE].astype(np.int64)
        good = (pages >= 0) & (pages < cache.shape[0])
        slots = np.where(good, pages * PAGE + j % PAGE, -1)
        kc, ks, vc, vs = held(cache, slots, D)
        k = kc.astype(np.float64) * ks[..., None]
        v = vc.astype(np.float64) * vs[..., None]
        x = rotate(q[q0: q0 + n].astype(np.float64), rope, pos[q0: q0 + n] if pos is not None else None, pairs)
        p = np.arange(L - n, L)[:, None]
        seen = good & (j <= p)
        if window:
            seen &= j > p - window
        some = seen.any(1)
        count = seen.sum(1)[:, None]
        for a in range(Hq):
            h, rows = a // G, slice(q0, q0 + n)
            # unseen places may hold anything: out of every sum and maximum
            kk, vv = np.where(good[:, None], k[:, h], 0), np.where(good[:, None], v[:, h], 0)
            s = np.where(seen, x[:, a] @ kk.T * scale, -np.inf)
            S = np.where(seen, np.abs(x[:, a]) @ np.abs(kk).T, 0).max(1, initial=0)[:, None] * abs(scale)
            m = np.where(some, s.max(1, initial=-np.inf), 0)[:, None]
            w = np.exp(s - m)
            z = w.sum(1, keepdims=True)
            w = w / np.where(z == 0, 1, z)
            out[rows, a] = w @ vv
            with np.errstate(divide="ignore"):
                lse[rows, a] = (m + np.log(z))[:, 0]
            ds = S * (2.0 ** -21 + (2 * D + 10) * 2.0 ** -24) + 2.0 ** -22
            A = w @ np.abs(vv)
            # the pieces' smallest step: 2^-40 of the largest share
            vmax = np.where(seen, np.abs(vv).max(1), 0).max(1, initial=0)[:, None]
            bo[rows, a] = A * (2 * ds + piece + (count + 64) * 2.0 ** -24) + 2.0 ** -40 * count * vmax
            bo[rows, a] += np.abs(out[rows, a]) * HALF_STEP[dtype] + (2.0 ** -25 if dtype == "f16" else 0)
            fin = np.where(some, lse[rows, a], 0)[:, None]
            bl[rows, a] = (ds + (count + 16) * 2.0 ** -24 + np.abs(fin) * 2.0 ** -22 + np.abs(m) * 2.0 ** -22)[:, 0]
            bo[rows, a][~some] = 0
    return out, lse, bo, bl


def logprobs(x, targets, n):
    """-> dict of (want, bound) and top ids, 64 bits, of fp32 logits x [T][V].

    Bounds: e^(x - m) has a relative error of the argument's rounding, |x - m|
    2^-23 and the exponential's 2^-22 - weighed by e^(x - m) itself, sum e^d |d|
    / Z is the entropy's own scale; the sums' of V terms are taken about the
    chunks' maxima, V 2^-24 in any order.
    """
    x = x.astype(np.float64)
    T, V = x.shape
    m = x.max(-1, keepdims=True)
    base = np.where(np.isneginf(m), 0, m)
    d = x - base
    e = np.exp(d)
    z = e.sum(-1)
    with np.errstate(divide="ignore", invalid="ignore"):
        lse = np.where(z == 0, -np.inf, base[:, 0] + np.log(z))
        ed = np.where(e > 0, e * np.where(np.isneginf(d), 0, d), 0)
        zz = np.where(z == 0, 1, z)
        entropy = np.where(z == 0, 0, np.log(zz) - ed.sum(-1) / zz)
        spread = np.abs(ed).sum(-1) / zz
        rel = (V + 64) * 2.0 ** -24 + spread * 2.0 ** -22 + 2.0 ** -21  # of Z
        order = np.argsort(-np.where(np.isnan(x), -np.inf, x), axis=-1, kind="stable")[:, :n]
        top = np.take_along_axis(x, order, -1)
        lsee = np.where(np.isinf(lse), 0, lse)
        ok = (targets >= 0) & (targets < V)
        xt = x[np.arange(T), np.clip(targets, 0, V - 1)]
        lp = np.where(ok, np.where(z == 0, -np.inf, xt - lse), np.nan)
        tl = np.where((z == 0)[:, None], -np.inf, top - lse[:, None])
    bl = rel + np.abs(lsee) * 2.0 ** -23 + np.abs(base[:, 0]) * 2.0 ** -23
    # e d: its own exponent error, |d| 2^-23 + 2^-22, once more by |d|
    be = rel * (1 + spread) + (np.abs(ed) * (np.abs(np.where(np.isneginf(d), 0, d)) * 2.0 ** -22)).sum(-1) / zz \
        + np.abs(entropy) * 2.0 ** -22 + spread * (V + 64) * 2.0 ** -24 + 2.0 ** -22
    fin = lambda a: np.where(np.isfinite(a), a, 0)  # noqa: E731
    return dict(logprob=(lp, bl + np.abs(fin(lp)) * 2.0 ** -23 + np.abs(fin(xt)) * 2.0 ** -24), lse=(lse, bl),
                entropy=(entropy, be), top_ids=order.astype(np.int32),
                top_logprob=(tl, bl[:, None] + np.abs(fin(tl)) * 2.0 ** -23))


def assert_within(got, want, bound, what=""):
    """|got - want| <= bound element by element; infinities and NaN in the same
    places.  A value check against the plain form: credits the pending kernels."""
    got = np.asarray(got, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), f"{what}: infinities differ"
    err = np.abs(got[fine] - want[fine])
    b = np.broadcast_to(bound, want.shape)[fine]
    bad = err > b
    if bad.any():
        i = np.argmax(err / np.maximum(b, 1e-300))
        at = np.argwhere(fine)[i]
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} out of bounds; worst at {tuple(at)}: got "
                             f"{got[fine][i]!r} want {want[fine][i]!r} err {err[i]:.3g} bound {b[i]:.3g}")
    census.CENSUS.credit()


assert_exact = gpu_helpers.assert_exact
