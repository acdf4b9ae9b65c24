"""The paged 4-bit cache and attention over it on the GPU, against plain numpy
forms (long_helpers.py): the cache byte for byte, attention within bounds
derived there."""
import numpy as np
import pytest

import long_helpers as lh
import serving_helpers as sh
from gpu_helpers import host, poisoned, to_dev
from serving_helpers import assert_exact, assert_within, back, q_dtype, round_to, to_dev_as, torch_dtype
from test_gpu_serving import APPEND, ATTEND, append_case, rope_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_q8kpack_fp32_amd as q

    return lh.tracked(q)


def cache4(q, raw, D):
    return q.KVCache(to_dev(raw), raw.shape[0], raw.shape[1], D, bits=4)


def fresh(pages, heads, D):
    return np.full((pages, heads, lh.record(4, D)), 0xFF, np.uint8)


def bytes_of(kv, D):
    return host(kv.data)[: kv.pages * kv.kv_heads * lh.record(4, D)].reshape(kv.pages, kv.kv_heads, -1)


# ---------------------------------------------------------------------- append
@pytest.mark.parametrize("D,dtype,pairs,rot,heads,T", APPEND)
@pytest.mark.parametrize("scattered", [True, False])
def test_append(q, D, dtype, pairs, rot, heads, T, scattered):
    g, row, pages, slots = append_case(D, dtype, heads, T, 11 + T, scattered)
    row[..., ::13] *= 8  # channels that stand out: factors of all sizes
    row[..., 32:40] *= 2.0 ** -9
    row = round_to(row, dtype)
    if not scattered and T > 200:
        slots[100:] += 5
        slots[150:] += 64
        slots[170:180] = slots[170:180][::-1].copy()
    table = sh.rope_table(g, 300, rot) if rot else None
    pos = g.integers(0, 300, T).astype(np.int32)
    if T > 16 and rot:
        pos[9], pos[10] = 300, -1  # outside the table: not written
    want = fresh(pages, heads, D)
    lh.append4(want, row[:, heads: 2 * heads], row[:, 2 * heads:], table, pos, pairs, slots, D)
    kv = cache4(q, fresh(pages, heads, D), D)
    rd = to_dev_as(row, dtype)
    q.q8k_kv4_append(q_dtype(q, dtype), rd[:, heads: 2 * heads], 3 * heads * D, rd[:, 2 * heads:], 3 * heads * D, T,
                     to_dev(pos), rope_of(q, table, pairs), to_dev(slots), kv)
    assert_exact(bytes_of(kv, D), want, f"cache {D} {dtype} {pairs} {rot}")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", sh.DTYPES)
def test_append_tiles(q, D, dtype):
    """The kernel for many tokens, of every type: its last tile of three tokens."""
    test_append(q, D, dtype, "half", D // 2, 32, 259, False)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T", [12, 8300])
def test_append_odd_rows(q, D, T):
    """NaN, infinities, zeros, values whose step's reciprocal overflows, groups far below the row's largest."""
    g = np.random.default_rng(D)
    row = g.standard_normal((T, 2, D)).astype(np.float32)
    row[0, :, 5] = np.nan
    row[1, :, 7] = np.inf
    row[2, 0, 7], row[2, 1, 8] = -np.inf, np.nan
    row[3] = np.nan
    row[4] = 0
    row[5] *= np.float32(1e-42)
    row[6, :, 32:] *= np.float32(1e-6)
    row[7, :, :32] = np.sign(row[7, :, :32]) * g.uniform(0, 3e38, (2, 32)).astype(np.float32)
    row[8, :, 33:] = 0
    row[9] = np.float32(-3.0)
    row[10, :, ::2] = 0.5  # ties
    row[11] *= np.float32(2.0 ** -120)
    slots = g.permutation(64 * (T // 64 + 2))[:T].astype(np.int32)
    pages = T // 64 + 2
    want = fresh(pages, 1, D)
    lh.append4(want, row[:, :1], row[:, 1:], None, np.zeros(T, int), "half", slots, D)
    kv = cache4(q, fresh(pages, 1, D), D)
    rd = to_dev(row)
    q.q8k_kv4_append(q.Q8K_F32, rd[:, :1], 2 * D, rd[:, 1:], 2 * D, T, None, None, to_dev(slots), kv)
    got = bytes_of(kv, D)
    # a scale of NaN has no bits of its own
    s = slice(68 * D, None)
    assert_exact(got[..., : 68 * D], want[..., : 68 * D], "codes and factors")
    assert_exact(np.nan_to_num(got[..., s].copy().view(np.float32), nan=-1), np.nan_to_num(want[..., s].copy().view(np.float32), nan=-1), "scales")


def test_append_one_by_one_and_at_once(q):
    D, heads, T = 128, 16, 520
    g, row, pages, slots = append_case(D, "f32", heads, T, 5, scattered=False)
    table = sh.rope_table(g, T, D)
    pos = np.arange(T, dtype=np.int32)
    rd, pd, sd = to_dev_as(row, "f32"), to_dev(pos), to_dev(slots)
    rope = rope_of(q, table, "half")
    want = fresh(pages, heads, D)
    lh.append4(want, row[:, heads: 2 * heads], row[:, 2 * heads:], table, pos, "half", slots, D)
    for cuts in ([0, T], list(range(T + 1)), [0, 1, 3, T]):
        kv = cache4(q, fresh(pages, heads, D), D)
        for a, b in zip(cuts, cuts[1:]):
            q.q8k_kv4_append(q.Q8K_F32, rd[a:b, heads: 2 * heads], 3 * heads * D, rd[a:b, 2 * heads:], 3 * heads * D,
                             b - a, pd[a:b], rope, sd[a:b], kv)
        assert_exact(bytes_of(kv, D), want, f"cuts {cuts[:4]}")


@pytest.mark.parametrize("D,heads,T", [(64, 1, 1), (128, 8, 70), (256, 3, 333), (64, 16, 600), (256, 32, 259), (128, 9, 1000)])
@pytest.mark.parametrize("dtype", sh.DTYPES)
def test_read(q, D, heads, T, dtype):
    import torch

    g = np.random.default_rng(T)
    pages = 20
    raw = lh.random_cache(g, 4, pages, heads, D)
    raw[..., 68 * D:] = np.abs(g.standard_normal((pages, heads, 128))).astype(np.float32).view(np.uint8)
    slots = g.integers(0, pages * 64, T).astype(np.int32)  # repeats are fine
    if T > 3:
        slots[0], slots[1], slots[2] = -5, pages * 64, 2 ** 31 - 1
        slots[T // 2:] = 64 + np.arange(T - T // 2)
    k, ks, v, vs = lh.held(4, raw, slots, D)
    kd = torch.full((T, heads, D), float("nan"), dtype=torch_dtype(dtype), device="cuda")
    vd = kd.clone()
    q.q8k_kv4_read(q_dtype(q, dtype), cache4(q, raw, D), to_dev(slots), T, kd, vd)
    assert_exact(back(kd), round_to(k.astype(np.float32) * ks[..., None], dtype), "keys")
    assert_exact(back(vd), round_to(v.astype(np.float32) * vs[..., None], dtype), "values")


# ---------------------------------------------------------------------- attend
def run_attend(q, raw, table, cu, lens, qx, D, dtype, window=0, rope_table=None, pos=None, pairs="half", extra_rows=2,
               max_len=None, max_q=None, scale=None):
    import torch

    Tq, Hq = qx.shape[0], qx.shape[1]
    kv = cache4(q, raw, D)
    qd = torch.full((Tq + extra_rows, Hq + 3, D), float("nan"), dtype=torch_dtype(dtype), device="cuda")
    qd[:Tq, :Hq] = to_dev_as(qx, dtype)
    out = torch.full((Tq + extra_rows, Hq, D), 7.0, dtype=torch_dtype(dtype), device="cuda")
    ls = torch.full((Tq + extra_rows, Hq), 7.0, device="cuda")
    max_len = int(max(lens)) if max_len is None else max_len
    max_q = int(np.diff(cu).max()) if max_q is None else max_q
    B = len(lens)
    need = q.qattend_kv4_workspace_bytes(kv, Hq, B, Tq + extra_rows, max_q, max_len)
    ws = poisoned(need) if need else None
    pd = to_dev(np.concatenate([pos, np.full(extra_rows, -1, np.int32)])) if pos is not None else None
    q.qattend_kv4(q_dtype(q, dtype), qd, (Hq + 3) * D, Hq, kv, B, to_dev(cu), Tq + extra_rows, max_q, to_dev(table),
                  table.shape[1], to_dev(np.asarray(lens, np.int32)), max_len, D ** -0.5 if scale is None else scale, window,
                  pd, rope_of(q, rope_table, pairs), out, ls, ws, need)
    o, l = back(out), back(ls)
    assert (o[Tq:] == 7.0).all() and (l[Tq:] == 7.0).all(), "rows of no sequence were written"
    return o[:Tq], l[:Tq]


def compare(q, D, dtype, Hq, H, lens, news, window, rot, pairs="half", max_len=None, more_pages=0, seed=0):
    g = np.random.default_rng(sum(lens) + D + seed)
    raw, table, cu = lh.paged(g, 4, D, H, lens, news)
    table = np.concatenate([table, np.full((len(lens), more_pages), -1, np.int32)], 1)
    Tq = int(cu[-1])
    qx = round_to(g.standard_normal((Tq, Hq, D)) * 1.5, dtype)
    rt = sh.rope_table(g, max(lens) + 8, rot) if rot else None
    pos = g.integers(0, max(lens) + 8, Tq).astype(np.int32) if rot else None
    want, lse, bo, bl = lh.attend(4, qx, cu, raw, table, lens, D ** -0.5, window, rt, pos, pairs, D, dtype)
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, dtype, window, rt, pos, pairs, max_len=max_len)
    assert_within(got, want, bo, "out")
    assert_within(gl, lse, bl, "lse")


@pytest.mark.parametrize("D,dtype,Hq,H,lens,news,window,rot,pairs", ATTEND)
def test_attend(q, D, dtype, Hq, H, lens, news, window, rot, pairs):
    compare(q, D, dtype, Hq, H, lens, news, window, rot, pairs)


KINDS = [(64, "f32", 64), (64, "bf16", 16), (64, "bf16", 0), (128, "f16", 128), (128, "bf16", 128), (128, "bf16", 0),
         (256, "f32", 64), (256, "bf16", 256), (256, "bf16", 0)]


@pytest.mark.parametrize("D,dtype,rot", KINDS)
@pytest.mark.parametrize("lens,news,H,max_len,window", [
    # few rows: four workgroups a tile, two, one, eight waves, in chunks
    ([70, 200], [1, 2], 2, 200, 0), ([70, 200], [1, 2], 40, 200, 0), ([70, 200], [1, 2], 66, 900, 0),
    ([70, 200], [1, 2], 150, 200, 0), ([1200, 700], [1, 2], 8, 2200, 0), ([1025, 300], [1, 3], 80, 1025, 500),
    # tiles of 64 rows, whole and in chunks; of 128 rows, whole and in chunks
    ([200, 140], [150, 70], 32, 200, 0), ([900, 300], [65, 33], 16, 2200, 100), ([129, 140], [129, 70], 64, 140, 100),
    ([900, 300], [128, 100], 32, 3200, 0), ([2300, 300], [100, 20], 36, 2300, 0),
])
def test_attend_every_kernel(q, D, dtype, rot, lens, news, H, max_len, window):
    compare(q, D, dtype, H if news[0] > 3 else 3 * H, H, lens, news, window, rot, max_len=max_len, more_pages=55)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("news", [[1, 1], [70, 70]])
def test_attend_smallest_and_largest_factors(q, D, news):
    """Operands down to fp16's subnormal numbers (code * 2^-18) and up to 8 * 31/16, all of them exact."""
    g = np.random.default_rng(D)
    lens = [130, 77]
    raw, table, cu = lh.paged(g, 4, D, 2, lens, news)
    f = raw[..., 64 * D: 68 * D]
    f[:] = g.choice(np.array([0, 1, 2, 15, 16, 17, 0xf0, 0xff], np.uint8), f.shape)
    raw[0::2, :, 64 * D: 66 * D] = g.integers(1, 16, raw[0::2, :, 64 * D: 66 * D].shape)  # pages of nothing else
    qx = g.standard_normal((cu[-1], 4, D)).astype(np.float32) * 1000
    want, lse, bo, bl = lh.attend(4, qx, cu, raw, table, lens, D ** -0.5, 0, None, None, "half", D, "f32")
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, "f32")
    assert_within(got, want, bo, "out")
    assert_within(gl, lse, bl, "lse")


def test_attend_a_page_of_one_value(q):
    """Each operand lane by itself: keys of one nonzero value, queries of another, so that a score is one product."""
    for D in (64, 128, 256):
        raw = np.full((1, 1, lh.record(4, D)), 0, np.uint8)
        g = np.random.default_rng(D)
        x = np.zeros((64, 1, D), np.float32)
        at = g.permutation(max(D, 64))[:64] % D
        x[np.arange(64), 0, at] = g.choice([-1.0, 1.0], 64) * (1 + np.arange(64) / 16)
        v = np.zeros((64, 1, D), np.float32)
        v[np.arange(64), 0, g.permutation(max(D, 64))[:64] % D] = 1 + np.arange(64)
        lh.append4(raw, x, v, None, np.zeros(64, int), "half", np.arange(64), D)
        qx = np.zeros((D, 1, D), np.float32)
        qx[np.arange(D), 0, np.arange(D)] = 8.0
        table, cu = np.zeros((1, 1), np.int32), np.array([0, D], np.int32)
        want, lse, bo, bl = lh.attend(4, qx, cu, raw, table, [64], 1.0, 0, None, None, "half", D, "f32")
        got, gl = run_attend(q, raw, table, cu, [64], qx, D, "f32", scale=1.0)
        assert_within(got, want, bo, f"out {D}")
        assert_within(gl, lse, bl, f"lse {D}")


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "f32"), (256, "f16")])
@pytest.mark.parametrize("news", [[1, 1, 1], [5, 1, 3], [80, 65, 70]])
def test_attend_what_a_row_does_not_see(q, D, dtype, news):
    """Later tokens, those before a window and those of other sequences hold infinite and NaN scales, a page lies
    outside the cache, a sequence is empty."""
    g = np.random.default_rng(D)
    lens = [300, 0, 200]
    news = [news[0], 0, news[2]]
    raw, table, cu = lh.paged(g, 4, D, 2, lens, news)
    window = 150
    s = raw[..., 68 * D:].view(np.float32)
    first = lens[0] - news[0] - window + 1  # what the first row sees begins here
    for j in range(max(0, first - 40), max(0, first)):  # (no row sees these)
        s[table[0, j // 64], :, j % 64] = np.inf
        s[table[0, j // 64], :, 64 + j % 64] = np.nan
    table[2, 1] = 2 ** 24  # a page that selects nothing
    qx = round_to(g.standard_normal((cu[-1], 6, D)), dtype)
    want, lse, bo, bl = lh.attend(4, qx, cu, raw, table, lens, D ** -0.5, window, None, None, "half", D, dtype)
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, dtype, window)
    assert_within(got, want, bo, "out")
    assert_within(gl, lse, bl, "lse")


@pytest.mark.parametrize("D,dtype,H,Hq,lens", [(128, "f32", 2, 8, [4099, 1]), (64, "bf16", 1, 4, [9001]),
                                               (128, "bf16", 8, 8, [2050, 777]), (256, "f32", 1, 2, [3001])])
def test_attend_counts_every_token(q, D, dtype, H, Hq, lens):
    """Keys that are all alike and values that count (token j has 7 at value j % D): a row's result is how many of its
    tokens fall on each value, over their number; one token more or less shows."""
    import serving_tight as st

    g = np.random.default_rng(D)
    raw, table, cu = lh.paged(g, 4, D, H, lens, [1] * len(lens))
    one = np.full(D, 1, np.int8)
    f = np.full(D // 32, 0xf0, np.uint8)
    for b, L in enumerate(lens):
        for j in range(L):
            v = np.zeros(D, np.int8)
            v[j % D] = 7
            for h in range(H):
                lh.put_token(4, raw[table[b, j // 64], h], D, j % 64, one, f, 0.01, v, f, 1.0)
    qx = round_to(g.standard_normal((len(lens), Hq, D)), dtype)
    got, _ = run_attend(q, raw, table, cu, lens, qx, D, dtype)
    for b, L in enumerate(lens):
        want = np.broadcast_to(7.0 * np.bincount(np.arange(L) % D, minlength=D) / L, (Hq, D))
        assert_within(got[b], want, want * st.counting_bound(dtype, D, L), f"sequence {b}")
        # a token more is one more of L / D and a bit: it would show
        assert L == 1 or st.counting_bound(dtype, D, L) * (L // D + 1) < 1


def test_two_caches_do_not_mix(q):
    """A cache of one kind is refused where the other is taken."""
    import torch

    kv8 = q.KVCache(torch.zeros(q.q8k_kv_bytes(1, 1, 64), dtype=torch.uint8, device="cuda"), 1, 1, 64)
    kv4 = q.KVCache(torch.zeros(q.q8k_kv4_bytes(1, 1, 64), dtype=torch.uint8, device="cuda"), 1, 1, 64, bits=4)
    x, s = torch.zeros(1, 1, 64, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="4 bits"):
        q.q8k_kv4_append(q.Q8K_F32, x, 64, x, 64, 1, None, None, s, kv8)
    with pytest.raises(ValueError, match="8 bits"):
        q.q8k_kv_append(q.Q8K_F32, x, 64, x, 64, 1, None, None, s, kv4)
    with pytest.raises(ValueError, match="8 bits"):
        q.q8k_kv_read(q.Q8K_F32, kv4, s, 1, x, x.clone())
