"""Accumulated attention weights on the GPU, over caches of 8 and 4 bits, against a
plain form in 64 bits (long_helpers.weights)."""
import numpy as np
import pytest

import long_helpers as lh
import serving_helpers as sh
from gpu_helpers import poisoned, to_dev
from serving_helpers import assert_within, back, q_dtype, round_to, to_dev_as, torch_dtype
from test_gpu_serving import rope_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_q8kpack_fp32_amd as q

    return lh.tracked(q)


def run(q, bits, raw, table, cu, lens, qx, D, dtype, lse, old=None, keep=1.0, window=0, rope_table=None, pos=None,
        pairs="half", max_len=None, max_q=None, scale=None, stride=None, same=False, extra_rows=1):
    """-> [B][heads][stride] as the call left it, of weights that were 7 everywhere."""
    import torch

    Tq, Hq = qx.shape[0], qx.shape[1]
    B, H = len(lens), raw.shape[1]
    kv = q.KVCache(to_dev(raw), raw.shape[0], H, D, bits=bits)
    qd = torch.full((Tq + extra_rows, Hq + 3, D), float("nan"), dtype=torch_dtype(dtype), device="cuda")
    qd[:Tq, :Hq] = to_dev_as(qx, dtype)
    ls = torch.full((Tq + extra_rows, Hq), float("nan"), device="cuda")
    ls[:Tq] = to_dev(np.ascontiguousarray(lse, np.float32))
    max_len = max([int(n) for n in lens]) if max_len is None else max_len
    max_q = int(np.diff(cu).max(initial=0)) if max_q is None else max_q
    stride = max_len + 5 if stride is None else stride
    w = torch.full((B, H, stride), 7.0, device="cuda")
    od = None
    if old is not None:
        od = w if same else torch.full((B, H, stride), float("nan"), device="cuda")
        od[..., : old.shape[-1]] = to_dev(old.astype(np.float32))
    need = q.qattend_weights_workspace_bytes(kv, Hq, B, Tq + extra_rows, max_q, max_len)
    ws = poisoned(need) if need else None
    pd = to_dev(np.concatenate([pos, np.full(extra_rows, -1, np.int32)])) if pos is not None else None
    q.qattend_weights(q_dtype(q, dtype), qd, (Hq + 3) * D, Hq, kv, B, to_dev(cu), Tq + extra_rows, max_q, to_dev(table),
                      table.shape[1], to_dev(np.asarray(lens, np.int32)), max_len, D ** -0.5 if scale is None else scale,
                      window, pd, rope_of(q, rope_table, pairs), ls, od, keep, w, stride, ws, need)
    return back(w)


def check(got, want, bound, lens, what="", rest=7.0):
    for b, L in enumerate(lens):
        assert_within(got[b, :, :L], want[b, :, :L], bound[b, :, :L], f"{what} sequence {b}")
        if rest is not None:
            assert (got[b, :, L:] == rest).all(), f"{what}: written behind sequence {b}"


def compare(q, bits, D, dtype, Hq, H, lens, news, window, rot, pairs="half", keep=None, max_len=None, seed=0, more_pages=0,
            same=False):
    g = np.random.default_rng(sum(lens) + D + seed)
    raw, table, cu = lh.paged(g, bits, D, H, lens, news)
    table = np.concatenate([table, np.full((len(lens), more_pages), -1, np.int32)], 1)
    Tq = int(cu[-1])
    qx = round_to(g.standard_normal((Tq, Hq, D)) * 1.5, dtype)
    rt = sh.rope_table(g, max(lens) + 8, rot) if rot else None
    pos = g.integers(0, max(lens) + 8, Tq).astype(np.int32) if rot else None
    args = (qx, cu, raw, table, lens, D ** -0.5, window, rt, pos, pairs, D)
    lse = lh.attend(bits, *args, dtype)[1].astype(np.float32)
    old = g.uniform(0, 9, (len(lens), H, max(lens))).astype(np.float32) if keep is not None else None
    want, bound = lh.weights(bits, *args, lse, old, keep)
    got = run(q, bits, raw, table, cu, lens, qx, D, dtype, lse, old, 1.0 if keep is None else keep, window, rt, pos, pairs,
              max_len=max_len, same=same)
    check(got, want, bound, lens, rest=None if same else 7.0)


CASES = [
    # D, dtype, q_heads, heads, lens, new tokens, window, rot, pairs, keep
    (128, "f32", 4, 1, [1], [1], 0, 128, "half", None),
    (128, "f32", 32, 8, [65], [1], 0, 128, "half", 1.0),
    (64, "f32", 1, 1, [63, 64, 65, 1, 0, 128], [1, 1, 1, 1, 0, 1], 0, 64, "adjacent", 0.5),
    (128, "f32", 8, 2, [513, 0, 200, 3], [1, 0, 0, 1], 0, 128, "adjacent", 1.0),  # one with nothing new
    (256, "f32", 6, 2, [300, 17], [1, 3], 0, 256, "half", None),
    (128, "bf16", 8, 1, [700, 64], [2, 1], 0, 64, "half", -0.25),
    (64, "f16", 16, 16, [190, 64, 5], [5, 4, 5], 100, 32, "half", 1.0),
    (128, "f32", 12, 4, [333, 129], [7, 1], 1, 0, "half", 0.0),
    (64, "bf16", 7, 1, [90], [3], 63, 8, "adjacent", None),
    (256, "f16", 2, 2, [130, 20], [20, 20], 64, 128, "adjacent", 2.0),
    (256, "bf16", 24, 1, [257], [1], 0, 0, "half", 1.0),
    (64, "bf16", 3, 1, [600], [40], 0, 0, "half", None),
    (128, "f32", 4, 2, [3, 2], [5, 2], 0, 0, "half", 1.0),  # more new tokens than length
    (128, "f32", 4, 1, [5000, 777], [1, 2], 0, 128, "half", 0.9),
    (64, "f32", 8, 2, [4000], [2], 500, 64, "half", 1.0),
    (128, "f32", 8, 2, [200, 333], [200, 70], 0, 128, "half", None),
    (128, "bf16", 4, 4, [257, 64], [130, 64], 0, 128, "adjacent", 0.5),
    (64, "f16", 8, 1, [150], [150], 40, 64, "half", 1.0),
    (256, "bf16", 4, 2, [190, 1], [150, 1], 0, 256, "half", None),
    (256, "f32", 8, 1, [300], [300], 0, 0, "half", 1.0),
    (64, "bf16", 64, 2, [1100, 900], [64, 33], 0, 0, "half", None),
    (128, "bf16", 32, 8, [1500, 300], [64, 64], 0, 0, "half", 1.0),
    (256, "bf16", 16, 1, [900], [100], 400, 0, "half", 1.0),
]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D,dtype,Hq,H,lens,news,window,rot,pairs,keep", CASES)
def test_weights(q, bits, D, dtype, Hq, H, lens, news, window, rot, pairs, keep):
    compare(q, bits, D, dtype, Hq, H, lens, news, window, rot, pairs, keep)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D,dtype,rot", [(64, "f32", 64), (64, "bf16", 0), (128, "f16", 64), (128, "bf16", 0),
                                         (256, "f32", 0), (256, "bf16", 0)])
@pytest.mark.parametrize("lens,news,H,G,max_len", [
    ([70, 200], [1, 2], 2, 4, 2000), ([2500, 90, 700], [1, 1, 1], 2, 1, 2500), ([600, 300], [17, 40], 1, 4, 900), ([600, 300], [3, 12], 2, 4, 900),
    ([1000], [200], 1, 8, 1000), ([130, 250, 77], [130, 70, 77], 4, 2, 300),
])
def test_weights_few_and_many_rows(q, bits, D, dtype, rot, lens, news, H, G, max_len):
    compare(q, bits, D, dtype, G * H, H, lens, news, 0, rot, keep=1.0, max_len=max_len, more_pages=40)


@pytest.mark.parametrize("bits", [8, 4])
def test_weights_in_place(q, bits):
    """old and weights in one buffer; what the new tokens' places held is not read."""
    g = np.random.default_rng(1)
    lens, news, D = [400, 130], [3, 130], 128
    raw, table, cu = lh.paged(g, bits, D, 2, lens, news)
    qx = g.standard_normal((cu[-1], 4, D)).astype(np.float32)
    args = (qx, cu, raw, table, lens, D ** -0.5, 0, None, None, "half", D)
    lse = lh.attend(bits, *args, "f32")[1].astype(np.float32)
    old = g.uniform(0, 9, (2, 2, 400)).astype(np.float32)
    for b in range(2):
        old[b, :, lens[b] - news[b]:] = np.nan
    want, bound = lh.weights(bits, *args, lse, old, 0.5)
    got = run(q, bits, raw, table, cu, lens, qx, D, "f32", lse, old, 0.5, same=True)
    check(got, want, bound, lens, rest=None)
    assert np.isnan(got[1, :, 130:400]).all(), "written behind the sequence"


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("news", [[2, 1], [90, 70]])
def test_weights_rows_and_tokens_that_do_not_count(q, bits, news):
    """Rows of lse -inf, rows beyond max_q, a page outside the cache, infinite and NaN scales of tokens that no row
    sees; one that a row sees is NaN in its own place alone."""
    g = np.random.default_rng(7)
    D, lens, window = 64, [400, 300], 120
    raw, table, cu = lh.paged(g, bits, D, 1, lens, news)
    s = raw[..., lh.record(bits, D) - 512:].view(np.float32)
    s[table[0, 1], :, 3], s[table[0, 1], :, 4] = np.nan, np.inf  # before every window
    seen = lens[1] - news[1] - 20
    s[table[1, seen // 64], :, seen % 64] = np.nan
    table[1, 3] = -7
    if seen // 64 == 3:
        seen = None
    qx = g.standard_normal((cu[-1], 6, D)).astype(np.float32)
    served = news[0] - 1
    args = (qx, cu, raw, table, lens, D ** -0.5, window, None, None, "half", D)
    lse = np.nan_to_num(g.uniform(2, 4, (cu[-1], 6))).astype(np.float32)
    lse[0, 2] = lse[-1, 1] = -np.inf
    want, bound = lh.weights(bits, *args, lse, None, 1.0, served=served)
    got = run(q, bits, raw, table, cu, lens, qx, D, "f32", lse, window=window, max_q=served)
    bad = np.zeros(want.shape, bool)
    if seen is not None:
        bad[1, :, seen] = True
        assert np.isnan(got[1, :, seen]).all()
    check(np.where(bad[..., : lens[0]], 0, got[..., : lens[0]]), np.where(bad, 0, np.nan_to_num(want, nan=0)), bound, [300, 300], rest=None)
    check(got[:1], want[:1], bound[:1], lens[:1])


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D,dtype,G,n,L", [(128, "f32", 4, 1, 3000), (64, "bf16", 8, 64, 1500), (128, "bf16", 8, 300, 1200)])
def test_weights_count_every_row(q, bits, D, dtype, G, n, L):
    """Keys that are all alike and lse of log(number of tokens): token j gets sum over the rows that see it of 1/their
    number; a row more or less shows."""
    g = np.random.default_rng(D)
    raw, table, cu = lh.paged(g, bits, D, 1, [L], [n])
    one, f = np.full(D, 1, np.int8), np.full(D // 32, 0xf0, np.uint8)
    for j in range(L):
        lh.put_token(bits, raw[table[0, j // 64], 0], D, j % 64, one, f, 0.01, one, f, 1.0)
    qx = round_to(g.standard_normal((n, G, D)), dtype)
    score = qx.astype(np.float64).sum(-1) * np.float64(np.float32(0.01)) * D ** -0.5
    number = L - n + 1 + np.arange(n)
    lse = (score + np.log(number)[:, None]).astype(np.float32)
    p = np.exp(score - lse.astype(np.float64))
    want = np.array([p[max(0, j - (L - n)):].sum() for j in range(L)])
    S = np.abs(qx.astype(np.float64)).sum(-1).max() * 0.01 * D ** -0.5
    # a score's pieces and its sum, lse's product and the exponent's rounding, and a lane's share of the rows one after
    # another: a sixteenth, rounded alike at every addition, then four additions over the lanes and the splits' sum
    rel = S * (2.0 ** -21 + 16 * 2.0 ** -24) + np.abs(lse).max() * 2.0 ** -22 + 2.0 ** -22 + (n * G / 16 + 24) * 2.0 ** -24
    assert rel * n * G < 0.5
    got = run(q, bits, raw, table, cu, [L], qx, D, dtype, lse)
    assert_within(got[0, 0, :L], want, want * rel, "weights")


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("n", [1, 100])
def test_weights_are_the_same_every_time(q, bits, n):
    g = np.random.default_rng(2)
    D, lens = 128, [2000, 500]
    raw, table, cu = lh.paged(g, bits, D, 2, lens, [n, n])
    qx = g.standard_normal((2 * n, 8, D)).astype(np.float32)
    lse = g.uniform(5, 8, (2 * n, 8)).astype(np.float32)
    first = run(q, bits, raw, table, cu, lens, qx, D, "f32", lse)
    for _ in range(3):
        assert np.array_equal(run(q, bits, raw, table, cu, lens, qx, D, "f32", lse), first)
