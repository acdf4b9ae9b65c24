"""Attention over the 4-bit cache, and its append, at the edges that the 8-bit ones are
held to: values that a row does not see, scores so far from zero that fp32 holds no
fraction of them, magnitudes near the limits, rows of infinities and NaN."""
import numpy as np
import pytest

import long_helpers as lh
import serving_helpers as sh
from gpu_helpers import to_dev
from serving_helpers import assert_exact, assert_within, q_dtype, round_to, to_dev_as
from test_gpu_kv4 import bytes_of, cache4, fresh, q, run_attend  # noqa: F401  (q is the fixture)
from test_gpu_serving import rope_of
from test_gpu_serving_cache import odd_rows
from test_gpu_serving_unseen import FEW, MANY

pytestmark = pytest.mark.gpu

SHAPES = [(D, dtype, H, group, lens, news, None) for D, dtype, H, group, lens, news in FEW] + \
         [(D, dtype, H, group, lens, news, most) for D, dtype in ((64, "f32"), (128, "bf16"), (128, "f32"), (256, "f32"))
          for lens, news, H, group, most in MANY]


def paged_case(D, H, lens, news, seed, max_len):
    g = np.random.default_rng(seed)
    raw, table, cu = lh.paged(g, 4, D, H, lens, news)
    if max_len is not None:
        table = np.concatenate([table, np.full((len(lens), -(-max_len // 64) - table.shape[1]), -1, np.int32)], 1)
    return g, raw, raw[..., 68 * D:].view(np.float32), table, cu


@pytest.mark.parametrize("kind", ["large", "huge", "inf", "nan"])
@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("D,dtype,H,group,lens,news,max_len", SHAPES)
def test_unseen_values(q, D, dtype, H, group, lens, news, max_len, window, kind):  # noqa: F811
    """Values near 1e-12, and of one token a sequence near 1, near 1e24, infinite or NaN: that counts only for the rows
    whose span holds it, which are then not finite."""
    g, raw, sc, table, cu = paged_case(D, H, lens, news, sum(lens) + D + H, max_len)
    sc[..., 64:] *= np.float32(1e-12)
    clean = raw.copy()
    csc = clean[..., 68 * D:].view(np.float32)
    marked = np.zeros(int(cu[-1]), bool)
    value = {"large": 0.2, "huge": 2e23, "inf": np.inf, "nan": np.nan}[kind]
    for b, (L, n) in enumerate(zip(lens, news)):
        j = L - n + n // 2 - (window if window else 0)
        sc[table[b, j // 64], :, 64 + j % 64] = value
        csc[table[b, j // 64], :, 64 + j % 64] = value if np.isfinite(value) else 0
        p = np.arange(L - n, L)
        marked[cu[b]: cu[b + 1]] = sees = (j <= p) & ((j > p - window) if window else True)
        assert not sees.all() and sees.any()
    qx = round_to(g.standard_normal((int(cu[-1]), group * H, D)), dtype)
    want, lse, bo, bl = lh.attend(4, qx, cu, clean, table, lens, D ** -0.5, window, None, None, "half", D, dtype)
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, dtype, window, max_len=max_len)
    assert_within(gl, lse, bl, "lse")
    if not np.isfinite(value):
        assert not np.isfinite(got[marked]).any(), "rows that see it"
        got, want, bo = got[~marked], want[~marked], bo[~marked]
    assert_within(got, want, bo, "out")


@pytest.mark.parametrize("size", [2.0 ** 18, 2.0 ** 30, 2.0 ** 60])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("D,dtype,H,group,lens,news,max_len", SHAPES)
def test_far_scores(q, D, dtype, H, group, lens, news, max_len, size, sign):  # noqa: F811
    """Keys of code 1 and factor 1 and the tokens' scales, so that a query's scores are one number times these: near `size`
    or `-size`.  The first token's, twice the next one's (negative scores: half), takes the whole probability."""
    g, raw, sc, table, cu = paged_case(D, H, lens, news, sum(lens) + D, max_len)
    raw[..., : 32 * D] = 0x66  # 1 + 8 in each four bits, which begin two bits on
    raw[..., 64 * D: 66 * D] = 0xf0
    assert (lh.held(4, raw, [0], D)[0] == 1).all()
    for b, L in enumerate(lens):
        for j in range(L):
            level = 4.0 if j == 0 else 2.0 if j == 1 else 1.0
            sc[table[b, j // 64], :, j % 64] = (level if sign > 0 else 1 / level) * size / 128
    qx = np.abs(round_to(g.standard_normal((int(cu[-1]), group * H, D)), dtype)) + np.float32(0.5)
    qx = round_to(qx * sign, dtype)
    want, lse, _, _ = lh.attend(4, qx, cu, raw, table, lens, D ** -0.5, 0, None, None, "half", D, dtype)
    assert np.abs(lse).min() >= size / 128
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, dtype, max_len=max_len)
    piece = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -21
    for b in range(len(news)):
        _, _, vc, vs = lh.held(4, raw, [table[b, 0] * 64], D)
        v = np.repeat(vc[0] * vs[0][:, None].astype(np.float64), group, 0)
        rows = slice(cu[b], cu[b + 1])
        w = np.broadcast_to(v, want[rows].shape)
        assert np.allclose(want[rows], w, rtol=1e-12, atol=0)
        # fp16 results: half a step of the smallest numbers too
        bound = np.abs(w) * (piece + sh.HALF_STEP[dtype] + 8 * 2.0 ** -24) + (2.0 ** -25 if dtype == "f16" else 0)
        assert_within(got[rows], w, bound, "out")
        # of the sum over D products and four fp32 roundings
        assert_within(gl[rows], lse[rows], np.abs(lse[rows]) * (2.0 ** -21 + (2 * D + 10) * 2.0 ** -24), "lse")


@pytest.mark.parametrize("exponent", [-92, -60, 60, 96])
@pytest.mark.parametrize("D,dtype,H,group,lens,news,max_len", [s for s in SHAPES if s[1] == "f32"])
def test_values_near_the_limits(q, D, dtype, H, group, lens, news, max_len, exponent):  # noqa: F811
    """Rows whose scale times 7 is from 2^-90 to 2^100."""
    g, raw, sc, table, cu = paged_case(D, H, lens, news, sum(lens) + D, max_len)
    v = sc[..., 64:]
    v[:] = np.where(np.isnan(v), np.nan, g.uniform(1, 2, v.shape) * 2.0 ** exponent).astype(np.float32)
    qx = round_to(g.standard_normal((int(cu[-1]), group * H, D)), dtype)
    want, lse, bo, bl = lh.attend(4, qx, cu, raw, table, lens, D ** -0.5, 0, None, None, "half", D, dtype)
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, dtype, max_len=max_len)
    assert_within(got, want, bo, "out")
    assert_within(gl, lse, bl, "lse")


@pytest.mark.parametrize("size", [2.0 ** -97, 2.0 ** 97])
@pytest.mark.parametrize("D,dtype,H,group,lens,news,max_len", [s for s in SHAPES if s[1] == "f32"])
def test_queries_and_keys_near_the_limits(q, D, dtype, H, group, lens, news, max_len, size):  # noqa: F811
    """Queries of 2^97 and more over keys as much smaller, and the other way round: ordinary scores."""
    g, raw, sc, table, cu = paged_case(D, H, lens, news, sum(lens) + D, max_len)
    sc[..., :64] *= np.float32(1 / size)
    qx = round_to(np.clip(g.standard_normal((int(cu[-1]), group * H, D)), -1.9, 1.9) * size, dtype)
    want, lse, bo, bl = lh.attend(4, qx, cu, raw, table, lens, D ** -0.5, 0, None, None, "half", D, dtype)
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, dtype, max_len=max_len)
    assert_within(got, want, bo, "out")
    assert_within(gl, lse, bl, "lse")


@pytest.mark.parametrize("dtype", sh.DTYPES)
@pytest.mark.parametrize("D,heads,T", [(64, 1, 11), (128, 3, 20), (256, 2, 12), (64, 16, 520), (128, 32, 300), (256, 32, 270)])
@pytest.mark.parametrize("pairs", [None, "half", "adjacent"])
def test_append_of_odd_rows(q, D, heads, T, dtype, pairs):  # noqa: F811
    """Of every type, turned and not, in both forms of the kernel."""
    g = np.random.default_rng(T + D)
    k, v = odd_rows(g, T, heads, D, dtype), odd_rows(g, T, heads, D, dtype)
    table = sh.rope_table(g, 50, D // 2) if pairs else None
    pos = g.integers(0, 50, T).astype(np.int32)
    pages = T // 64 + 2
    slots = (5 + np.arange(T)).astype(np.int32)
    want = fresh(pages, heads, D)
    with np.errstate(invalid="ignore"):
        lh.append4(want, k, v, table, pos, pairs or "half", slots, D)
    kv = cache4(q, fresh(pages, heads, D), D)
    on_device = to_dev if dtype == "f32" else (lambda x: to_dev_as(x, dtype))
    q.q8k_kv4_append(q_dtype(q, dtype), on_device(k), heads * D, on_device(v), heads * D, T, to_dev(pos),
                     rope_of(q, table, pairs), to_dev(slots), kv)
    assert_exact(bytes_of(kv, D), want, "cache")
