"""The serving operators within tolerances that one token or one logit more or
less exceeds (serving_tight.py)."""
import numpy as np
import pytest

import census
import serving_helpers as sh
import serving_tight as tight
from serving_helpers import assert_exact, assert_within, round_to
from test_gpu_serving import attend_case, check_logprobs, q, run_attend, run_logprobs  # noqa: F401  (q is the fixture)
from test_gpu_serving_unseen import FEW, MANY

pytestmark = pytest.mark.gpu

# ------------------------------------------------------------ log probabilities
# in one round of 256 and of 1024 threads, cut into parts, and whole in several rounds
ROWS = [(5, 7), (5, 500), (3, 8191), (3, 8193), (4, 32001), (2, 32769), (2, 70001), (1, 131073), (100, 40003), (260, 40003),
        (260, 66001), (300, 1003)]


@pytest.mark.parametrize("T,V", ROWS)
@pytest.mark.parametrize("dtype", sh.DTYPES)
def test_logprobs(q, T, V, dtype):
    g = np.random.default_rng(T * V)
    x = round_to(g.standard_normal((T, V)) * 2, dtype)
    x[0, : V // 2] = -np.inf
    t = g.integers(0, V, T).astype(np.int32)
    n = min(V, 9)
    check_logprobs(run_logprobs(q, x, dtype, t, n, stride=V + V % 3), tight.logprobs(x, t, n), f"{T} {V} {dtype}")


@pytest.mark.parametrize("T,V", ROWS)
def test_logprobs_of_equal_logits(q, T, V):
    """One logit left out or counted twice changes lse by 1 / V."""
    level = np.array([0.0, -3.0, 2.0])[np.arange(T) % 3]
    x = np.repeat(level[:, None], V, 1).astype(np.float32)
    t = np.full(T, V - 1, np.int32)
    got = run_logprobs(q, x, "f32", t, 0)
    bound = tight.even_rows(V, 3.0)
    assert bound < 0.5 / V or V > 2 ** 20
    assert_within(got["lse"], level + np.log(V), bound, "lse")
    assert_within(got["entropy"], np.full(T, np.log(V)), bound, "entropy")
    assert_within(got["logprob"], np.full(T, -np.log(V)), 2 * bound, "logprob")


@pytest.mark.parametrize("whole,V", [(False, 70001), (False, 32771), (False, 131071), (True, 40003), (True, 66007), (False, 8190),
                                     (False, 31999)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_logprobs_at_the_edges(q, whole, V, dtype):
    """Most of a row's mass in one logit, at every place where the walk through the row has a border."""
    cut = V > tight.ROUND and not whole
    at = tight.edges(V, tight.part_length(100, V) if cut else 4096)
    at = (at * (1 + 100 // len(at)))[:100] if not whole else (at * (1 + 260 // len(at)))[:max(260, len(at))]
    T = len(at)
    assert T <= 128 if cut else T >= 100
    g = np.random.default_rng(V)
    x = round_to(g.standard_normal((T, V)), dtype)
    x[np.arange(T), at] = 14.0
    t = np.array(at, np.int32)
    want = tight.logprobs(x, t, 3)
    assert np.array_equal(want["top_ids"][:, 0], t)
    check_logprobs(run_logprobs(q, x, dtype, t, 3), want, f"{V} {dtype}")


def rank(x, n):
    """Ids by (logit descending, id ascending), NaN behind every number."""
    order = [sorted(np.flatnonzero(~np.isnan(r)), key=lambda i: (-r[i], i))[:n] if (~np.isnan(r)).sum() < 50 else
             list(np.argsort(-np.where(np.isnan(r), -np.inf, r), kind="stable")[: 4 * n]) for r in x]
    out = []
    for r, o in zip(x, order):
        o = [i for i in o if not np.isnan(r[i])][:n]
        o += [i for i in np.flatnonzero(np.isnan(r))[:n]][: n - len(o)]
        out.append(o)
    return np.array(out, np.int32)


@pytest.mark.parametrize("T,V", [(40, 70001), (3, 32769), (260, 70001), (260, 32769), (20, 20000), (20, 5000)])
@pytest.mark.parametrize("n", [0, 6])
def test_logprobs_of_odd_rows(q, T, V, n):
    """NaN, +inf and rows of nothing, in the first, a middle and the last round or part, beside ordinary rows."""
    g = np.random.default_rng(T + V)
    x = g.standard_normal((T, V)).astype(np.float32)
    places = [0, V // 2, V - 1]
    odd = []
    for r in range(min(T, 20)):
        p = places[r % 3]
        kind = r // 3
        if kind == 0:
            x[r, p] = np.nan
        elif kind == 1:
            x[r, p] = np.inf
        elif kind == 2:
            x[r] = -np.inf
        elif kind == 3:
            x[r, :] = np.nan
            x[r, p] = 1.0
        elif kind == 4:
            x[r, p], x[r, V - 1 - p // 2] = np.nan, np.inf
        elif kind == 5:
            x[r] = -np.inf
            x[r, p] = np.nan
        else:
            continue
        odd.append(r)
    t = g.integers(0, V, T).astype(np.int32)
    t[1::7] = V  # outside: NaN
    got = run_logprobs(q, x, "f32", t, n)
    fine = [r for r in range(T) if r not in odd or r // 3 == 2]
    want = tight.logprobs(x[fine], t[fine], n)
    check_logprobs({k: v[fine] for k, v in got.items()}, want, "rows beside")
    rest = [r for r in odd if r // 3 != 2]
    for k in ("logprob", "lse", "entropy"):
        assert np.isnan(got[k][rest]).all(), k
    if n:
        assert np.isnan(got["top_logprob"][rest]).all()
        assert_exact(got["top_ids"][rest], rank(x[rest], n), "ids of odd rows")


# -------------------------------------------------------------------- attention
SHAPES = [(D, dtype, H, group, lens, news, None) for D, dtype, H, group, lens, news in FEW] + \
         [(D, dtype, H, group, lens, news, most) for D, dtype in ((64, "f32"), (128, "bf16"), (128, "f32"), (256, "f32"))
          for lens, news, H, group, most in MANY] + \
         [(64, "f32", 1, 1, [64 * k + e for k in (8, 24, 32, 33, 100) for e in (-1, 0, 1)], [1] * 15, None),
          (128, "f32", 1, 2, [20000, 1], [1, 1], None), (256, "f32", 1, 1, [6000, 1537], [3, 1], None),
          (64, "f16", 4, 1, [9000], [65], None)]


@pytest.mark.parametrize("window", [0, 1, 64, 65, 700])
@pytest.mark.parametrize("D,dtype,H,group,lens,news,max_len", SHAPES)
def test_every_token_counts_once(q, D, dtype, H, group, lens, news, max_len, window):
    g = np.random.default_rng(D + sum(lens))
    raw, table = tight.counting_cache(g, D, H, lens)
    if max_len is not None:
        table = np.concatenate([table, np.full((len(lens), -(-max_len // 64) - table.shape[1]), -1, np.int32)], 1)
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    Tq = int(cu[-1])
    qx = round_to(g.standard_normal((Tq, group * H, D)), dtype)
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, dtype, window, None, None, "half", max_len=max_len)
    for b, (L, n) in enumerate(zip(lens, news)):
        rows = slice(cu[b], cu[b + 1])
        want, number = tight.counted(D, L, n, window)
        w = np.broadcast_to(want[:, None], got[rows].shape)
        assert_within(got[rows], w, np.abs(w) * tight.counting_bound(dtype, D, L), f"out of sequence {b}")
        s = qx[rows].astype(np.float64).sum(-1) * np.float64(np.float32(0.01)) * D ** -0.5
        lse = s + np.log(number)[:, None]
        bound = tight.counting_lse_bound(qx[rows], s, L, D)
        assert_within(gl[rows], lse, bound, f"lse of sequence {b}")


@pytest.mark.parametrize("rot", [0, 32])
@pytest.mark.parametrize("D,dtype,H,group,lens,news,max_len", [s for s in SHAPES if s[1] == "f32"])
def test_precision(q, D, dtype, H, group, lens, news, max_len, rot):
    """fp32 results are off by what two fp16 pieces leave, not by what one does."""
    g, raw, table, cu = attend_case(D, H, lens, news, sum(lens))
    if max_len is not None:
        table = np.concatenate([table, np.full((len(lens), -(-max_len // 64) - table.shape[1]), -1, np.int32)], 1)
    sc = raw[..., 128 * D:].view(np.float32)
    sc[..., 64:] = np.where(np.isnan(sc[..., 64:]), np.nan, 1.0).astype(np.float32)
    Tq = int(cu[-1])
    qx = g.standard_normal((Tq, group * H, D)).astype(np.float32)
    rt = sh.rope_table(g, 40, rot) if rot else None
    pos = g.integers(0, 40, Tq).astype(np.int32) if rot else None
    want, lse, _, _ = sh.attend(qx, cu, raw, table, lens, D ** -0.5, 0, rt, pos, "half", D, dtype)
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, dtype, 0, rt, pos, "half", max_len=max_len)
    # queries of variance 1, keys of 73 codes RMS with scales of sqrt((0.2^2 + 0.4 + 2^2) / 3) / 73 RMS
    scores = np.float64(1.22)
    off, limit = tight.rms(got.astype(np.float64), want), tight.rms_limit(scores)
    assert off < limit, (off, limit)
    off, limit = np.sqrt(np.mean(np.square(gl - lse))), tight.rms_limit_lse(scores, lse)
    assert off < limit, (off, limit)
    census.CENSUS.credit()
