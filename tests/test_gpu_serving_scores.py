"""Attention scores of every size: rows whose largest scores are so far from
zero that fp32 holds no fraction of them."""
import numpy as np
import pytest

import serving_helpers as sh
import serving_tight as tight
from serving_helpers import assert_within, round_to
from test_gpu_serving import attend_case, q, run_attend  # noqa: F401  (q is the fixture)
from test_gpu_serving_unseen import FEW, MANY

pytestmark = pytest.mark.gpu

SHAPES = [(D, dtype, H, group, lens, news, None) for D, dtype, H, group, lens, news in FEW] + \
         [(D, dtype, H, group, lens, news, most) for D, dtype in ((64, "f32"), (128, "bf16"), (128, "f32"), (256, "f32"))
          for lens, news, H, group, most in MANY]


@pytest.mark.parametrize("size", [2.0 ** 18, 2.0 ** 30, 2.0 ** 60])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("D,dtype,H,group,lens,news,max_len", SHAPES)
def test_far_scores(q, D, dtype, H, group, lens, news, max_len, size, sign):
    """Every key a head holds is one row times the token's scale, so that a query's scores are one number times the
    tokens' scales: near `size` or `-size`, all distinct.  The scale that is largest (smallest for negative scores)
    among those that a row sees is twice (half) the next, and takes the whole probability."""
    g, raw, table, cu = attend_case(D, H, lens, news, sum(lens) + D)
    if max_len is not None:
        table = np.concatenate([table, np.full((len(lens), -(-max_len // 64) - table.shape[1]), -1, np.int32)], 1)
    sc = raw[..., 128 * D:].view(np.float32)
    kc = raw[..., : 64 * D].view(np.int8)
    kc[:] = 1
    for b, L in enumerate(lens):
        for j in range(L):
            # among any row's tokens a last token of a run stands alone: three levels, each twice the one before
            level = 4.0 if j == 0 else 2.0 if j == 1 else 1.0
            sc[table[b, j // 64], :, j % 64] = (level if sign > 0 else 1 / level) * size / 128
    Tq = int(cu[-1])
    qx = np.abs(round_to(g.standard_normal((Tq, group * H, D)), dtype)) + np.float32(0.5)
    qx = round_to(qx * sign, dtype)
    want, lse, bo, bl = sh.attend(qx, cu, raw, table, lens, D ** -0.5, 0, None, None, "half", D, dtype)
    # at least sqrt(D) / 1024 of `size`: D products of 1/2 and a level of 1/4, over 128
    assert np.abs(lse).min() >= size / 128
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, dtype, 0, None, None, "half", max_len=max_len)
    # the token of the largest score alone counts: its value row, within the pieces' and the result's rounding
    for b, n in enumerate(news):
        _, _, vc, vs = sh.held(raw, [table[b, 0] * 64], D)
        v = np.repeat(vc[0].astype(np.float64) * vs[0][:, None], group, 0)
        rows = slice(cu[b], cu[b + 1])
        w = np.broadcast_to(v, want[rows].shape)
        assert np.allclose(want[rows], w, rtol=1e-12, atol=0)
        piece = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -21
        assert_within(got[rows], w, np.abs(w) * (piece + sh.HALF_STEP[dtype] + 8 * 2.0 ** -24), "out")
        # of the sum over D products and four fp32 roundings
        assert_within(gl[rows], lse[rows], np.abs(lse[rows]) * (2.0 ** -21 + (2 * D + 10) * 2.0 ** -24), "lse")


@pytest.mark.parametrize("exponent", [-97, -60, 60, 92])
@pytest.mark.parametrize("D,dtype,H,group,lens,news,max_len", [s for s in SHAPES if s[1] == "f32"])
def test_values_near_the_limits(q, D, dtype, H, group, lens, news, max_len, exponent):
    """Values from 2^-90 to 2^100: codes up to 127 of scales from 2^-97 and to 2^93."""
    g, raw, table, cu = attend_case(D, H, lens, news, sum(lens) + D)
    if max_len is not None:
        table = np.concatenate([table, np.full((len(lens), -(-max_len // 64) - table.shape[1]), -1, np.int32)], 1)
    sc = raw[..., 128 * D:].view(np.float32)[..., 64:]
    sc[:] = np.where(np.isnan(sc), np.nan, g.uniform(1, 2, sc.shape) * 2.0 ** exponent).astype(np.float32)
    Tq = int(cu[-1])
    qx = round_to(g.standard_normal((Tq, group * H, D)), dtype)
    want, lse, bo, bl = sh.attend(qx, cu, raw, table, lens, D ** -0.5, 0, None, None, "half", D, dtype)
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, dtype, 0, None, None, "half", max_len=max_len)
    assert_within(got, want, bo, "out")
    assert_within(gl, lse, bl, "lse")
    assert tight.rms(got.astype(np.float64) * 2.0 ** -exponent, want * 2.0 ** -exponent) < tight.rms_limit(np.float64(1.22))


@pytest.mark.parametrize("size", [2.0 ** -99, 2.0 ** 99])
@pytest.mark.parametrize("D,dtype,H,group,lens,news,max_len", [s for s in SHAPES if s[1] == "f32"])
def test_queries_and_keys_near_the_limits(q, D, dtype, H, group, lens, news, max_len, size):
    """Queries of 2^99 over keys as much smaller, and the other way round: ordinary scores."""
    g, raw, table, cu = attend_case(D, H, lens, news, sum(lens) + D)
    if max_len is not None:
        table = np.concatenate([table, np.full((len(lens), -(-max_len // 64) - table.shape[1]), -1, np.int32)], 1)
    sc = raw[..., 128 * D:].view(np.float32)
    sc[..., :64] *= np.float32(1 / size)
    Tq = int(cu[-1])
    qx = round_to(np.clip(g.standard_normal((Tq, group * H, D)), -1.9, 1.9) * size, dtype)
    want, lse, bo, bl = sh.attend(qx, cu, raw, table, lens, D ** -0.5, 0, None, None, "half", D, dtype)
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, dtype, 0, None, None, "half", max_len=max_len)
    assert_within(got, want, bo, "out")
    assert_within(gl, lse, bl, "lse")
