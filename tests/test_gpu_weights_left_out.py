"""Accumulated attention weights of rows whose lse is -inf: they add nothing, whatever
the queries and keys they meet hold."""
import numpy as np
import pytest

import long_helpers as lh
from test_gpu_weights import check, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_q8kpack_fp32_amd as q

    return lh.tracked(q)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("odd", ["key", "query"])
@pytest.mark.parametrize("D,G,news", [(64, 4, [1, 2]), (128, 8, [5, 3]), (256, 2, [90, 70])])
def test_rows_of_minus_infinity_add_nothing(q, bits, odd, D, G, news):
    """The last token of each sequence, which its last new token alone sees, has a key of infinite or NaN scale, or the
    last new token's queries are NaN and infinite; that token's rows are left out."""
    g = np.random.default_rng(D)
    lens = [300, 200]
    raw, table, cu = lh.paged(g, bits, D, 2, lens, news)
    qx = g.standard_normal((int(cu[-1]), 2 * G, D)).astype(np.float32)
    args = (qx.copy(), cu, raw.copy(), table, lens, D ** -0.5, 0, None, None, "half", D)
    lse = lh.attend(bits, *args, "f32")[1].astype(np.float32)
    last = cu[1:] - 1
    lse[last] = -np.inf
    old = g.uniform(0, 9, (2, 2, 300)).astype(np.float32)
    want, bound = lh.weights(bits, *args, lse, old, 0.5)
    assert (want[np.arange(2), :, np.array(lens) - 1] == 0).all()
    if odd == "key":
        s = raw[..., lh.record(bits, D) - 512:].view(np.float32)
        for b, scale in enumerate((np.inf, np.nan)):
            j = lens[b] - 1
            s[table[b, j // 64], :, j % 64] = scale
    else:
        qx[last[0]], qx[last[1], :, 3] = np.nan, np.inf
    got = run(q, bits, raw, table, cu, lens, qx, D, "f32", lse, old, 0.5)
    check(got, want, bound, lens)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D,G,news,window", [(64, 4, [3, 2], 100), (128, 8, [5, 3], 70), (256, 2, [90, 70], 65), (64, 1, [1, 1], 1)])
def test_rows_of_nan_reach_what_they_see_alone(q, bits, D, G, news, window):
    """The lse of one query head of the first new token is NaN: so are, for its key head, the tokens of its window."""
    g = np.random.default_rng(D + window)
    lens = [300, 200]
    raw, table, cu = lh.paged(g, bits, D, 2, lens, news)
    qx = g.standard_normal((int(cu[-1]), 2 * G, D)).astype(np.float32)
    args = (qx, cu, raw, table, lens, D ** -0.5, window, None, None, "half", D)
    lse = lh.attend(bits, *args, "f32")[1].astype(np.float32)
    lse[cu[:2], G] = np.nan  # the second key head's first
    want, bound = lh.weights(bits, *args, np.nan_to_num(lse, nan=-np.inf), None, 1.0)
    for b in range(2):
        p = lens[b] - news[b]
        want[b, 1, max(0, p - window + 1): p + 1] = np.nan
    got = run(q, bits, raw, table, cu, lens, qx, D, "f32", lse, window=window)
    check(got, want, bound, lens)
