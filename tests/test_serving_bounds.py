"""The tolerances of serving_tight.py see the mistakes that they are for: each
is planted in a plain form here, on the CPU."""
import numpy as np
import pytest

import serving_helpers as sh
import serving_tight as tight


@pytest.mark.parametrize("V", [500, 8191, 32001, 70001, 131073])
def test_a_logit_left_out_of_a_row(V):
    assert 1.0 / V > 1.5 * tight.even_rows(V, 3.0)


@pytest.mark.parametrize("V,lost", [(8191, 8), (8193, 8), (32000, 8), (32769, 64), (70001, 64), (131072, 512)])
def test_logits_left_out_of_ordinary_rows(V, lost):
    g = np.random.default_rng(V)
    x = g.standard_normal((3, V)).astype(np.float32) * 2
    t = np.zeros(3, np.int32)
    want = tight.logprobs(x, t, 0)
    x[:, V - lost:] = -np.inf
    got = tight.logprobs(x, t, 0)
    for k in ("lse", "logprob"):
        assert (np.abs(got[k][0] - want[k][0]) > want[k][1]).all(), k


def pieces(x, n):
    """What n fp16 pieces hold of x: one rounded, or one truncated and its rest rounded."""
    x = np.asarray(x, np.float32)
    if n == 1:
        return x.astype(np.float16).astype(np.float64)
    h = x.astype(np.float16).astype(np.float32)
    h = np.where(np.abs(h) > np.abs(x), np.nextafter(h.astype(np.float16), np.float16(0)).astype(np.float32), h)
    return h.astype(np.float64) + (x - h).astype(np.float16).astype(np.float64)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [40, 3333])
def test_one_piece_in_place_of_two(D, n):
    g = np.random.default_rng(n)
    qx = g.standard_normal((20, D)).astype(np.float32)
    k = g.integers(-127, 128, (n, D)) * (g.uniform(0.2, 2.0, (n, 1)) / 73)
    v = g.integers(-127, 128, (n, D)).astype(np.float64)

    def attend(nq, np_, lost=None):
        s = pieces(qx, nq) @ k.T * D ** -0.5
        e = np.exp(s - s.max(-1, keepdims=True))
        z = e.sum(-1, keepdims=True)
        e = pieces(e * 2.0 ** 14, np_) * 2.0 ** -14 if np_ else e
        return e @ v / z

    s = qx.astype(np.float64) @ k.T * D ** -0.5
    e = np.exp(s - s.max(-1, keepdims=True))
    want = e @ v / e.sum(-1, keepdims=True)
    limit = tight.rms_limit(s)
    assert limit < 1.5 * tight.rms_limit(np.float64(1.22))
    assert tight.rms(attend(2, 2), want) < 0.5 * limit
    assert tight.rms(attend(1, 2), want) > 10 * limit
    assert tight.rms(attend(2, 1), want) > 10 * limit


@pytest.mark.parametrize("dtype", sh.DTYPES)
@pytest.mark.parametrize("D,L", [(64, 70), (64, 9000), (128, 5000), (256, 6000)])
def test_a_token_more_or_less(D, L, dtype):
    want, number = tight.counted(D, L, 1, 0)
    bound = want * tight.counting_bound(dtype, D, L)
    for j in (0, 1, L // 2, L - 1):
        for sign in (-1, 1):
            got = (want * number[:, None] + sign * 127.0 * (np.arange(D) == j % D)) / (number[:, None] + sign)
            assert (np.abs(got - want) > 1.5 * bound)[0, j % D], (j, sign)
    # and in lse, whatever the results' type, of a query of ones
    qx = np.ones((1, D))
    assert 1.0 / (L + 1) > 1.2 * tight.counting_lse_bound(qx, 0.01 * D ** 0.5, L, D).max()
