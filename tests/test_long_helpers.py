"""The plain forms of the operators for long contexts, against hand-worked cases
and their own definition (no GPU)."""
import numpy as np
import pytest

import long_helpers as lh


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_every_byte_of_a_record_is_one_tokens(bits, D):
    at = lh.token_bytes(bits, D)
    assert sorted(at.flatten()) == list(range(lh.record(bits, D)))


def test_factors():
    f = lh.FACTORS
    assert f[0] == 0 and f[1] == 2.0 ** -18 and f[16] == 2.0 ** -14 and f[0xf0] == 1.0
    assert (np.diff(f) > 0).all()
    assert np.array_equal(f.astype(np.float16), (np.arange(256, dtype=np.uint16) << 6).view(np.float16))


def test_quantise4_by_hand():
    x = np.zeros((1, 64), np.float32)
    x[0, :4] = [7.0, -3.4, 0.5, 0.51]
    x[0, 32:36] = [3.5, -0.25, 0.26, 1.75]
    c, b, s = lh.quantise4(x)
    assert s[0] == 1.0 and list(b[0]) == [0xf0, 0xe0]  # 1 and 1/2
    assert list(c[0, :4]) == [7, -3, 0, 1] and list(c[0, 32:36]) == [7, 0, 1, 4]
    # 3.5 / 7 + a little: the next factor up, 17/32
    x[0, 32] = np.nextafter(np.float32(3.5), np.float32(4))
    assert lh.quantise4(x)[1][0, 1] == 0xe1


@pytest.mark.parametrize("D", [64, 256])
def test_quantise4_is_within_half_a_step(D):
    g = np.random.default_rng(3)
    x = (g.standard_normal((200, D)) * 10.0 ** g.uniform(-5, 5, (200, 1))).astype(np.float32)
    x[:, :32] *= 10.0 ** g.uniform(-6, 0, (200, 1)).astype(np.float32)
    c, b, s = lh.quantise4(x)
    step = np.repeat(lh.FACTORS[b], 32, -1) * s[:, None]
    assert np.abs(c).max() == 7
    assert (np.abs(c * step - x) <= step * (0.5 + 2.0 ** -20)).all()


def test_quantise4_odd_rows():
    x = np.zeros((5, 64), np.float32)
    x[1, 3], x[1, 40] = np.nan, 2.0
    x[2, 3], x[2, 40] = np.inf, 2.0
    x[3, 0], x[3, 40] = 1e-42, -2e-42  # 1 / step overflows
    x[4, 0], x[4, 40] = 1.0, 1e-8  # below the least factor: still one
    c, b, s = lh.quantise4(x)
    assert not c[0].any() and s[0] == 0
    assert c[1, 3] == 0 and c[1, 40] == 7 and s[1] == np.float32(2.0) / np.float32(7)
    assert not c[2].any() and np.isinf(s[2])
    assert c[3, 0] == 7 and c[3, 40] == -7
    assert b[4, 1] == 1 and c[4, 40] == 0


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_token_goes_in_and_comes_out(D):
    g = np.random.default_rng(D)
    x, y = g.standard_normal((2, 64, 1, D)).astype(np.float32)
    cache = np.zeros((1, 1, lh.record(4, D)), np.uint8)
    lh.append4(cache, x, y, None, np.zeros(64, int), "half", np.arange(64)[::-1], D)
    k, ks, v, vs = lh.held(4, cache, np.arange(64)[::-1], D)
    for t in (0, 5, 63):  # byte by byte, the same
        one = lh.get_token(4, cache[0, 0], D, 63 - t)
        assert all(np.array_equal(a, b[t, 0]) for a, b in zip(one, (k, ks, v, vs)))
    for got, s, want in ((k, ks, x), (v, vs, y)):
        c, b, sc = lh.quantise4(want)
        assert np.array_equal(got, c * np.repeat(lh.FACTORS[b], 32, -1)) and np.array_equal(s, sc)


def test_choose_by_hand():
    w = np.array([5, 1, 3, 3, np.nan, -np.inf, 3, 0, 9, 2], np.float32)
    assert list(lh.choose(w, 10, 10, 0, 0)) == list(range(10))
    assert list(lh.choose(w, 10, 4, 1, 1)) == [0, 2, 8, 9]
    assert list(lh.choose(w, 10, 5, 1, 1)) == [0, 2, 3, 8, 9]
    assert list(lh.choose(w, 10, 9, 0, 0)) == [0, 1, 2, 3, 5, 6, 7, 8, 9]
    assert list(lh.choose(w, 10, 2, 0, 2)) == [8, 9]
    assert list(lh.choose(w, 4, 2, 2, 0)) == [0, 1]
