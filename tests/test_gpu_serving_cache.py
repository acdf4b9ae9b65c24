"""What the cache makes of rows that hold infinities and NaN: q8k_pack's rule."""
import numpy as np
import pytest

import serving_helpers as sh
from gpu_helpers import host, pack_on_device, split_act, to_dev
from serving_helpers import assert_exact, q_dtype, round_to, to_dev_as
from test_gpu_serving import cache_bytes, cache_of, poisoned_cache, q, rope_of  # noqa: F401  (q is the fixture)

pytestmark = pytest.mark.gpu


def quantise(x):
    """The largest magnitude is taken over the numbers (0 without any), a NaN's code is 0, and so are all codes of
    a row with an infinity, whose scale is infinite."""
    x = x.astype(np.float32)
    amax = np.fmax.reduce(np.abs(x), axis=-1, initial=np.float32(0))
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        r = np.rint(x * (np.float32(127.0) / amax)[..., None])
    r = np.where(np.isnan(r), 0, np.clip(r, -127, 127))
    r[amax == 0] = 0
    return r.astype(np.int8), (amax / np.float32(127.0)).astype(np.float32)


def odd_rows(g, T, heads, D, dtype):
    x = round_to(g.standard_normal((T, heads, D)), dtype)
    with np.errstate(invalid="ignore"):
        x[0] = np.nan
        x[1, :, D // 2] = np.nan
        x[2, :, 1:] = np.nan
        x[3, :, 3] = np.inf
        x[4, :, D - 1], x[4, :, 0] = -np.inf, np.nan
        x[5] = -np.inf
        x[6, :, ::2] = np.nan
        x[6, :, 1::2] = 0
    if dtype == "f32":  # NaN of other patterns: their low bits must not become codes
        x.view(np.uint32)[7, :, ::5] = 0x7FC000FF
        x.view(np.uint32)[8, :, ::3] = 0xFFC00080
        x.view(np.uint32)[9] = 0x7FFFFFFF
        x.view(np.uint32)[10, :, 2] = 0x7F800001
    return x


@pytest.mark.parametrize("dtype", sh.DTYPES)
@pytest.mark.parametrize("D,heads,T", [(64, 1, 11), (128, 3, 20), (256, 2, 12), (64, 16, 300), (128, 8, 515), (256, 32, 130)])
@pytest.mark.parametrize("pairs", [None, "half", "adjacent"])
def test_append_of_odd_rows(q, D, heads, T, dtype, pairs):
    g = np.random.default_rng(T + D)
    k, v = odd_rows(g, T, heads, D, dtype), odd_rows(g, T, heads, D, dtype)
    table = sh.rope_table(g, 50, D // 2) if pairs else None
    pos = g.integers(0, 50, T).astype(np.int32)
    pages = T // 64 + 2
    slots = (5 + np.arange(T)).astype(np.int32)
    with np.errstate(invalid="ignore"):
        kq, ks = quantise(sh.rotate(k, table, pos, pairs))
    vq, vs = quantise(v)
    kv = cache_of(q, poisoned_cache(pages, heads, D), D)
    bits = {"f32": lambda x: to_dev(x)}.get(dtype, lambda x: to_dev_as(x, dtype))
    q.q8k_kv_append(q_dtype(q, dtype), bits(k), heads * D, bits(v), heads * D, T, to_dev(pos),
                    rope_of(q, table, pairs), to_dev(slots), kv)
    gk, gks, gv, gvs = sh.held(cache_bytes(kv, pages, heads, D), slots, D)
    assert_exact(gk, kq, "key codes")
    assert_exact(gv, vq, "value codes")
    assert_exact(gks, ks, "key scales")
    assert_exact(gvs, vs, "value scales")


def test_as_the_pack(q):
    """The same rows, as blocks of 256 values, through q8k_pack."""
    T, D = 40, 256
    g = np.random.default_rng(1)
    x = odd_rows(g, T, 1, D, "f32")
    kv = cache_of(q, poisoned_cache(1, 1, D), D)
    xd = to_dev(x)
    q.q8k_kv_append(q.Q8K_F32, xd, D, xd, D, T, None, None, to_dev(np.arange(T, dtype=np.int32)), kv)
    k, ks, v, vs = sh.held(cache_bytes(kv, 1, 1, D), np.arange(T), D)
    xq = pack_on_device(q, x.reshape(T, D))
    codes, d, _ = split_act(q, host(xq), T, D)
    want, scale = quantise(x)
    assert_exact(codes, want[:, 0], "packed codes")
    assert_exact(d[:, 0], scale[:, 0], "packed scales")
    for got in (k, v):
        assert_exact(got[:, 0], codes, "codes")
    for got in (ks, vs):
        assert_exact(got[:, 0], d[:, 0], "scales")
