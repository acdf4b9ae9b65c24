"""Attention rows beside values that they do not see: a token's value row, of
any size, infinite or NaN, counts only for the rows whose span holds it."""
import numpy as np
import pytest

import serving_helpers as sh
from serving_helpers import assert_within, round_to
from test_gpu_serving import attend_case, q, run_attend  # noqa: F401  (q is the fixture)

pytestmark = pytest.mark.gpu


def unseen_case(q, D, dtype, H, group, lens, news, window, kind, max_len=None):
    """Values near 1e-12, and of one token a sequence near 1 (kind "large"), near 1e24 ("huge"), infinite or NaN: the one in
    the middle of the new tokens, which the first of them do not see, or with a window one that leaves it among them."""
    g, raw, table, cu = attend_case(D, H, lens, news, sum(lens) + D + H)
    if max_len is not None:
        table = np.concatenate([table, np.full((len(lens), -(-max_len // 64) - table.shape[1]), -1, np.int32)], 1)
    sc = raw[..., 128 * D:].view(np.float32)
    sc[..., 64:] *= np.float32(1e-12)  # NaN stays NaN where there is no token
    clean = raw.copy()
    csc = clean[..., 128 * D:].view(np.float32)
    Tq = int(cu[-1])
    marked = np.zeros(Tq, bool)
    value = {"large": 0.01, "huge": 1e22, "inf": np.inf, "nan": np.nan}[kind]
    for b, (L, n) in enumerate(zip(lens, news)):
        j = L - n + n // 2 - (window if window else 0)
        sc[table[b, j // 64], :, 64 + j % 64] = value
        csc[table[b, j // 64], :, 64 + j % 64] = value if np.isfinite(value) else 0
        p = np.arange(L - n, L)
        marked[cu[b]: cu[b + 1]] = sees = (j <= p) & ((j > p - window) if window else True)
        assert not sees.all() and sees.any()
    qx = round_to(g.standard_normal((Tq, group * H, D)), dtype)
    want, lse, bo, bl = sh.attend(qx, cu, clean, table, lens, D ** -0.5, window, None, None, "half", D, dtype)
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, dtype, window, None, None, "half", max_len=max_len)
    assert_within(gl, lse, bl, "lse")
    if not np.isfinite(value):
        assert not np.isfinite(got[marked]).any(), "rows that see it"
        got, want, bo = got[~marked], want[~marked], bo[~marked]
    assert_within(got, want, bo, "out")


# sixteen rows a tile: four, two and one workgroups a tile, eight waves, chunks
FEW = [
    (64, "f32", 1, 2, [70], [5]),
    (128, "f32", 2, 4, [70, 130], [3, 5]),
    (128, "bf16", 20, 2, [90, 200], [4, 6]),
    (128, "f32", 70, 1, [90, 200], [4, 6]),
    (64, "bf16", 70, 2, [900, 1010], [4, 6]),
    (128, "f32", 2, 4, [5000, 777], [4, 3]),
    (64, "bf16", 1, 2, [4100], [7]),
    (256, "f32", 2, 4, [300, 129], [3, 2]),
    (256, "bf16", 2, 2, [3000], [6]),
]


@pytest.mark.parametrize("kind", ["large", "huge", "inf", "nan"])
@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("D,dtype,H,group,lens,news", FEW)
def test_few_rows(q, D, dtype, H, group, lens, news, window, kind):
    unseen_case(q, D, dtype, H, group, lens, news, window, kind)


# tiles of 64 rows, whole and in chunks, and of 128, whole and in chunks
MANY = [
    ([200, 140], [150, 70], 32, 1, 200),
    ([330], [140], 8, 4, 330),
    ([900, 300], [65, 33], 16, 1, 2200),
    ([129, 140], [128, 70], 64, 1, 140),
    ([240, 140], [128, 70], 16, 8, 240),
    ([900, 300], [128, 100], 32, 1, 3200),
]


@pytest.mark.parametrize("kind", ["large", "huge", "inf", "nan"])
@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("D,dtype", [(64, "f32"), (64, "bf16"), (128, "f32"), (128, "bf16"), (256, "f32"), (256, "bf16")])
@pytest.mark.parametrize("lens,news,H,group,max_len", MANY)
def test_many_rows(q, D, dtype, H, group, lens, news, window, kind, max_len):
    unseen_case(q, D, dtype, H, group, lens, news, window, kind, max_len)


@pytest.mark.parametrize("kind", ["inf", "nan"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,news,H,group,max_len", MANY + [([70, 130], [3, 5], 2, 4, 130)])
def test_half_precision(q, D, H, group, lens, news, kind, max_len):
    """fp16 results cannot hold values of 1e-12: what the rows that do not see the token have is compared with zeros' bound."""
    unseen_case(q, D, "f16", H, group, lens, news, 0, kind, max_len)
