"""Attention over the 4-bit cache gives the same bits every time, whatever else ran in
between: whole tiles, chunks and their join, rows by sixteens and tiles of them."""
import numpy as np
import pytest

import long_helpers as lh
from serving_helpers import round_to
from test_gpu_kv4 import run_attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_q8kpack_fp32_amd as q

    return lh.tracked(q)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,Hq,H,lens,news", [(128, 8, 2, [5000, 700], [1, 1]), (64, 4, 2, [300, 200], [2, 1]),
                                              (128, 32, 4, [1500, 900], [300, 256]), (256, 8, 8, [600], [200]),
                                              (128, 32, 4, [7000, 6500], [400, 300])])
def test_attend_is_the_same_every_time(q, dtype, D, Hq, H, lens, news):
    import torch

    g = np.random.default_rng(D)
    raw, table, cu = lh.paged(g, 4, D, H, lens, news)
    qx = round_to(g.standard_normal((int(cu[-1]), Hq, D)), dtype)
    first = run_attend(q, raw, table, cu, lens, qx, D, dtype)
    x = torch.randn(1024, 1024, device="cuda")
    for _ in range(4):
        x = torch.tanh(x @ x)
        again = run_attend(q, raw, table, cu, lens, qx, D, dtype)
        assert all(np.array_equal(a, b) for a, b in zip(first, again))
