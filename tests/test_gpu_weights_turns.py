"""Accumulated attention weights of few rows where a wave has several pages, one after
another: batches of many key heads over long sequences."""
import os
import re

import numpy as np
import pytest

import long_helpers as lh
import serving_helpers as sh
from serving_helpers import round_to
from test_gpu_weights import check, run

pytestmark = pytest.mark.gpu

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_q8kpack_fp32_amd", "csrc",
                      "attend_weights.hip")


@pytest.fixture(scope="module")
def q():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_q8kpack_fp32_amd as q

    return lh.tracked(q)


def turns(rows, pages):
    """Pages that a wave has at most: four waves a workgroup, as many workgroups a sequence and head as its pages or
    the whole device asks for."""
    text = open(SOURCE).read()
    fill = int(re.search(r"FEW_WGS = (\d+)", text).group(1))
    waves = int(re.search(r"WAVES = (\d+)", text).group(1))
    groups = min(-(-pages // waves), -(-fill // rows))
    return -(-pages // (waves * groups))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D,dtype,rot,B,H,G,n,longest,window,keep", [
    # up to 16 rows a head, whose operand stays in registers
    (64, "f32", 64, 16, 8, 2, 1, 4500, 0, 1.0), (128, "bf16", 0, 32, 4, 4, 2, 2500, 0, None),
    (256, "f16", 128, 64, 2, 1, 1, 2300, 0, 0.5), (64, "bf16", 0, 16, 8, 2, 5, 3000, 1000, 1.0),
    # up to 64, in LDS
    (64, "f32", 64, 16, 8, 4, 5, 4500, 0, 1.0), (128, "bf16", 0, 32, 4, 4, 16, 2500, 0, None),
    (256, "f32", 0, 64, 2, 1, 17, 2300, 0, 0.5), (64, "f16", 32, 16, 8, 8, 6, 3000, 700, 0.9),
])
def test_weights_of_several_turns(q, bits, D, dtype, rot, B, H, G, n, longest, window, keep):
    """A page outside the cache in the first turn and in later ones, lengths that end in any of them."""
    g = np.random.default_rng(D + n)
    lens = [longest] + [int(x) for x in g.integers(n, longest, B - 1)]
    lens[1], lens[2], lens[3] = longest - 1, longest // 2, n
    news = [n] + [int(x) for x in g.integers(0, n + 1, B - 1)]
    pages = -(-longest // 64)
    assert turns(B * H, pages) >= 2
    raw, table, cu = lh.paged(g, bits, D, H, lens, news)
    table[0, 0], table[0, pages - 2], table[1, pages // 2] = -1, 2 ** 24, raw.shape[0]
    qx = round_to(g.standard_normal((int(cu[-1]), H * G, D)) * 1.5, dtype)
    rt = sh.rope_table(g, longest + 8, rot) if rot else None
    pos = g.integers(0, longest + 8, int(cu[-1])).astype(np.int32) if rot else None
    args = (qx, cu, raw, table, lens, D ** -0.5, window, rt, pos, "half", D)
    lse = lh.attend(bits, *args, dtype)[1].astype(np.float32)
    old = g.uniform(0, 9, (B, H, longest)).astype(np.float32) if keep is not None else None
    want, bound = lh.weights(bits, *args, lse, old, keep)
    got = run(q, bits, raw, table, cu, lens, qx, D, dtype, lse, old, 1.0 if keep is None else keep, window, rt, pos)
    check(got, want, bound, lens)
