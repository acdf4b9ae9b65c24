"""Eviction of rows of more weights than a workgroup holds at once (16384): the digits
are counted, and the kept tokens numbered, over several turns."""
import numpy as np
import pytest

import long_helpers as lh
from test_gpu_evict import compare

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_q8kpack_fp32_amd as q

    return lh.tracked(q)


def weights_of(g, kind, shape):
    if kind == "random":
        w = g.random(shape) ** 8 * 50
    elif kind == "equal":
        w = np.full(shape, 0.25)
    elif kind == "few":
        w = g.integers(0, 3, shape) * 1.0
    elif kind == "odd":
        w = g.choice([np.nan, np.inf, -np.inf, 0.0, -0.0, 1.0, 1e-42, -1.0], shape)
    elif kind == "ascending":
        w = np.broadcast_to(np.arange(shape[2]) * 1.0, shape)
    else:  # digits: bits that differ in the top eleven (sign and exponent), the next eleven or the last ten
        low, width = np.array([21, 10, 0]), np.array([11, 11, 10])
        which = g.integers(0, 3, shape)
        change = (g.integers(0, 2048, shape) & ((1 << width[which]) - 1)) << low[which]
        return (np.uint32(0x3fc12345) ^ change.astype(np.uint32)).view(np.float32)
    return np.ascontiguousarray(w.astype(np.float32))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("same_weights", [False, True])
@pytest.mark.parametrize("kind,lens,budget,first,last", [
    ("random", [16384], 700, 4, 60), ("random", [16385, 40000, 300, 16384], 900, 4, 100),
    ("equal", [40000, 16390], 17000, 0, 0),  # the kept ones go on behind the first turn
    ("few", [40000], 20000, 10, 10),  # the border lies among equal ones of the second turn
    ("digits", [33000, 20000], 1500, 0, 0), ("odd", [20000], 15000, 4, 60), ("ascending", [50000], 400, 3, 5),
    ("random", [16385], 600, 0, 500),  # the last ones lie on both sides of a turn's end
    ("random", [20000], 16700, 16500, 20), ("random", [65537], 500, 4, 100), ("few", [17000], 1, 0, 0),
])
def test_evict_long_rows(q, bits, same_weights, kind, lens, budget, first, last):
    """In place where the weights are kept in place, else to other pages."""
    g = np.random.default_rng(sum(lens) + budget)
    w = weights_of(g, kind, (len(lens), 1, max(lens) + 3))
    compare(q, g, bits, 64, 1, lens, w, budget, first, last, same_weights, same_weights=same_weights)


@pytest.mark.parametrize("L,budget", [(1500, 200), (4096, 1000), (9000, 3000)])
def test_evict_every_digit(q, L, budget):
    """Signs, exponents and both ends of the mantissa decide."""
    g = np.random.default_rng(L)
    w = weights_of(g, "digits", (1, 4, L))
    compare(q, g, 4, 64, 4, [L], w, budget, 0, 0, False)
