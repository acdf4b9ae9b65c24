"""Eviction on the GPU, from caches of 8 and 4 bits, against a plain form
(long_helpers.evict): the cache byte for byte, indices and weights exactly."""
import numpy as np
import pytest

import long_helpers as lh
from gpu_helpers import host, to_dev
from serving_helpers import assert_exact

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_q8kpack_fp32_amd as q

    return lh.tracked(q)


def case(g, bits, D, H, lens, budget, in_place, extra=2):
    """A cache of random bytes, the sequences' page table and the new one."""
    per = [-(-n // 64) for n in lens]
    to = -(-budget // 64)
    pages = sum(per) + (0 if in_place else len(lens) * to) + extra
    raw = g.integers(0, 256, (pages, H, lh.record(bits, D)), dtype=np.uint8)
    order = g.permutation(pages).astype(np.int32)
    table = np.full((len(lens), max(per + [to if in_place else 1])), -1, np.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at: at + n]
        at += n
    return raw, table, table if in_place else order[at: at + len(lens) * to].reshape(len(lens), to)


def run(q, bits, raw, table, lens, w, budget, first, last, out_table, D, in_place, own_weights=True, same_weights=False,
        max_len=None):
    import torch

    B, H = len(lens), raw.shape[1]
    kv = q.KVCache(to_dev(raw), raw.shape[0], H, D, bits=bits)
    td = to_dev(table)
    od = td if in_place else to_dev(out_table)
    wd = to_dev(w)
    ow = wd if same_weights else torch.full((B, H, budget + 3), 7.0, device="cuda") if own_weights else None
    kept = torch.full((B, H, budget), -9, dtype=torch.int32, device="cuda")
    new = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    q.q8k_kv_evict(kv, B, td, table.shape[1], to_dev(np.asarray(lens, np.int32)),
                   int(max(lens)) if max_len is None else max_len, wd, w.shape[2], budget, first, last, od, od.shape[1], ow,
                   ow.shape[2] if ow is not None else 0, kept, new)
    return host(kv.data).reshape(raw.shape), host(kept), None if ow is None else host(ow), host(new)


def compare(q, g, bits, D, H, lens, w, budget, first, last, in_place, same_weights=False, max_len=None):
    raw, table, out_table = case(g, bits, D, H, lens, budget, in_place)
    cut = [min(n, max_len) for n in lens] if max_len is not None else lens
    want, kept, ow, new = lh.evict(bits, raw, table, cut, w, budget, first, last, out_table, D)
    got, gk, gw, gn = run(q, bits, raw, table, lens, w, budget, first, last, out_table, D, in_place,
                          same_weights=same_weights, max_len=max_len)
    assert_exact(gk, kept, "kept")
    assert_exact(gn, new, "new lengths")
    assert_exact(got, want, "cache")
    rest = w[..., :budget] if same_weights else np.float32(7)
    if same_weights and rest.shape[2] < budget:
        return
    there = kept >= 0
    assert np.array_equal(np.where(there, gw[..., :budget], 0).view(np.uint32), np.where(there, ow, 0).view(np.uint32))
    assert np.array_equal(np.where(there, 0, gw[..., :budget]).view(np.uint32), np.where(there, 0, rest).astype(np.float32).view(np.uint32))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("D,H,lens,budget,first,last", [
    (64, 1, [2], 1, 0, 0), (64, 1, [1, 0, 3], 2, 1, 1), (128, 2, [65, 64, 63], 64, 0, 0), (128, 3, [200, 70, 130], 100, 4, 20),
    (256, 2, [300, 129], 128, 0, 64), (128, 2, [513], 65, 65, 0), (64, 4, [700, 333], 300, 0, 300), (64, 2, [1500], 1, 0, 1),
    (256, 1, [1100, 40, 1024], 1000, 2, 2), (128, 1, [3000, 2100], 2047, 4, 256), (64, 1, [5000], 777, 4, 100),
    (128, 2, [90, 20], 200, 4, 100),
])
def test_evict(q, bits, in_place, D, H, lens, budget, first, last):
    g = np.random.default_rng(sum(lens) + D)
    w = (g.random((len(lens), H, max(lens) + 3)) ** 8 * 50).astype(np.float32)
    compare(q, g, bits, D, H, lens, w, budget, first, last, in_place)


@pytest.mark.parametrize("bits,D", [(8, 64), (4, 128)])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["equal", "few", "odd", "signs", "digits", "ascending", "descending"])
def test_evict_ties_and_odd_weights(q, bits, D, in_place, kind):
    """Equal weights go by ascending index, NaN below all numbers, -0 as 0; in descending order nothing moves, in
    ascending order everything does."""
    g = np.random.default_rng(5)
    lens, H, budget = [2600, 1025, 300], 2, 500
    shape = (3, H, 2600)
    w = {"equal": np.full(shape, 0.25), "few": g.integers(0, 3, shape) * 1.0,
         "odd": g.choice([np.nan, np.inf, -np.inf, 0.0, -0.0, 1.0, 1e-42, -1.0], shape),
         "signs": g.choice([0.0, -0.0], shape), "digits": g.integers(0, 2 ** 31 - 2 ** 24, shape),
         "ascending": np.broadcast_to(np.arange(2600) * 1.0, shape),
         "descending": np.broadcast_to(3000.0 - np.arange(2600), shape)}[kind].astype(np.float32)
    if kind == "digits":  # bits that differ in one of their four digits
        w = (np.float32(1.5).view(np.uint32) ^ (g.integers(0, 256, shape) << (8 * g.integers(0, 3, shape)))).astype(np.uint32).view(np.float32)
    compare(q, g, bits, D, H, lens, np.ascontiguousarray(w), budget, 4, 60, in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_weights_in_place(q, in_place):
    g = np.random.default_rng(6)
    w = g.random((2, 3, 1700)).astype(np.float32)
    compare(q, g, 4, 64, 3, [1700, 90], w, 600, 4, 50, in_place, same_weights=True)


def test_evict_longer_than_the_limit(q):
    """A length over max_len is cut to it."""
    g = np.random.default_rng(8)
    w = g.random((2, 1, 500)).astype(np.float32)
    compare(q, g, 8, 64, 1, [500, 300], w, 100, 4, 50, False, max_len=400)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_pages_outside_the_cache(q, bits, in_place):
    """Tokens of a page that is none arrive as zeros, those for a new page that is none do not."""
    g = np.random.default_rng(9)
    D, lens, budget = 64, [600, 400], 200
    raw, table, out_table = case(g, bits, D, 2, lens, budget, in_place)
    table[0, 4], table[1, 2] = -1, 2 ** 24
    if not in_place:
        out_table[0, 1] = raw.shape[0]
    w = g.random((2, 2, 600)).astype(np.float32)
    want, kept, _, new = lh.evict(bits, raw, table, lens, w, budget, 4, 20, table if in_place else out_table, D)
    got, gk, _, gn = run(q, bits, raw, table, lens, w, budget, 4, 20, out_table, D, in_place)
    assert_exact(gk, kept, "kept")
    assert_exact(got, want, "cache")


def test_evict_without_weights_out(q):
    g = np.random.default_rng(10)
    raw, table, out_table = case(g, 4, 128, 2, [300], 100, False)
    w = g.random((1, 2, 300)).astype(np.float32)
    want, kept, _, _ = lh.evict(4, raw, table, [300], w, 100, 4, 20, out_table, 128)
    got, gk, gw, _ = run(q, 4, raw, table, [300], w, 100, 4, 20, out_table, 128, False, own_weights=False)
    assert gw is None
    assert_exact(gk, kept, "kept")
    assert_exact(got, want, "cache")
