"""Accumulated attention weights on the GPU under limits far above what the sequences
hold: many sequences, long rows of weights, 2^32 of them in all."""
import numpy as np
import pytest

import long_helpers as lh
from gpu_helpers import poisoned, to_dev
from serving_helpers import assert_within, back, to_dev_as

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_q8kpack_fp32_amd as q

    return lh.tracked(q)


@pytest.mark.parametrize("bits", [8, 4])
def test_weights_of_many_sequences_under_long_limits(q, bits):
    """Rows too few to be cut into shares: the call has no join, whose workgroups (2^32 threads of them here) then
    stand in no one's way.  The last rows of weights lie 2^32 elements on."""
    import torch

    g = np.random.default_rng(bits)
    B, H, G, D, max_q, max_pages = 4096, 8, 8, 64, 9, 2048
    max_len = max_pages * 64
    live = {0: (9, 130), 17: (1, 300), 4095: (8, 65)}  # sequence: new tokens, length
    lens = np.zeros(B, np.int32)
    news = np.zeros(B, np.int64)
    for b, (n, length) in live.items():
        news[b], lens[b] = n, length
    raw, small, cu = lh.paged(g, bits, D, H, [live[b][1] for b in live], [live[b][0] for b in live])
    table = np.full((B, small.shape[1]), -1, np.int32)
    table[list(live)] = small
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    Tq = int(cu[-1])
    qx = g.standard_normal((Tq, H * G, D)).astype(np.float32)
    args = (qx, cu, raw, table, lens, D ** -0.5, 0, None, None, "half", D)
    lse = lh.attend(bits, *args, "f32")[1].astype(np.float32)
    want, bound = lh.weights(bits, *args, lse, None, 1.0)
    kv = q.KVCache(to_dev(raw), raw.shape[0], H, D, bits=bits)
    td = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    td[:, : table.shape[1]] = to_dev(table)
    need = q.qattend_weights_workspace_bytes(kv, H * G, B, Tq, max_q, max_len)
    w = torch.full((B, H, max_len), 7.0, device="cuda")
    q.qattend_weights(q.Q8K_F32, to_dev_as(qx, "f32"), H * G * D, H * G, kv, B, to_dev(cu), Tq, max_q, td, max_pages,
                      to_dev(lens), max_len, D ** -0.5, 0, None, None, to_dev(lse), None, 1.0, w, max_len, poisoned(need),
                      need)
    for b in live:
        got = back(w[b, :, : lens[b] + 64])
        assert_within(got[:, : lens[b]], want[b, :, : lens[b]], bound[b, :, : lens[b]], f"sequence {b}")
        assert (got[:, lens[b]:] == 7).all()
        w[b, :, : lens[b]] = 7.0
    assert bool((w.view(-1)[-(1 << 20):] == 7).all()) and float(w.amax()) == float(w.amin()) == 7.0
