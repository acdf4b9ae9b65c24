"""The operators for long contexts as they are used together, on the GPU: a prompt
in chunks into the cache, attention over it, what its tokens gathered, eviction,
and decoding on; captured graphs, other streams, addresses past 32 bits."""
import numpy as np
import pytest

import long_helpers as lh
import serving_helpers as sh
from gpu_helpers import host, poisoned, to_dev
from serving_helpers import assert_exact, assert_within, back, q_dtype, round_to, to_dev_as, torch_dtype
from test_gpu_serving import rope_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_q8kpack_fp32_amd as q

    return lh.tracked(q)


def calls(q, bits):
    if bits == 8:
        return q.q8k_kv_append, q.qattend, q.qattend_workspace_bytes
    return q.q8k_kv4_append, q.qattend_kv4, q.qattend_kv4_workspace_bytes


def append_np(bits, cache, k, v, table, pos, pairs, slots, D):
    (sh.append if bits == 8 else lh.append4)(cache, k, v, table, pos, pairs, slots, D)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_conversation(q, bits, dtype):
    """Two sequences, prompts in two chunks, three rounds of decode steps and an eviction (in place) between them."""
    import torch

    g = np.random.default_rng(bits)
    B, H, G, D, pages, most = 2, 2, 3, 128, 24, 12
    Hq = H * G
    append, attend, need_of = calls(q, bits)
    cache = np.full((pages, H, lh.record(bits, D)), 0x55, np.uint8)
    cache[..., lh.record(bits, D) - 512:] = 0xFF
    kv = q.KVCache(to_dev(cache), pages, H, D, bits=bits)
    page_table = g.permutation(pages).astype(np.int32).reshape(B, most)
    td = to_dev(page_table)
    rope_table = sh.rope_table(g, 1000, 64)
    rope = rope_of(q, rope_table, "half")
    w_np = np.zeros((B, H, most * 64), np.float32)
    wd = torch.zeros(B, H, most * 64, device="cuda")
    lens, at = [0, 0], [0, 0]  # cached tokens, and positions (which eviction does not touch)
    ws = poisoned(1 << 24)

    def step(news):
        cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        Tq = int(cu[-1])
        row = round_to(g.standard_normal((Tq, Hq + 2 * H, D)), dtype)
        pos = np.concatenate([np.arange(at[b], at[b] + news[b]) for b in range(B)]).astype(np.int32)
        slots = np.concatenate([[page_table[b, j // 64] * 64 + j % 64 for j in range(lens[b], lens[b] + news[b])]
                                for b in range(B)]).astype(np.int32)
        for b in range(B):
            lens[b] += news[b]
            at[b] += news[b]
        rd, pd, ld = to_dev_as(row, dtype), to_dev(pos), to_dev(np.array(lens, np.int32))
        stride = (Hq + 2 * H) * D
        append(q_dtype(q, dtype), rd[:, Hq: Hq + H], stride, rd[:, Hq + H:], stride, Tq, pd, rope, to_dev(slots), kv)
        append_np(bits, cache, row[:, Hq: Hq + H], row[:, Hq + H:], rope_table, pos, "half", slots, D)
        assert_exact(host(kv.data).reshape(cache.shape), cache, "cache")
        out = torch.empty(Tq, Hq, D, dtype=torch_dtype(dtype), device="cuda")
        lse = torch.empty(Tq, Hq, device="cuda")
        need = need_of(kv, Hq, B, Tq, max(news), max(lens))
        args = (q_dtype(q, dtype), rd[:, :Hq], stride, Hq, kv, B, to_dev(cu), Tq, max(news), td, most, ld, max(lens),
                D ** -0.5, 0, pd, rope)
        attend(*args, out, lse, ws, need)
        plain = (row[:, :Hq], cu, cache, page_table, lens, D ** -0.5, 0, rope_table, pos, "half", D)
        want, wl, bo, bl = lh.attend(bits, *plain, dtype)
        assert_within(back(out), want, bo, "out")
        assert_within(back(lse), wl, bl, "lse")
        need = q.qattend_weights_workspace_bytes(kv, Hq, B, Tq, max(news), max(lens))
        q.qattend_weights(*args, lse, wd, 0.75, wd, most * 64, ws, need)
        ww, wb = lh.weights(bits, *plain, back(lse), w_np, 0.75)
        got = back(wd)
        for b in range(B):
            assert_within(got[b, :, : lens[b]], ww[b, :, : lens[b]], wb[b, :, : lens[b]], f"weights {b}")
        w_np[:] = got

    def evict(budget, first, last):
        kept = torch.empty(B, H, budget, dtype=torch.int32, device="cuda")
        new = torch.empty(B, dtype=torch.int32, device="cuda")
        q.q8k_kv_evict(kv, B, td, most, to_dev(np.array(lens, np.int32)), max(lens), wd, most * 64, budget, first, last, td,
                       most, wd, most * 64, kept, new)
        after, k, ow, n = lh.evict(bits, cache, page_table, lens, w_np, budget, first, last, page_table, D)
        cache[:] = after
        w_np[..., :budget] = np.where(k >= 0, ow, w_np[..., :budget])
        lens[:] = [int(x) for x in n]
        assert_exact(host(kept), k, "kept")
        assert_exact(host(new), n, "new lengths")
        assert_exact(host(kv.data).reshape(cache.shape), cache, "cache after eviction")
        assert np.array_equal(host(wd), w_np)

    step([200, 130])
    step([150, 40])
    evict(160, 4, 40)
    for _ in range(2):
        step([1, 1])
    evict(160, 4, 40)  # one over the budget, and one not
    step([5, 1])
    evict(64, 0, 64)  # the last ones only
    step([1, 1])


@pytest.mark.parametrize("bits", [8, 4])
def test_captured_steps_share_a_workspace(q, bits):
    """A decode step and a chunk, captured once each over one workspace, replayed as the sequences grow, with eager work
    between; every replay gives what the eager calls give."""
    import torch

    g = np.random.default_rng(3)
    B, H, G, D, dtype = 3, 2, 4, 64, "f32"
    append, attend, need_of = calls(q, bits)
    most = 40
    raw, table, _ = lh.paged(g, bits, D, H, [most * 64] * B, [1] * B)
    kv = q.KVCache(to_dev(raw), raw.shape[0], H, D, bits=bits)
    td = to_dev(table)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    out_table = to_dev(g.permutation(raw.shape[0])[: B * 8].astype(np.int32).reshape(B, 8))
    steps = []
    need = max(max(need_of(kv, H * G, B, B * n, n, most * 64), q.qattend_weights_workspace_bytes(kv, H * G, B, B * n, n, most * 64))
               for n in (1, 70))
    assert need > 0
    ws = poisoned(need)
    for n in (1, 70):
        x = to_dev(g.standard_normal((B * n, H * G, D)).astype(np.float32))
        cu = to_dev((np.arange(B + 1) * n).astype(np.int32))
        out, lse = torch.zeros(B * n, H * G, D, device="cuda"), torch.zeros(B * n, H * G, device="cuda")
        w, ow = torch.zeros(B, H, most * 64, device="cuda"), torch.zeros(B, H, 500, device="cuda")
        kept, new = torch.zeros(B, H, 500, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")

        def run(n=n, x=x, cu=cu, out=out, lse=lse, w=w, ow=ow, kept=kept, new=new):
            args = (q.Q8K_F32, x, H * G * D, H * G, kv, B, cu, B * n, n, td, most, lens, most * 64, D ** -0.5, 0, None, None)
            attend(*args, out, lse, ws, need)
            q.qattend_weights(*args, lse, None, 1.0, w, most * 64, ws, need)
            q.q8k_kv_evict(kv, B, td, most, lens, most * 64, w, most * 64, 500, 4, 60, out_table, 8, ow, 500, kept, new)

        steps.append((run, (out, lse, w, ow, kept, new)))
    # (the moves go to pages of the same cache: other ones than the sequences use at these lengths)
    used = set(table[:, :25].reshape(-1).tolist())
    free = [p for p in range(raw.shape[0]) if p not in used][: B * 8]
    out_table.copy_(torch.tensor(free, dtype=torch.int32).view(B, 8))
    lens.copy_(torch.tensor([700, 1500, 80], dtype=torch.int32))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for run, _ in steps:
            run()
    torch.cuda.synchronize()
    graphs = []
    for run, _ in steps:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        graphs.append(graph)
    for now in ([700, 1500, 80], [1, 0, 1600], [513, 1599, 501], [70, 71, 900]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        for (run, outs), graph in zip(steps, graphs):
            for o in outs:
                o.zero_()
            run()
            torch.cuda.synchronize()
            want, pages = [o.clone() for o in outs], kv.data.clone()
            for _ in range(2):
                for o in outs:
                    o.zero_()
                graph.replay()
                torch.cuda.synchronize()
                for a, b in zip(outs, want):
                    assert torch.equal(a.view(torch.int32), b.view(torch.int32))
                assert torch.equal(kv.data, pages)


@pytest.mark.parametrize("bits", [8, 4])
def test_on_another_stream_and_two_at_once(q, bits):
    import torch

    g = np.random.default_rng(4)
    D, H, G, L = 128, 2, 4, 1200
    append, attend, need_of = calls(q, bits)
    raw, table, cu = lh.paged(g, bits, D, H, [L], [1])
    table = np.concatenate([table, np.full((1, 30), -1, np.int32)], 1)
    kv, td, cud = q.KVCache(to_dev(raw), raw.shape[0], H, D, bits=bits), to_dev(table), to_dev(cu)
    lens = to_dev(np.array([L], np.int32))
    xs = [to_dev(g.standard_normal((1, H * G, D)).astype(np.float32)) for _ in range(2)]
    need = need_of(kv, H * G, 1, 1, 1, 3000)

    def run(x, stream=None):
        out, lse = torch.zeros(1, H * G, D, device="cuda"), torch.zeros(1, H * G, device="cuda")
        w = torch.zeros(1, H, 3000, device="cuda")
        kept, new = torch.zeros(1, H, 300, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        moved = q.KVCache(kv.data.clone(), raw.shape[0], H, D, bits=bits)
        ws = poisoned(max(need, 16))
        torch.cuda.synchronize()
        args = (q.Q8K_F32, x, H * G * D, H * G, kv, 1, cud, 1, 1, td, table.shape[1], lens, 3000, D ** -0.5, 0, None, None)
        attend(*args, out, lse, ws, need, stream=stream)
        q.qattend_weights(*args, lse, None, 1.0, w, 3000, stream=stream)
        q.q8k_kv_evict(moved, 1, td, table.shape[1], lens, 3000, w, 3000, 300, 4, 30, td, table.shape[1], w, 3000, kept, new,
                       stream=stream)
        return out, lse, w, kept, new, moved.data, ws

    want = [run(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        got = [run(x, s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for i in range(6):
                assert torch.equal(a[i], b[i]), i


@pytest.mark.parametrize("bits,heads,D", [(4, 3, 256), (8, 2, 128)])
def test_addresses_past_32_bits(q, bits, heads, D):
    """A cache of more than 2^32 bytes: tokens on its last pages."""
    import torch

    g = np.random.default_rng(5)
    rec = lh.record(bits, D)
    pages = 2 ** 32 // (rec * heads) + 5
    data = torch.zeros(pages * heads * rec, dtype=torch.uint8, device="cuda")
    kv = q.KVCache(data, pages, heads, D, bits=bits)
    append, attend, need_of = calls(q, bits)
    read = q.q8k_kv_read if bits == 8 else q.q8k_kv4_read
    x = g.standard_normal((100, 2 * heads, D)).astype(np.float32)
    last = [pages - 1, pages - 3]
    slots = np.concatenate([last[0] * 64 + np.arange(64), last[1] * 64 + np.arange(36)]).astype(np.int32)
    rd = to_dev(x)
    append(q.Q8K_F32, rd[:, :heads], 2 * heads * D, rd[:, heads:], 2 * heads * D, 100, None, None, to_dev(slots), kv)
    small = np.zeros((2, heads, rec), np.uint8)
    own = np.concatenate([np.arange(64), 64 + np.arange(36)]).astype(np.int32)
    append_np(bits, small, x[:, :heads], x[:, heads:], None, np.zeros(100, int), "half", own, D)
    view = data.view(pages, heads, rec)
    for i in range(2):
        assert_exact(host(view[last[i]]), small[i], f"page {i}")
    assert int(view[:4].sum()) == 0 and int(view[pages // 2].sum()) == 0
    k, v = torch.zeros(100, heads, D, device="cuda"), torch.zeros(100, heads, D, device="cuda")
    read(q.Q8K_F32, kv, to_dev(slots), 100, k, v)
    kc, ks, vc, vs = lh.held(bits, small, own, D)
    assert_exact(back(k), kc.astype(np.float32) * ks[..., None], "keys")
    assert_exact(back(v), vc.astype(np.float32) * vs[..., None], "values")
    qx = g.standard_normal((1, heads, D)).astype(np.float32)
    table, near = np.array([last], np.int32), np.array([[0, 1]], np.int32)
    cu = np.array([0, 1], np.int32)
    plain = (qx, cu, small, near, [100], D ** -0.5, 0, None, None, "half", D)
    want, wl, bo, bl = lh.attend(bits, *plain, "f32")
    out, lse = torch.zeros(1, heads, D, device="cuda"), torch.zeros(1, heads, device="cuda")
    args = (q.Q8K_F32, to_dev(qx), heads * D, heads, kv, 1, to_dev(cu), 1, 1, to_dev(table), 2, to_dev(np.array([100], np.int32)),
            100, D ** -0.5, 0, None, None)
    attend(*args, out, lse)
    assert_within(back(out), want, bo, "out")
    w = torch.zeros(1, heads, 100, device="cuda")
    q.qattend_weights(*args, lse, None, 1.0, w, 100)
    ww, wb = lh.weights(bits, *plain, back(lse), None, 1.0)
    assert_within(back(w), ww, wb, "weights")
    kept, new = torch.zeros(1, heads, 40, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    to = np.array([[pages - 2]], np.int32)
    q.q8k_kv_evict(kv, 1, to_dev(table), 2, to_dev(np.array([100], np.int32)), 100, w, 100, 40, 2, 8, to_dev(to), 1, None, 0,
                   kept, new)
    three = np.concatenate([small, np.zeros((1, heads, rec), np.uint8)])
    after, kk, _, _ = lh.evict(bits, three, near, [100], back(w), 40, 2, 8, np.array([[2]], np.int32), D)
    assert_exact(host(kept), kk, "kept")
    assert_exact(host(view[pages - 2]), after[2], "the new page")
