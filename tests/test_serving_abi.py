"""Refusals and sizing of the cache, attention and log probability calls on the
CPU: every bad argument is refused by name before the GPU is touched, and
nothing is enqueued."""
import pytest

import serving_helpers as sh

A16 = 1 << 20  # an aligned fake device address: never dereferenced (refused first)


@pytest.fixture(scope="module")
def q():
    import quantized_q8kpack_fp32_amd as q

    return q


def refused(q, status, fn, *args):
    with pytest.raises(q.Q8KError) as ei:
        fn(*args)
    assert ei.value.name == status, str(ei.value)
    assert q.q8k_debug_last_launches() == []
    return str(ei.value)


def test_kv_bytes(q):
    assert q.q8k_kv_bytes(3, 8, 128) == 3 * 8 * sh.record(128) == 3 * 8 * 16896
    assert q.q8k_kv_bytes(1, 1, 64) == 64 * 128 + 512
    assert q.q8k_kv_bytes(0, 1, 256) == 0
    for bad in ((1, 1, 96), (1, 1, 0), (-1, 1, 64), (1, 0, 64), ((1 << 24) + 1, 1, 64), (1, 4097, 64)):
        assert q.q8k_kv_bytes(*bad) == 0, bad


def test_places_are_a_permutation(q):
    assert sorted(sh.place(t) for t in range(64)) == list(range(64))


def kv(q, data=A16, pages=4, heads=2, dim=64):
    return q.KVCache(data, pages, heads, dim)


def app(q, dtype=0, k=A16, ks=128, v=A16, vs=128, T=1, pos=A16, rope=None, slots=A16, cache=None):
    q.q8k_kv_append(dtype, k, ks, v, vs, T, pos, rope, slots, cache or kv(q), 0)


def test_append_refusals(q):
    assert "dtype=7" in refused(q, "Q8K_ERR_ARG", lambda: app(q, dtype=7))
    assert "head_dim=96" in refused(q, "Q8K_ERR_SHAPE", lambda: app(q, cache=kv(q, dim=96)))
    refused(q, "Q8K_ERR_SHAPE", lambda: app(q, cache=kv(q, heads=0)))
    refused(q, "Q8K_ERR_SHAPE", lambda: app(q, cache=kv(q, pages=-1)))
    refused(q, "Q8K_ERR_SHAPE", lambda: app(q, cache=kv(q, pages=(1 << 24) + 1)))
    refused(q, "Q8K_ERR_NULL", lambda: app(q, cache=kv(q, data=None)))
    refused(q, "Q8K_ERR_ALIGN", lambda: app(q, cache=kv(q, data=A16 + 8)))
    refused(q, "Q8K_ERR_SHAPE", lambda: app(q, T=-1))
    assert "k_stride=120" in refused(q, "Q8K_ERR_SHAPE", lambda: app(q, ks=120))
    refused(q, "Q8K_ERR_SHAPE", lambda: app(q, ks=132))  # not a multiple of 8
    refused(q, "Q8K_ERR_SHAPE", lambda: app(q, vs=0))
    refused(q, "Q8K_ERR_NULL", lambda: app(q, k=None))
    refused(q, "Q8K_ERR_NULL", lambda: app(q, slots=None))
    refused(q, "Q8K_ERR_ALIGN", lambda: app(q, v=A16 + 4))
    refused(q, "Q8K_ERR_ALIGN", lambda: app(q, slots=A16 + 2))
    R = lambda **k: q.Rope(**{**dict(table=A16, positions=8, dim=64, pairs=0), **k})  # noqa: E731
    refused(q, "Q8K_ERR_NULL", lambda: app(q, pos=None, rope=R()))
    refused(q, "Q8K_ERR_NULL", lambda: app(q, rope=R(table=None)))
    refused(q, "Q8K_ERR_SHAPE", lambda: app(q, rope=R(dim=12)))
    refused(q, "Q8K_ERR_SHAPE", lambda: app(q, rope=R(dim=72)))  # more than head_dim
    refused(q, "Q8K_ERR_SHAPE", lambda: app(q, rope=R(dim=0)))
    refused(q, "Q8K_ERR_SHAPE", lambda: app(q, rope=R(positions=0)))
    refused(q, "Q8K_ERR_ARG", lambda: app(q, rope=R(pairs=2)))
    app(q, T=0)  # nothing to do
    app(q, cache=kv(q, pages=0))  # no page: every slot is outside
    assert q.q8k_debug_last_launches() == []


def test_read_refusals(q):
    f = q.q8k_kv_read
    refused(q, "Q8K_ERR_ARG", f, -1, kv(q), A16, 1, A16, A16, 0)
    refused(q, "Q8K_ERR_SHAPE", f, 0, kv(q, dim=32), A16, 1, A16, A16, 0)
    refused(q, "Q8K_ERR_SHAPE", f, 0, kv(q), A16, -1, A16, A16, 0)
    refused(q, "Q8K_ERR_NULL", f, 0, kv(q), None, 1, A16, A16, 0)
    refused(q, "Q8K_ERR_ALIGN", f, 0, kv(q), A16, 1, A16 + 8, A16, 0)
    f(0, kv(q), A16, 0, A16, A16, 0)


def att(q, dtype=0, qp=A16, qs=256, heads=4, cache=None, B=2, cu=A16, Tq=2, max_q=1, table=A16, max_pages=4, lens=A16,
        max_len=200, scale=0.1, window=0, pos=None, rope=None, out=A16, lse=None, ws=A16, wsb=1 << 40):
    q.qattend(dtype, qp, qs, heads, cache or kv(q), B, cu, Tq, max_q, table, max_pages, lens, max_len, scale, window,
              pos, rope, out, lse, ws, wsb, 0)


def test_attend_refusals(q):
    refused(q, "Q8K_ERR_ARG", lambda: att(q, dtype=3))
    assert "q_heads=3" in refused(q, "Q8K_ERR_SHAPE", lambda: att(q, heads=3))
    refused(q, "Q8K_ERR_SHAPE", lambda: att(q, heads=0))
    refused(q, "Q8K_ERR_SHAPE", lambda: att(q, cache=kv(q, dim=80)))
    refused(q, "Q8K_ERR_SHAPE", lambda: att(q, B=-1))
    refused(q, "Q8K_ERR_SHAPE", lambda: att(q, Tq=-1))
    refused(q, "Q8K_ERR_SHAPE", lambda: att(q, max_q=3))  # more than Tq
    refused(q, "Q8K_ERR_SHAPE", lambda: att(q, max_len=-1))
    msg = refused(q, "Q8K_ERR_SHAPE", lambda: att(q, cache=kv(q, heads=1), heads=4096, qs=1 << 18, Tq=1 << 20, max_q=1 << 20))
    assert "2^30" in msg
    assert "257" in refused(q, "Q8K_ERR_SHAPE", lambda: att(q, max_len=257))  # 4 pages hold 256
    refused(q, "Q8K_ERR_SHAPE", lambda: att(q, window=-1))
    refused(q, "Q8K_ERR_ARG", lambda: att(q, scale=float("inf")))
    refused(q, "Q8K_ERR_ARG", lambda: att(q, scale=float("nan")))
    refused(q, "Q8K_ERR_SHAPE", lambda: att(q, qs=248))
    refused(q, "Q8K_ERR_SHAPE", lambda: att(q, qs=260))
    for name in ("qp", "cu", "table", "lens", "out"):
        refused(q, "Q8K_ERR_NULL", lambda: att(q, **{name: None}))
    refused(q, "Q8K_ERR_ALIGN", lambda: att(q, qp=A16 + 8))
    refused(q, "Q8K_ERR_ALIGN", lambda: att(q, out=A16 + 4))
    refused(q, "Q8K_ERR_ALIGN", lambda: att(q, lse=A16 + 2))
    refused(q, "Q8K_ERR_NULL", lambda: att(q, rope=q.Rope(A16, 8, 64, 0)))  # a rotation without positions
    need = q.qattend_workspace_bytes(kv(q, pages=400), 4, 2, 2, 1, 20000)
    assert need > 0
    big = dict(cache=kv(q, pages=400), max_pages=400, max_len=20000)
    refused(q, "Q8K_ERR_WORKSPACE", lambda: att(q, wsb=need - 1, **big))
    refused(q, "Q8K_ERR_NULL", lambda: att(q, ws=None, **big))
    refused(q, "Q8K_ERR_ALIGN", lambda: att(q, ws=A16 + 8, **big))
    att(q, B=0)
    att(q, Tq=0, max_q=0)


def test_attend_workspace_is_bounded(q):
    """The parts' results take no more than one item a tile and the 512 items
    that fill the device, whatever the lengths: a call captured for a million
    tokens costs no more than one for ten thousand."""
    for B in (1, 3, 64, 256, 1000):
        for n in (1, 5, 8, 9, 700):
            c = kv(q, heads=8, dim=128)
            rows = 16 if 4 * n <= 32 else 128
            tiles = B * -(-4 * n // rows)
            last = 0
            for length in (n, 4000, 10000, 1 << 20):
                need = q.qattend_workspace_bytes(c, 32, B, B * n, n, length)
                assert last <= need <= (tiles + 64) * 8 * rows * (128 * 4 + 8) + 256, (B, n, length)
                last = need
    assert q.qattend_workspace_bytes(kv(q, heads=8, dim=128), 32, 1, 1, 1, 64) == 0
    bad = kv(q, dim=72)
    assert q.qattend_workspace_bytes(bad, 4, 1, 1, 1, 100) == 0
    assert q.qattend_workspace_bytes(kv(q), 3, 1, 1, 1, 100) == 0


def lps(q, dtype=0, x=A16, stride=100, T=2, V=100, targets=A16, lp=A16, ent=None, lse=None, n=0, ids=None, tl=None,
        ws=A16, wsb=1 << 40):
    q.qlogprobs(dtype, x, stride, T, V, targets, lp, ent, lse, n, ids, tl, ws, wsb, 0)


def test_logprobs_refusals(q):
    refused(q, "Q8K_ERR_ARG", lambda: lps(q, dtype=9))
    refused(q, "Q8K_ERR_SHAPE", lambda: lps(q, T=-1))
    refused(q, "Q8K_ERR_SHAPE", lambda: lps(q, V=0))
    refused(q, "Q8K_ERR_SHAPE", lambda: lps(q, V=(1 << 20) + 1, stride=1 << 21))
    assert "stride=99" in refused(q, "Q8K_ERR_SHAPE", lambda: lps(q, stride=99))
    refused(q, "Q8K_ERR_ARG", lambda: lps(q, n=-1))
    refused(q, "Q8K_ERR_ARG", lambda: lps(q, n=33, ids=A16, tl=A16))
    refused(q, "Q8K_ERR_ARG", lambda: lps(q, V=4, n=5, ids=A16, tl=A16))
    refused(q, "Q8K_ERR_NULL", lambda: lps(q, x=None))
    refused(q, "Q8K_ERR_NULL", lambda: lps(q, lp=None))  # targets without logprob
    refused(q, "Q8K_ERR_NULL", lambda: lps(q, targets=None))
    refused(q, "Q8K_ERR_NULL", lambda: lps(q, n=3, tl=A16))
    refused(q, "Q8K_ERR_NULL", lambda: lps(q, n=3, ids=A16))
    refused(q, "Q8K_ERR_ALIGN", lambda: lps(q, x=A16 + 2))
    refused(q, "Q8K_ERR_ALIGN", lambda: lps(q, dtype=2, x=A16 + 1))
    refused(q, "Q8K_ERR_ALIGN", lambda: lps(q, ent=A16 + 2))
    # few long rows are cut into parts, whose results meet in the workspace
    assert q.qlogprobs_workspace_bytes(2, 32768, 4) == 0 and q.qlogprobs_workspace_bytes(300, 200000, 4) == 0
    need = q.qlogprobs_workspace_bytes(2, 40000, 4)
    assert 0 < need <= 2 * 16 * (12 + 4 * 8) + 256
    big = dict(V=40000, stride=40000, n=4, ids=A16, tl=A16)
    refused(q, "Q8K_ERR_WORKSPACE", lambda: lps(q, wsb=need - 1, **big))
    refused(q, "Q8K_ERR_NULL", lambda: lps(q, ws=None, **big))
    refused(q, "Q8K_ERR_ALIGN", lambda: lps(q, ws=A16 + 8, **big))
    lps(q, T=0)
    assert q.qlogprobs_workspace_bytes(0, 100, 4) == 0 and q.qlogprobs_workspace_bytes(1, 3, 4) == 0


def test_binding_checks_tensors(q):
    import torch

    with pytest.raises(ValueError):
        q.KVCache(torch.zeros(100, dtype=torch.uint8), 1, 1, 64)
    with pytest.raises(ValueError):
        q.Rope(torch.zeros(4, 64, dtype=torch.float64), 4, 64)
    with pytest.raises(ValueError):
        q.Rope(torch.zeros(4, 64), 5, 64)
    with pytest.raises(TypeError):
        app(q, slots=torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="slots must be contiguous"):
        app(q, slots=torch.zeros(4, 2, dtype=torch.int32)[:, 0])
    with pytest.raises(ValueError, match="page_table must be contiguous"):
        att(q, table=torch.zeros(2, 8, dtype=torch.int32)[:, :4])
    with pytest.raises(TypeError):
        att(q, lse=torch.zeros(2, 4, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="top_ids must be contiguous"):
        lps(q, n=2, ids=torch.zeros(2, 4, dtype=torch.int32)[:, :2], tl=A16)
