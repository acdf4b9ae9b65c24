"""Refusals and sizing of the operators for long contexts on the CPU: every bad
argument is refused by name before the GPU is touched, and nothing is enqueued;
what the binding refuses of its tensors."""
import pytest
import torch

import long_helpers as lh
from test_serving_abi import A16, q, refused  # noqa: F401  (q is the fixture)


def kv(q, bits=4, data=A16, pages=4, heads=2, dim=64):
    return q.KVCache(data, pages, heads, dim, bits=bits)


def test_kv4_bytes(q):
    assert q.q8k_kv4_bytes(3, 8, 128) == 3 * 8 * lh.record(4, 128) == 3 * 8 * 9216
    assert q.q8k_kv4_bytes(1, 1, 64) == 68 * 64 + 512
    assert q.q8k_kv4_bytes(0, 1, 256) == 0
    for bad in ((1, 1, 96), (1, 1, 0), (-1, 1, 64), (1, 0, 64), ((1 << 24) + 1, 1, 64), (1, 4097, 64)):
        assert q.q8k_kv4_bytes(*bad) == 0, bad


def app(q, dtype=0, k=A16, ks=128, v=A16, vs=128, T=1, pos=A16, rope=None, slots=A16, cache=None):
    q.q8k_kv4_append(dtype, k, ks, v, vs, T, pos, rope, slots, cache or kv(q), 0)


def test_append_refusals(q):
    assert "q8k_kv4_append: dtype=7" in refused(q, "Q8K_ERR_ARG", lambda: app(q, dtype=7))
    refused(q, "Q8K_ERR_SHAPE", lambda: app(q, cache=kv(q, dim=96)))
    refused(q, "Q8K_ERR_SHAPE", lambda: app(q, cache=kv(q, heads=0)))
    refused(q, "Q8K_ERR_SHAPE", lambda: app(q, cache=kv(q, pages=(1 << 24) + 1)))
    refused(q, "Q8K_ERR_NULL", lambda: app(q, cache=kv(q, data=None)))
    refused(q, "Q8K_ERR_ALIGN", lambda: app(q, cache=kv(q, data=A16 + 8)))
    refused(q, "Q8K_ERR_SHAPE", lambda: app(q, T=-1))
    refused(q, "Q8K_ERR_SHAPE", lambda: app(q, ks=120))
    refused(q, "Q8K_ERR_SHAPE", lambda: app(q, vs=132))
    refused(q, "Q8K_ERR_NULL", lambda: app(q, v=None))
    refused(q, "Q8K_ERR_ALIGN", lambda: app(q, k=A16 + 8))
    refused(q, "Q8K_ERR_ALIGN", lambda: app(q, slots=A16 + 2))
    refused(q, "Q8K_ERR_NULL", lambda: app(q, pos=None, rope=q.Rope(A16, 8, 64, 0)))
    refused(q, "Q8K_ERR_SHAPE", lambda: app(q, rope=q.Rope(A16, 8, 72, 0)))
    app(q, T=0)  # nothing to do
    app(q, cache=kv(q, pages=0))  # no page: every slot is outside
    assert q.q8k_debug_last_launches() == []


def test_read_refusals(q):
    f = q.q8k_kv4_read
    refused(q, "Q8K_ERR_ARG", f, -1, kv(q), A16, 1, A16, A16, 0)
    refused(q, "Q8K_ERR_SHAPE", f, 0, kv(q, dim=32), A16, 1, A16, A16, 0)
    refused(q, "Q8K_ERR_SHAPE", f, 0, kv(q), A16, -1, A16, A16, 0)
    refused(q, "Q8K_ERR_NULL", f, 0, kv(q), None, 1, A16, A16, 0)
    refused(q, "Q8K_ERR_ALIGN", f, 0, kv(q), A16, 1, A16 + 8, A16, 0)
    f(0, kv(q), A16, 0, A16, A16, 0)


def att(q, dtype=0, qp=A16, qs=256, heads=4, cache=None, B=2, cu=A16, Tq=2, max_q=1, table=A16, max_pages=4, lens=A16,
        max_len=200, scale=0.1, window=0, pos=None, rope=None, out=A16, lse=None, ws=A16, wsb=1 << 40):
    q.qattend_kv4(dtype, qp, qs, heads, cache or kv(q), B, cu, Tq, max_q, table, max_pages, lens, max_len, scale, window,
                  pos, rope, out, lse, ws, wsb, 0)


def wts(q, bits=4, dtype=0, qp=A16, qs=256, heads=4, cache=None, B=2, cu=A16, Tq=2, max_q=1, table=A16, max_pages=4,
        lens=A16, max_len=200, scale=0.1, window=0, pos=None, rope=None, lse=A16, old=None, keep=1.0, weights=A16,
        stride=200, ws=A16, wsb=1 << 40):
    q.qattend_weights(dtype, qp, qs, heads, cache or kv(q, bits), B, cu, Tq, max_q, table, max_pages, lens, max_len, scale,
                      window, pos, rope, lse, old, keep, weights, stride, ws, wsb, 0)


@pytest.mark.parametrize("call", [att, wts])
def test_attend_and_weights_refusals(q, call):
    name = "qattend_kv4" if call is att else "qattend_weights"
    assert name + ":" in refused(q, "Q8K_ERR_ARG", lambda: call(q, dtype=3))
    assert "q_heads=3" in refused(q, "Q8K_ERR_SHAPE", lambda: call(q, heads=3))
    refused(q, "Q8K_ERR_SHAPE", lambda: call(q, cache=kv(q, dim=80)))
    refused(q, "Q8K_ERR_SHAPE", lambda: call(q, B=-1))
    refused(q, "Q8K_ERR_SHAPE", lambda: call(q, Tq=-1))
    refused(q, "Q8K_ERR_SHAPE", lambda: call(q, max_q=3))
    refused(q, "Q8K_ERR_SHAPE", lambda: call(q, max_len=-1))
    assert "257" in refused(q, "Q8K_ERR_SHAPE", lambda: call(q, max_len=257))  # 4 pages hold 256
    refused(q, "Q8K_ERR_SHAPE", lambda: call(q, window=-1))
    refused(q, "Q8K_ERR_ARG", lambda: call(q, scale=float("inf")))
    refused(q, "Q8K_ERR_SHAPE", lambda: call(q, qs=248))
    for arg in ("qp", "cu", "table", "lens"):
        refused(q, "Q8K_ERR_NULL", lambda: call(q, **{arg: None}))
    refused(q, "Q8K_ERR_ALIGN", lambda: call(q, qp=A16 + 8))
    refused(q, "Q8K_ERR_NULL", lambda: call(q, rope=q.Rope(A16, 8, 64, 0)))
    call(q, B=0)
    call(q, B=0, Tq=0, max_q=0)


def test_attend_workspace(q):
    assert q.qattend_kv4_workspace_bytes(kv(q, heads=8, dim=128), 32, 1, 1, 1, 64) == 0
    need = q.qattend_kv4_workspace_bytes(kv(q, pages=400), 4, 2, 2, 1, 20000)
    assert need > 0
    big = dict(cache=kv(q, pages=400), max_pages=400, max_len=20000)
    refused(q, "Q8K_ERR_WORKSPACE", lambda: att(q, wsb=need - 1, **big))
    refused(q, "Q8K_ERR_NULL", lambda: att(q, ws=None, **big))
    refused(q, "Q8K_ERR_NULL", lambda: att(q, out=None))
    refused(q, "Q8K_ERR_ALIGN", lambda: att(q, lse=A16 + 2))
    assert q.qattend_kv4_workspace_bytes(kv(q, dim=72), 4, 1, 1, 1, 100) == 0


@pytest.mark.parametrize("bits", [8, 4])
def test_weights_refusals(q, bits):
    refused(q, "Q8K_ERR_NULL", lambda: wts(q, bits, lse=None))
    refused(q, "Q8K_ERR_NULL", lambda: wts(q, bits, weights=None))
    refused(q, "Q8K_ERR_ALIGN", lambda: wts(q, bits, old=A16 + 2))
    assert "w_stride=199" in refused(q, "Q8K_ERR_SHAPE", lambda: wts(q, bits, stride=199))
    refused(q, "Q8K_ERR_ARG", lambda: wts(q, bits, keep=float("nan")))
    refused(q, "Q8K_ERR_ARG", lambda: wts(q, bits, keep=float("-inf")))
    # few rows need no workspace, many bring theirs as operands
    assert q.qattend_weights_workspace_bytes(kv(q, bits), 4, 2, 64, 32, 200) == 0
    need = q.qattend_weights_workspace_bytes(kv(q, bits), 4, 2, 100, 50, 200)
    assert need >= 100 * 4 * 64 * 4
    refused(q, "Q8K_ERR_WORKSPACE", lambda: wts(q, bits, Tq=100, max_q=50, wsb=need - 1))
    refused(q, "Q8K_ERR_NULL", lambda: wts(q, bits, Tq=100, max_q=50, ws=None))
    refused(q, "Q8K_ERR_ALIGN", lambda: wts(q, bits, Tq=100, max_q=50, ws=A16 + 4))
    wts(q, bits, max_len=0, stride=0)
    assert q.qattend_weights_workspace_bytes(kv(q, bits, dim=72), 4, 1, 1, 1, 100) == 0
    assert q.qattend_weights_workspace_bytes(kv(q, bits), 3, 1, 1, 1, 100) == 0


def evi(q, bits=4, cache=None, B=2, table=A16, max_pages=4, lens=A16, max_len=200, w=A16, stride=200, budget=100, first=4,
        last=20, out_table=2 * A16, out_pages=2, ow=None, out_stride=0, kept=A16, new=2 * A16):
    q.q8k_kv_evict(cache or kv(q, bits), B, table, max_pages, lens, max_len, w, stride, budget, first, last, out_table,
                   out_pages, ow, out_stride, kept, new, 0)


@pytest.mark.parametrize("bits", [8, 4])
def test_evict_refusals(q, bits):
    E = lambda **k: (lambda: evi(q, bits, **k))  # noqa: E731
    refused(q, "Q8K_ERR_SHAPE", E(cache=kv(q, bits, dim=96)))
    refused(q, "Q8K_ERR_NULL", E(cache=kv(q, bits, data=None)))
    refused(q, "Q8K_ERR_SHAPE", E(B=-1))
    refused(q, "Q8K_ERR_SHAPE", E(max_len=257))
    refused(q, "Q8K_ERR_SHAPE", E(max_pages=-1))
    for bad in (0, -5, 129):  # two pages hold 128
        assert f"budget={bad}" in refused(q, "Q8K_ERR_SHAPE", E(budget=bad))
    for first, last in ((-1, 0), (0, -1), (101, 0), (0, 101), (60, 41), (1 << 62, 1 << 62)):
        refused(q, "Q8K_ERR_ARG", E(first=first, last=last))
    refused(q, "Q8K_ERR_SHAPE", E(stride=199))
    refused(q, "Q8K_ERR_SHAPE", E(ow=A16 + 64, out_stride=99))
    refused(q, "Q8K_ERR_ARG", E(ow=A16, out_stride=201))  # in place: one stride
    refused(q, "Q8K_ERR_ARG", E(out_table=A16, out_pages=3))  # in place: one table
    refused(q, "Q8K_ERR_ARG", E(new=A16))  # new_len is kv_len
    for arg in ("table", "lens", "w", "out_table", "kept", "new"):
        refused(q, "Q8K_ERR_NULL", E(**{arg: None}))
    for arg in ("table", "lens", "w", "out_table", "kept", "new", "ow"):
        refused(q, "Q8K_ERR_ALIGN", E(**{arg: 3 * A16 + 2, "out_stride": 200}))
    refused(q, "Q8K_ERR_SHAPE", E(B=1 << 20, cache=kv(q, bits, heads=4096)))  # more workgroups than a launch has
    evi(q, bits, B=0)
    evi(q, bits, B=0, first=50, last=50)


def test_other_bits_are_refused(q):
    with pytest.raises(ValueError, match="8 or 4 bits"):
        kv(q, bits=5)
    lib = q.lib
    for bits in (0, 16):
        st = lib.q8k_kv_evict(bits, kv(q).ref, 0, A16, 4, A16, 200, A16, 200, 100, 4, 20, 2 * A16, 2, None, 0, A16, 2 * A16, 0)
        assert q.q8k_status_str(st) == "Q8K_ERR_ARG" and f"bits={bits}" in q.q8k_last_error()
        st = lib.qattend_weights(0, bits, A16, 256, 4, kv(q).ref, 0, A16, 2, 1, A16, 4, A16, 200, 0.1, 0, None, None, A16, None,
                                 1.0, A16, 200, None, 0, 0)
        assert q.q8k_status_str(st) == "Q8K_ERR_ARG"


def test_binding_checks_tensors(q):
    with pytest.raises(ValueError):
        q.KVCache(torch.zeros(68 * 64 + 511, dtype=torch.uint8), 1, 1, 64, bits=4)
    q.KVCache(torch.zeros(68 * 64 + 512, dtype=torch.uint8), 1, 1, 64, bits=4)
    for call, bits in ((app, 8), (att, 8)):
        with pytest.raises(ValueError, match="takes a cache of 4 bits, kv is one of 8"):
            call(q, cache=kv(q, bits))
    with pytest.raises(ValueError, match="takes a cache of 8 bits, kv is one of 4"):
        q.q8k_kv_read(0, kv(q), A16, 1, A16, A16, 0)
    with pytest.raises(TypeError):
        wts(q, lse=torch.zeros(2, 4, dtype=torch.float64))
    with pytest.raises(TypeError):
        evi(q, kept=torch.zeros(2, 2, 100, dtype=torch.int64))
    f = torch.zeros
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    for good, bad, call in (
            (f(2, 2, 200), f(2, 2, 199), lambda t: wts(q, B=2, weights=t, stride=t.shape[-1] if t.shape[-1] >= 200 else 200)),
            (f(2, 2, 200), f(3, 200), lambda t: wts(q, weights=t)),
            (f(2, 2, 200), f(2, 2, 400)[..., ::2], lambda t: wts(q, old=t)),
            (f(2, 4), f(7), lambda t: wts(q, lse=t)),
            (f(2, 2, 200), f(2, 200, 2).transpose(1, 2), lambda t: evi(q, w=t)),
            (i(2, 2, 100), i(2, 2, 99), lambda t: evi(q, kept=t)),
            (i(2, 2), i(3), lambda t: evi(q, out_table=t)),
            (i(2), i(1), lambda t: evi(q, new=t)),
            (f(2, 2, 100), f(2, 2, 99), lambda t: evi(q, ow=t, out_stride=100))):
        with pytest.raises(ValueError):
            call(bad)
        with pytest.raises(Exception) as e:  # behind the binding's checks: no such device memory is ever used
            call_refused(q, call, good)
        assert isinstance(e.value, q.Q8KError), e.value


def call_refused(q, call, good):
    """The call with tensors that fit, on a cache whose head_dim the C side refuses."""
    real = kv
    globals()["kv"] = lambda q, bits=4, **k: real(q, bits, **{**k, "data": None})
    try:
        call(good)
    finally:
        globals()["kv"] = real
